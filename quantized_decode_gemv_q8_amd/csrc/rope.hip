// Rotary positions: pairs of channels of a row at position p turn by p * f_i,
//   (x, y) -> amplitude * (x cos - y sin, x sin + y cos),
// with one frequency per pair; the inverse turns back (which is the gradient).
//
// The angle is exact at any position: a frequency is held as a fraction of a turn
// in 64 bits, and its product with the position, modulo 2^64, is the fraction of a turn
// that is left.  In f32 a position of 100000 would be off by 4e-3 radians.  What is left
// is brought to the nearest quarter turn, and sine and cosine come from their power
// series on |a| <= pi / 4: up to a^9 and a^10, off by less than 2e-9 there.
//
// Bound by memory: every row once in and once out.  A workgroup takes a row; a
// thread makes the angles of its pairs once and takes them through all heads of all
// tensors.
#include <algorithm>

#include "cache_rows.h"
#include "rope.h"

namespace q8 {
namespace {

template <typename E, int N>
struct __attribute__((packed, aligned(sizeof(E)))) Run {
  E x[N];
};

__device__ __forceinline__ void angle_of(uint64_t turns, int position, float &cosine, float &sine) {
  const uint64_t phase = turns * (uint64_t)(int64_t)position;
  const uint32_t top = (uint32_t)(phase >> 32);        // of a turn, in units of 2^-32
  const uint32_t quarter = (top + 0x20000000u) >> 30;  // the nearest one
  const float a = (float)(int32_t)(top - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = a * a;
  const float s = fmaf(a * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), a);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const bool swap = quarter & 1;
  cosine = swap ? s : c;
  sine = swap ? c : s;
  if ((quarter + 1) & 2) cosine = -cosine;  // quarters 1 and 2
  if (quarter & 2) sine = -sine;            // quarters 2 and 3
}

// P: pairs of a thread, neighbouring ones.
template <RowType T, bool INTERLEAVED, int P>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs p, int lanes_shift) {
  typedef typename Elem<T>::type E;
  const uint32_t row = p.row0 + blockIdx.x;  // below rows, by the launcher's grid
  int position;
  if (p.positions != nullptr) {
    position = p.positions[row];
  } else {
    const Place at = find_row(p.s, (int)row, threadIdx.x & 63);
    if (!at.found) return;  // no sequence's row: left as it was
    position = (int)((uint32_t)at.seq.length - (uint32_t)at.seq.n + (uint32_t)at.index);
  }
  const int half = p.rot / 2, turning = half / P;  // threads of a head that turn pairs
  const int tail = p.copy ? (p.dim - p.rot + 2 * P - 1) / (2 * P) : 0;  // and that copy the rest
  const int lanes = 1 << lanes_shift, step = kThreads >> lanes_shift;
  for (int k = threadIdx.x & (lanes - 1); k < turning + tail; k += lanes) {
    const bool turn = k < turning;
    float c[P], s[P];
    if (turn) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        angle_of(p.turns[k * P + i], position, c[i], s[i]);
        c[i] *= p.amplitude;
        s[i] *= p.inverse ? -p.amplitude : p.amplitude;
      }
    }
    for (int h = threadIdx.x >> lanes_shift; h < p.heads; h += step) {
      int n = 0, h0 = 0;
#pragma unroll
      for (int i = 1; i < kRopeTensors; ++i)
        if (h >= p.upto[i - 1]) {
          n = i;
          h0 = p.upto[i - 1];
        }
      const E *x = static_cast<const E *>(p.x[n]) + (int64_t)row * p.x_stride[n] + (int64_t)(h - h0) * p.dim;
      E *out = static_cast<E *>(p.out[n]) + (int64_t)row * p.out_stride[n] + (int64_t)(h - h0) * p.dim;
      if (!turn) {
        const int d0 = p.rot + (k - turning) * 2 * P;
#pragma unroll
        for (int i = 0; i < 2 * P; ++i)
          if (d0 + i < p.dim) out[d0 + i] = x[d0 + i];
      } else if constexpr (INTERLEAVED) {
        const Run<E, 2 * P> in = *reinterpret_cast<const Run<E, 2 * P> *>(x + 2 * P * k);
        Run<E, 2 * P> to;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float u = Elem<T>::to_float(in.x[2 * i]), v = Elem<T>::to_float(in.x[2 * i + 1]);
          to.x[2 * i] = Elem<T>::from_float(u * c[i] - v * s[i]);
          to.x[2 * i + 1] = Elem<T>::from_float(u * s[i] + v * c[i]);
        }
        *reinterpret_cast<Run<E, 2 * P> *>(out + 2 * P * k) = to;
      } else {
        const Run<E, P> iu = *reinterpret_cast<const Run<E, P> *>(x + P * k);
        const Run<E, P> iv = *reinterpret_cast<const Run<E, P> *>(x + half + P * k);
        Run<E, P> ou, ov;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float u = Elem<T>::to_float(iu.x[i]), v = Elem<T>::to_float(iv.x[i]);
          ou.x[i] = Elem<T>::from_float(u * c[i] - v * s[i]);
          ov.x[i] = Elem<T>::from_float(u * s[i] + v * c[i]);
        }
        *reinterpret_cast<Run<E, P> *>(out + P * k) = ou;
        *reinterpret_cast<Run<E, P> *>(out + half + P * k) = ov;
      }
    }
  }
}

template <RowType T, bool INTERLEAVED>
hipError_t launch_typed(const RopeArgs &args, hipStream_t stream) {
  RopeArgs a = args;
  const int pairs = a.rot / 2 % 4 == 0 ? 4 : 1;
  const int threads = a.rot / 2 / pairs + (a.copy ? (a.dim - a.rot + 2 * pairs - 1) / (2 * pairs) : 0);
  int shift = 0;
  while (shift < 8 && (1 << shift) < threads) ++shift;
  for (int64_t row0 = 0; row0 < a.s.rows; row0 += kMostGroups) {
    a.row0 = (int)row0;
    const dim3 grid((unsigned)std::min<int64_t>(a.s.rows - row0, kMostGroups));
    if (pairs == 4)
      hipLaunchKernelGGL((rope_kernel<T, INTERLEAVED, 4>), grid, dim3(kThreads), 0, stream, a, shift);
    else
      hipLaunchKernelGGL((rope_kernel<T, INTERLEAVED, 1>), grid, dim3(kThreads), 0, stream, a, shift);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, RowType type, bool interleaved, hipStream_t stream) {
  switch (type) {
    case kRowF32: return interleaved ? launch_typed<kRowF32, true>(a, stream) : launch_typed<kRowF32, false>(a, stream);
    case kRowBf16: return interleaved ? launch_typed<kRowBf16, true>(a, stream) : launch_typed<kRowBf16, false>(a, stream);
    case kRowF16: return interleaved ? launch_typed<kRowF16, true>(a, stream) : launch_typed<kRowF16, false>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace q8
