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
// Bound by memory: every row once in and once out.  The angles of a row are made once
// for all heads of all tensors.
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

// A workgroup takes a row, where there are fewer than this many rows and a wave would not have
// all heads of one in flight at once; otherwise each of its waves does.  40 heads of 128,
// bf16: 256 rows 4.2 us, a wave each 5.5; 1024 6.1 and 6.7; 2048 10.4 and 10.2; 8192 31.9
// and 29.2.  4 heads: 256 rows 3.5 both ways, 2048 6.0 and 3.8.
constexpr int kFewRows = 2048;
// Heads that a thread has in flight at a time.
constexpr int kRopeHeads = 4;

// A row is taken by TPR threads.  Each makes some of the row's angles, which meet in
// LDS; then 2^lanes_shift of them share a head, and P neighbouring pairs are one
// thread's.  The first heads are asked for before the row's position is looked for.
template <RowType T, bool INTERLEAVED, int P, int TPR>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs p, int lanes_shift) {
  typedef typename Elem<T>::type E;
  extern __shared__ float2 angles[];  // [kThreads / TPR][rot / 2]
  const int half = p.rot / 2;
  const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t row = (int64_t)p.row0 + (int64_t)blockIdx.x * (kThreads / TPR) + sub;
  if (row >= p.s.rows) return;  // whole waves
  float2 *mine = angles + sub * half;
  const int turning = half / P;  // threads of a head that turn pairs
  const int chunks = turning + (p.copy ? (p.dim - p.rot + 2 * P - 1) / (2 * P) : 0);  // and that copy the rest
  const int lanes = 1 << lanes_shift, step = TPR >> lanes_shift;
  const int k0 = tid & (lanes - 1), first_head = tid >> lanes_shift;

  // A chunk of a head: two runs of P elements, half a rotation apart or next to each other.
  struct Chunk {
    Run<E, P> u, v;
  };
  auto place = [&](int h, int &n) -> int64_t {  // of head h: its tensor, and the element within the row
    n = 0;
    int h0 = 0;
#pragma unroll
    for (int i = 1; i < kRopeTensors; ++i)
      if (h >= p.upto[i - 1]) {
        n = i;
        h0 = p.upto[i - 1];
      }
    return (int64_t)(h - h0) * p.dim;
  };
  auto source = [&](int h) {
    int n;
    const int64_t at = place(h, n);
    return static_cast<const E *>(p.x[n]) + row * p.x_stride[n] + at;
  };
  auto begin_of = [&](int k) { return k < turning ? (INTERLEAVED ? 2 : 1) * P * k : p.rot + 2 * P * (k - turning); };
  auto second_of = [&](int k) { return k < turning && !INTERLEAVED ? P * k + half : begin_of(k) + P; };
  auto is_whole = [&](int k) { return k < turning || begin_of(k) + 2 * P <= p.dim; };  // else a last piece, by elements
  Chunk x[kRopeHeads];
  auto load = [&](int k, int h0) {
#pragma unroll
    for (int j = 0; j < kRopeHeads; ++j)
      if (h0 + j * step < p.heads) {
        const E *from = source(h0 + j * step);
        x[j].u = *reinterpret_cast<const Run<E, P> *>(from + begin_of(k));
        x[j].v = *reinterpret_cast<const Run<E, P> *>(from + second_of(k));
      }
  };
  if (k0 < chunks && is_whole(k0)) load(k0, first_head);

  int position;
  if (p.positions != nullptr) {
    position = p.positions[row];
  } else {
    const Place at = find_row(p.s, (int)row, threadIdx.x & 63);
    if (!at.found) return;  // no sequence's row: left as it was
    position = (int)((uint32_t)at.seq.length - (uint32_t)at.seq.n + (uint32_t)at.index);
  }
  for (int i = tid; i < half; i += TPR) {
    float c, s;
    angle_of(p.turns[i], position, c, s);
    mine[i] = float2{c * p.amplitude, s * (p.inverse ? -p.amplitude : p.amplitude)};
  }
  if constexpr (TPR == 64) {  // a wave's own: no other waits for it
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }

  for (int k = k0; k < chunks; k += lanes) {
    const int begin = begin_of(k), second = second_of(k);
    const bool turn = k < turning, whole = is_whole(k);
    float2 cs[P];
    if (turn)
#pragma unroll
      for (int i = 0; i < P; ++i) cs[i] = mine[k * P + i];
    for (int h0 = first_head; h0 < p.heads; h0 += kRopeHeads * step) {
      if (whole && (k != k0 || h0 != first_head)) load(k, h0);
#pragma unroll
      for (int j = 0; j < kRopeHeads; ++j) {
        const int h = h0 + j * step;
        if (h >= p.heads) continue;
        int n;
        const int64_t at = place(h, n);
        E *to = static_cast<E *>(p.out[n]) + row * p.out_stride[n] + at;
        if (!whole) {
          const E *from = source(h);
          for (int d = begin; d < p.dim; ++d) to[d] = from[d];
          continue;
        }
        if (turn) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            // The i-th pair: interleaved, of the two runs taken as one.
            E &eu = !INTERLEAVED ? x[j].u.x[i] : 2 * i < P ? x[j].u.x[2 * i % P] : x[j].v.x[2 * i % P];
            E &ev = !INTERLEAVED ? x[j].v.x[i] : 2 * i + 1 < P ? x[j].u.x[(2 * i + 1) % P] : x[j].v.x[(2 * i + 1) % P];
            const float u = Elem<T>::to_float(eu), v = Elem<T>::to_float(ev);
            eu = Elem<T>::from_float(u * cs[i].x - v * cs[i].y);
            ev = Elem<T>::from_float(u * cs[i].y + v * cs[i].x);
          }
        }
        *reinterpret_cast<Run<E, P> *>(to + begin) = x[j].u;
        *reinterpret_cast<Run<E, P> *>(to + second) = x[j].v;
      }
    }
  }
}

template <RowType T, bool INTERLEAVED, int P, int TPR>
hipError_t launch_rows(RopeArgs a, hipStream_t stream) {
  const int threads = a.rot / 2 / P + (a.copy ? (a.dim - a.rot + 2 * P - 1) / (2 * P) : 0);
  int shift = 0;
  while ((1 << shift) < TPR && (1 << shift) < threads) ++shift;
  constexpr int kRows = kThreads / TPR;
  const size_t lds = (size_t)kRows * (a.rot / 2) * sizeof(float2);  // at most 64 KiB
  for (int64_t row0 = 0; row0 < a.s.rows; row0 += (int64_t)kMostGroups * kRows) {
    a.row0 = (int)row0;
    const dim3 grid((unsigned)std::min<int64_t>((a.s.rows - row0 + kRows - 1) / kRows, kMostGroups));
    hipLaunchKernelGGL((rope_kernel<T, INTERLEAVED, P, TPR>), grid, dim3(kThreads), lds, stream, a, shift);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <RowType T, bool INTERLEAVED, int P>
hipError_t launch_pairs(const RopeArgs &a, hipStream_t stream) {
  const bool many_heads = (int64_t)a.heads * (a.rot / 2 / P) > 64 * kRopeHeads;
  if (a.s.rows < kFewRows && many_heads) return launch_rows<T, INTERLEAVED, P, kThreads>(a, stream);
  return launch_rows<T, INTERLEAVED, P, 64>(a, stream);
}

template <RowType T, bool INTERLEAVED>
hipError_t launch_typed(const RopeArgs &a, hipStream_t stream) {
  // Runs of 16 bytes where the pairs come in whole ones.
  constexpr int kWide = T == kRowF32 ? 4 : 8;
  if (a.rot / 2 % kWide == 0) return launch_pairs<T, INTERLEAVED, kWide>(a, stream);
  if (a.rot / 2 % 4 == 0) return launch_pairs<T, INTERLEAVED, 4>(a, stream);
  return launch_pairs<T, INTERLEAVED, 1>(a, stream);
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
