// The Q8_0 cache: quantising rows as they are written, reading them back, and
// moving accepted drafts to the front of a sequence's new tokens.
//
// Q8_0 per 32 channels x of a row: s = f32(max|x| / 127), code = x / s rounded
// to the nearest (ties to even), value = code * s.  Every step is exact or
// correctly rounded, so codes and scales do not depend on how the work is
// split:
//   * the scale is one correctly rounded division;
//   * the code is x times the scale's reciprocal, rounded, then corrected by at
//     most one step with the exact remainder x - code * s (a multiple of
//     ulp(s) / 2 no larger than 2 s, so the fused multiply-add that forms it
//     does not round).
// A block that holds an infinity or a NaN has no scale; it is stored as s =
// NaN and reads back as NaN.
//
// All three are bound by memory: they touch each byte once.  A row of dim
// channels belongs to 16 lanes; lane j holds channel pair j of every block,
// which is the cache's pair order, so codes leave (or come) in one access of
// dim / 16 bytes and the row outside in dim / 32 accesses, each of 16
// neighbouring pairs.
#include <algorithm>

#include "cache_rows.h"

namespace q8 {
namespace {

// f32(top / 127) for finite top >= 0.  1 / 127 is 2^-28 from its f32, so the
// product is within an ulp of the quotient and one corrected step rounds it
// correctly; not where the quotient loses bits to denormals.
__device__ __forceinline__ float scale_of(float top) {
  if (top < 0x1p-90f) return top / 127.f;
  constexpr float r = 1.f / 127.f;
  const float q = top * r;
  return fmaf(fmaf(-q, 127.f, top), r, q);
}

// x / s to the nearest whole number, ties to even, for any finite x and s > 0
// with |x| < 2^8 s or so: from the reciprocal's product, off by less than one,
// and the exact remainder.
__device__ __forceinline__ float exact_code(float x, float s) {
  const float up = s < 0x1p-100f ? 0x1p100f : 1.f;  // exact, and the reciprocal does not overflow
  const float step = s * up, y = x * up;
  float c = rintf(y * __builtin_amdgcn_rcpf(step));
  const float rest = fmaf(-c, step, y);
  const float twice = 2.f * fabsf(rest);
  if (twice > step || (twice == step && ((int)c & 1) != 0)) c += rest > 0.f ? 1.f : -1.f;
  return fminf(fmaxf(c, -127.f), 127.f);
}

template <int DIM>
struct CodeWord;  // the dim / 16 bytes of one lane
template <>
struct CodeWord<64> { typedef uint32_t type; };
template <>
struct CodeWord<128> { typedef uint2 type; };
template <>
struct CodeWord<256> { typedef uint4 type; };

// (head, K or V) rows per 16-lane group.  With one, two and four a step of 64
// tokens is written and read back in 6.3, 7.2 and 8.8 us, 18432 tokens of
// prompts in 65, 58 and 60 us, and 147000 tokens are read in 149, 130 and 135.
constexpr int kRowsPerGroup = 2;
constexpr int kRowsPerWave = kRowsPerGroup * 4;

// A wave takes one token's rows r = kRowsPerWave * blockIdx.y ..: row r is
// head r / 2, K for even r and V for odd.
template <RowType T, int DIM>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheRowsArgs p) {
  typedef typename Elem<T>::type E;
  typedef typename CodeWord<DIM>::type Word;
  constexpr int NB = DIM / 32;
  const int lane = threadIdx.x & 63;
  const uint32_t row = __builtin_amdgcn_readfirstlane(p.row0 + blockIdx.x * kWaves + (threadIdx.x >> 6));
  if (row >= (uint32_t)p.s.rows) return;  // unsigned: the last workgroup may pass 2^31
  const int t = (int)row;
  const int group = lane >> 4, j = lane & 15;
  const int nrows = 2 * p.c.heads;
  const int r0 = blockIdx.y * kRowsPerWave + group;

  float x[kRowsPerGroup][NB][2];
#pragma unroll
  for (int q = 0; q < kRowsPerGroup; ++q) {
    const int r = r0 + 4 * q;
    const int rr = r < nrows ? r : 0;
    const E *from = static_cast<const E *>((rr & 1) ? p.v : p.k) + (int64_t)t * ((rr & 1) ? p.v_stride : p.k_stride) +
                   (int64_t)(rr >> 1) * DIM;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const Pair<E> v = *reinterpret_cast<const Pair<E> *>(from + 32 * b + 2 * j);
      x[q][b][0] = Elem<T>::to_float(v.x);
      x[q][b][1] = Elem<T>::to_float(v.y);
    }
  }
  const Place at = find_row(p.s, t, lane);
  if (!at.found || at.seq.bad) return;
  const int64_t base = token_row(p.c, p.s, at.b, at.seq.length - at.seq.n + at.index);
  if (base < 0) return;
#pragma unroll
  for (int q = 0; q < kRowsPerGroup; ++q) {
    const int r = r0 + 4 * q;
    union {
      Word w;
      int8_t c[2 * NB];
    } out;
    float mine = 0.f;  // lane b keeps block b's scale
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float x0 = x[q][b][0], x1 = x[q][b][1];
      const uint32_t top = group_max(max(__float_as_uint(x0) & 0x7fffffffu, __float_as_uint(x1) & 0x7fffffffu));
      const bool fine = top < 0x7f800000u;
      const float s = fine ? scale_of(__uint_as_float(top)) : NAN;
      if (j == b) mine = s;
      // The rounded product with the reciprocal is the code unless the exact
      // remainder comes to half a step: about once in a million values.
      const float r = __builtin_amdgcn_rcpf(s);
      float c0 = rintf(x0 * r), c1 = rintf(x1 * r);
      const float rest = fmaxf(fabsf(fmaf(-c0, s, x0)), fabsf(fmaf(-c1, s, x1)));
      const bool sure = s >= 0x1p-100f && 2.f * rest < s;  // not for NaN, zero or tiny scales
      if (!sure) {
        const bool some = fine && s > 0.f;
        c0 = some ? exact_code(x0, s) : 0.f;
        c1 = some ? exact_code(x1, s) : 0.f;
      }
      out.c[2 * b] = (int8_t)(int)c0;
      out.c[2 * b + 1] = (int8_t)(int)c1;
    }
    if (r < nrows) {
      const int64_t at_head = base + ((int64_t)(r >> 1) << p.c.page_shift);
      int8_t *codes = (r & 1) ? p.c.V : p.c.K;
      float *scales = (r & 1) ? p.c.VS : p.c.KS;
      *reinterpret_cast<Word *>(codes + at_head * DIM + j * (DIM / 16)) = out.w;
      if (j < NB) scales[at_head * NB + j] = mine;
    }
  }
}

// PAST: the rows are written past the caches.  They leave the Infinity Cache
// anyway where they are larger than it (376 MB of f16 rows: 138 us through the
// caches, 130 past them; 512 MB of f32 rows: 188 and 179); smaller ones are
// better kept for whoever reads them.
constexpr int64_t kPastCachesBytes = (int64_t)256 << 20;
template <RowType T, int DIM, bool PAST>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheRowsArgs p) {
  typedef typename Elem<T>::type E;
  typedef typename CodeWord<DIM>::type Word;
  constexpr int NB = DIM / 32;
  const int lane = threadIdx.x & 63;
  const uint32_t row = __builtin_amdgcn_readfirstlane(p.row0 + blockIdx.x * kWaves + (threadIdx.x >> 6));
  if (row >= (uint32_t)p.s.rows) return;  // unsigned: the last workgroup may pass 2^31
  const int t = (int)row;
  const int group = lane >> 4, j = lane & 15;
  const int nrows = 2 * p.c.heads;
  const int r0 = blockIdx.y * kRowsPerWave + group;
  const Place at = find_row(p.s, t, lane);
  if (!at.found) return;  // no sequence's row: left as it was
  int64_t base = -1;
  if (!at.seq.bad) base = token_row(p.c, p.s, at.b, at.seq.length - at.seq.n + at.index);
#pragma unroll
  for (int q = 0; q < kRowsPerGroup; ++q) {
    const int r = r0 + 4 * q;
    if (r >= nrows) continue;
    union {
      Word w;
      int8_t c[2 * NB];
    } in;
    float s[NB];
    if (base >= 0) {
      const int64_t at_head = base + ((int64_t)(r >> 1) << p.c.page_shift);
      in.w = *reinterpret_cast<const Word *>(((r & 1) ? p.c.V : p.c.K) + at_head * DIM + j * (DIM / 16));
      const float *scales = ((r & 1) ? p.c.VS : p.c.KS) + at_head * NB;
#pragma unroll
      for (int b = 0; b < NB; ++b) s[b] = scales[b];
    } else {  // no such token: NaN, never a wrong value
      in.w = Word{};
#pragma unroll
      for (int b = 0; b < NB; ++b) s[b] = NAN;
    }
    E *out = static_cast<E *>((r & 1) ? p.v : p.k) + (int64_t)t * ((r & 1) ? p.v_stride : p.k_stride) +
             (int64_t)(r >> 1) * DIM;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      typedef E Two __attribute__((ext_vector_type(2)));
      typedef Two Unaligned __attribute__((aligned(sizeof(E))));
      const Two v = {Elem<T>::from_float((float)in.c[2 * b] * s[b]), Elem<T>::from_float((float)in.c[2 * b + 1] * s[b])};
      Unaligned *to = reinterpret_cast<Unaligned *>(out + 32 * b + 2 * j);
      if constexpr (PAST)
        __builtin_nontemporal_store(v, to);
      else
        *to = v;
    }
  }
}

// keep: one workgroup per (sequence, head).  The kept indexes ascend strictly,
// so place a is at or before the place of keep[a], and never one that a later
// step reads (keep[a'] > keep[a] >= a for a' > a).  It may be one that an
// earlier step reads, so a chunk's rows are all read before any is written.
template <int DIM>
__global__ __launch_bounds__(kThreads) void cache_keep_kernel(CacheKeepArgs p) {
  typedef typename CodeWord<DIM>::type Word;
  constexpr int NB = DIM / 32;
  constexpr int kChunk = kThreads / 16;  // 16-lane groups: one kept token each
  const int b = p.seq0 + blockIdx.x;
  const int tid = threadIdx.x;
  const int group = tid >> 4, j = tid & 15;
  const Seq seq = seq_at(p.s, b);
  if (seq.n == 0 || seq.bad) return;
  const int first = seq.length - seq.n;
  const int *keep = p.keep + (int64_t)b * p.width;

  for (int a0 = 0; a0 < p.width; a0 += kChunk) {
    // How many of this chunk's entries are kept: up to the first that is not
    // an index of a new token or does not ascend.
    const int a = a0 + group;
    int from = -1, before = -1;
    if (a < p.width) {
      from = keep[a];
      if (a > 0) before = keep[a - 1];
    }
    const bool ok = a < p.width && from > before && from < seq.n && from >= 0;
    __shared__ int good[kChunk];
    if (j == 0) good[group] = ok;
    __syncthreads();
    int count = 0;
    while (count < kChunk && good[count]) ++count;
    const bool mine = group < count;
    int64_t src = -1, dst = -1;
    if (mine) {
      src = token_row(p.c, p.s, b, first + from);
      dst = token_row(p.c, p.s, b, first + a);
    }
    const bool move = mine && src >= 0 && dst >= 0 && src != dst;
    for (int h = blockIdx.y; h < p.c.heads; h += gridDim.y) {
      const int64_t head = (int64_t)h << p.c.page_shift;
      Word kw{}, vw{};
      float ks = 0.f, vs = 0.f;
      if (move) {
        kw = *reinterpret_cast<const Word *>(p.c.K + (src + head) * DIM + j * (DIM / 16));
        vw = *reinterpret_cast<const Word *>(p.c.V + (src + head) * DIM + j * (DIM / 16));
        if (j < NB) {
          ks = p.c.KS[(src + head) * NB + j];
          vs = p.c.VS[(src + head) * NB + j];
        }
      }
      // Every wave's rows of this chunk have arrived before any is written.
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (move) {
        *reinterpret_cast<Word *>(p.c.K + (dst + head) * DIM + j * (DIM / 16)) = kw;
        *reinterpret_cast<Word *>(p.c.V + (dst + head) * DIM + j * (DIM / 16)) = vw;
        if (j < NB) {
          p.c.KS[(dst + head) * NB + j] = ks;
          p.c.VS[(dst + head) * NB + j] = vs;
        }
      }
    }
    if (count < kChunk) return;  // the same in every thread
    __syncthreads();             // `good` is written again
  }
}

template <RowType T>
hipError_t launch_rows(const CacheRowsArgs &a, int rows, bool write, hipStream_t stream) {
  const dim3 grid((unsigned)((rows + kWaves - 1) / kWaves), (unsigned)((2 * a.c.heads + kRowsPerWave - 1) / kRowsPerWave));
  const bool past = 2 * (int64_t)sizeof(typename Elem<T>::type) * a.s.rows * a.c.heads * a.c.dim > kPastCachesBytes;
#define Q8_LAUNCH(DIM)                                                                                   \
  case DIM:                                                                                              \
    if (write)                                                                                           \
      hipLaunchKernelGGL((cache_write_kernel<T, DIM>), grid, dim3(kThreads), 0, stream, a);              \
    else if (past)                                                                                       \
      hipLaunchKernelGGL((cache_read_kernel<T, DIM, true>), grid, dim3(kThreads), 0, stream, a);         \
    else                                                                                                 \
      hipLaunchKernelGGL((cache_read_kernel<T, DIM, false>), grid, dim3(kThreads), 0, stream, a);        \
    return hipGetLastError();
  switch (a.c.dim) {
    Q8_LAUNCH(64)
    Q8_LAUNCH(128)
    Q8_LAUNCH(256)
  }
#undef Q8_LAUNCH
  return hipErrorInvalidValue;
}

hipError_t launch_typed(CacheRowsArgs a, RowType type, bool write, hipStream_t stream) {
  for (int64_t row0 = 0; row0 < a.s.rows; row0 += kMostGroups * kWaves) {
    a.row0 = (int)row0;
    const int rows = (int)std::min<int64_t>(a.s.rows - row0, kMostGroups * kWaves);
    hipError_t e = hipErrorInvalidValue;
    switch (type) {
      case kRowF32: e = launch_rows<kRowF32>(a, rows, write, stream); break;
      case kRowBf16: e = launch_rows<kRowBf16>(a, rows, write, stream); break;
      case kRowF16: e = launch_rows<kRowF16>(a, rows, write, stream); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_cache_write(const CacheRowsArgs &a, RowType type, hipStream_t stream) {
  return launch_typed(a, type, true, stream);
}

hipError_t launch_cache_read(const CacheRowsArgs &a, RowType type, hipStream_t stream) {
  return launch_typed(a, type, false, stream);
}

hipError_t launch_cache_keep(const CacheKeepArgs &args, hipStream_t stream) {
  CacheKeepArgs a = args;
  hipError_t e = hipSuccess;
  for (int64_t seq0 = 0; seq0 < a.s.seqs && e == hipSuccess; seq0 += kMostGroups) {
    a.seq0 = (int)seq0;
    const dim3 grid((unsigned)std::min<int64_t>(a.s.seqs - seq0, kMostGroups), (unsigned)std::min(a.c.heads, 65535));
    switch (a.c.dim) {
      case 64: hipLaunchKernelGGL((cache_keep_kernel<64>), grid, dim3(kThreads), 0, stream, a); break;
      case 128: hipLaunchKernelGGL((cache_keep_kernel<128>), grid, dim3(kThreads), 0, stream, a); break;
      case 256: hipLaunchKernelGGL((cache_keep_kernel<256>), grid, dim3(kThreads), 0, stream, a); break;
      default: return hipErrorInvalidValue;
    }
    e = hipGetLastError();
  }
  return e;
}

}  // namespace q8
