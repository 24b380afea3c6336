// The cache in 4-bit floats: quantising rows as they are written, reading them
// back, and moving accepted drafts to the front of a sequence's new tokens.
//
// Per 32 channels x of a row: s = the smallest power of two with max|x| <= 7 s
// (2^-125 .. 2^125), code = x / s to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with
// its sign, ties to the even code, above 6 6.  At 7 the error of the largest
// value, 1, is half the step between 4 and 6: a smaller bound would waste
// codes, a larger one cut more off than it rounds (mean square error of normal
// values, relative: 0.0136 with 6, 0.0126 with 7, 0.0134 with 8).  Scales are powers
// of two, so every step but the rounding to a code is exact.
//
// All three are bound by memory: they touch each byte once.  A row of dim
// channels belongs to 16 lanes.  In the cache a lane's bytes are channel pair j of
// every block, which keep and read take as they are; write takes dim / 16 channels of one
// block per lane, so that a block's maximum needs few exchanges and its scale is found
// few times, and swaps the codes' bytes between lanes at the end (19600 tokens of prompts
// of 8 heads of 128, bf16, written and read: 46 us, 49 from pairs; f32 rows are as fast
// either way).
#include <algorithm>

#include "cache_rows.h"
#include "mx4_cache.h"

namespace q8 {
namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// The dim / 32 bytes of one lane, which are also a row's scales.
template <int DIM>
struct PairBytes;
template <>
struct PairBytes<64> { typedef uint16_t type; };
template <>
struct PairBytes<128> { typedef uint32_t type; };
template <>
struct PairBytes<256> { typedef uint64_t type; };

// First byte of lane j's pairs of the token `at` of a page's head.
template <int DIM>
__device__ __forceinline__ int pair_place(bool value, int at, int j) {
  constexpr int NB = DIM / 32;
  return value ? (at >> 2) * (2 * DIM) + (4 * j + (at & 3)) * NB : at * (DIM / 2) + j * NB;
}

// Scale byte of a block with the largest magnitude `top` (as bits).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  // 1.75 * 2^e is 7 quarters of 2^e: above it the scale is one step larger.
  const int e = (int)((top + 0x1fffffu) >> 23) - 2;
  return (uint32_t)min(max(e, kMx4Least), kMx4Most);
}

// (head, K or V) rows per 16-lane group.  19600 tokens of prompts of 8 heads are written
// and read back in 49.8, 45.7 and 44.9 us with one, two and four (bf16, dim 128), 43, 34.9
// and 31.9 (dim 64), 94, 96.8 and 87.9 (dim 256); f32 rows in 88, 91 and 82 (dim 128), but
// 136 and 139.5 with two and four at dim 256.  A step of 1536 drafts takes 17.1 and 17.6.
template <RowType T, int DIM>
constexpr int kRowsPerGroup = T == kRowF32 && DIM == 256 ? 2 : 4;

template <typename E, int N>
struct __attribute__((packed, aligned(sizeof(E)))) Run {
  E x[N];
};

// The value of lane l ^ D, for D = 1, 2, 4 and 8.
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t x) {
  if constexpr (D == 4) return across<1>(across<2>(__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xf, 0xf, true)));  // l ^ 7 first
  constexpr int ctrl = D == 1 ? 0xb1 : D == 2 ? 0x4e : 0x128;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, 0xf, 0xf, true);
}

// Which lanes of a row's 16 are block `block` of it, and which part of that.
template <int NB>
struct Piece {
  int block, part;
  __device__ __forceinline__ explicit Piece(int j) {
    if constexpr (NB == 8) {
      block = (j & 3) | (j >> 1 & 4);
      part = j >> 2 & 1;
    } else {
      block = j & (NB - 1);
      part = j / NB;
    }
  }
};

// Largest of a block's 16 / NB lanes.
template <int NB>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  if constexpr (NB == 2) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xf, 0xf, true));  // row_ror:2, 4, 8
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, true));
    m = max(m, across<8>(m));
  } else if constexpr (NB == 4) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, true));
    m = max(m, across<8>(m));
  } else {
    m = max(m, across<4>(m));
  }
  return m;
}

// Byte i of the lane of block b, to byte b of that block's i-th lane: for every part
// of the row, NB lanes that hold NB bytes each.
template <int NB>
__device__ __forceinline__ void turn_bytes(uint32_t (&w)[(NB + 3) / 4], int block) {
  if constexpr (NB == 8) {
    const bool high = block & 4;
    const uint32_t other = across<8>(high ? w[0] : w[1]);
    if (high)
      w[0] = other;
    else
      w[1] = other;
  }
#pragma unroll
  for (int k = 0; k < (NB + 3) / 4; ++k) {
    w[k] = __builtin_amdgcn_perm(across<1>(w[k]), w[k], block & 1 ? 0x03070105u : 0x06020400u);
    if constexpr (NB > 2) w[k] = __builtin_amdgcn_perm(across<2>(w[k]), w[k], block & 2 ? 0x03020706u : 0x05040100u);
  }
}

// A wave takes one token's rows r = 4 * kRowsPerGroup * blockIdx.y ..: row r is
// head r / 2, K for even r and V for odd.
template <RowType T, int DIM>
__global__ __launch_bounds__(kThreads) void mx4_write_kernel(CacheRowsArgs p) {
  typedef typename Elem<T>::type E;
  typedef typename PairBytes<DIM>::type Word;
  constexpr int ROWS = kRowsPerGroup<T, DIM>;
  constexpr int NB = DIM / 32, N = 2 * NB, NW = (NB + 3) / 4;  // channels of a lane; words of its codes
  // A lane's channels come in runs of at most 16 bytes, and those of a block's lanes lie
  // side by side (f32 rows of dim 256, written and read: 135.6 us, 136.7 with a lane's runs
  // side by side).
  constexpr int RUN = N * sizeof(E) <= 16 ? N : 16 / (int)sizeof(E), RUNS = N / RUN;
  const int lane = threadIdx.x & 63;
  const uint32_t row = __builtin_amdgcn_readfirstlane(p.row0 + blockIdx.x * kWaves + (threadIdx.x >> 6));
  if (row >= (uint32_t)p.s.rows) return;  // unsigned: the last workgroup may pass 2^31
  const int t = (int)row;
  const int group = lane >> 4, j = lane & 15;
  const Piece<NB> piece(j);
  const int nrows = 2 * p.c.heads;
  const int r0 = blockIdx.y * 4 * ROWS + group;
  // The pair whose codes the lane holds in the end: the block-th of its part's.
  const int pair = 16 / RUNS * (piece.block / (RUN / 2)) + RUN / 2 * piece.part + piece.block % (RUN / 2);

  Run<E, RUN> x[ROWS][RUNS];
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    const int r = r0 + 4 * q;
    const int rr = r < nrows ? r : 0;
    const E *from = static_cast<const E *>((rr & 1) ? p.v : p.k) + (int64_t)t * ((rr & 1) ? p.v_stride : p.k_stride) +
                   (int64_t)(rr >> 1) * DIM;
#pragma unroll
    for (int k = 0; k < RUNS; ++k)
      x[q][k] = *reinterpret_cast<const Run<E, RUN> *>(from + 32 * piece.block + 32 / RUNS * k + RUN * piece.part);
  }
  const Place at = find_row(p.s, t, lane);
  if (!at.found || at.seq.bad) return;
  const int64_t base = token_row(p.c, p.s, at.b, at.seq.length - at.seq.n + at.index);
  if (base < 0) return;
  const int inside = (int)(base & ((1 << p.c.page_shift) - 1));
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    const int r = r0 + 4 * q;
    float y[N];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      y[i] = Elem<T>::to_float(x[q][i / RUN].x[i % RUN]);
      top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
    }
    const uint32_t e = scale_byte(block_max<NB>(top));
    uint32_t w[NW];
    // Only the scale's exponent counts; values past 6 s become 6 s.
    const float s = __uint_as_float(e << 23);
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float *z = y + 8 * k;
      w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, z[0], z[1], s, 0);
      w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], z[2], z[3], s, 1);
      if constexpr (NB > 2) {
        w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], z[4], z[5], s, 2);
        w[k] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[k], z[6], z[7], s, 3);
      }
      if (e == 255) w[k] = 0;
    }
    turn_bytes<NB>(w, piece.block);
    // The scales of all blocks, in every lane of a part.
    uint32_t es[NW];
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      es[k] = piece.block >> 2 == k ? e << (8 * (piece.block & 3)) : 0u;
      es[k] |= across<1>(es[k]);
      if constexpr (NB > 2) es[k] |= across<2>(es[k]);
      if constexpr (NB > 4) es[k] |= across<8>(es[k]);
    }
    if (r < nrows) {
      const int64_t page = (base - inside) + ((int64_t)(r >> 1) << p.c.page_shift);  // its first token, of this head
      uint8_t *to = reinterpret_cast<uint8_t *>((r & 1) ? p.c.V : p.c.K) + page * (DIM / 2);
      uint8_t *st = reinterpret_cast<uint8_t *>((r & 1) ? p.c.VS : p.c.KS) + (page + inside) * NB;
      Word codes = (Word)w[0], scales = (Word)es[0];
      if constexpr (NW == 2) {
        codes |= (Word)w[1] << 32;
        scales |= (Word)es[1] << 32;
      }
      *reinterpret_cast<Word *>(to + pair_place<DIM>(r & 1, inside, pair)) = codes;
      if (j == 0) *reinterpret_cast<Word *>(st) = scales;
    }
  }
}

// The two values of byte b of a lane's codes, of a block with scale byte e.
template <typename Word>
__device__ __forceinline__ float2 pair_values(Word codes, Word scales, int b) {
  const uint32_t e = (uint32_t)(scales >> (8 * b)) & 0xffu;
  const v2bf v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)(codes >> (8 * b)), __uint_as_float(e << 23), 0);
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  return float2{__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)};
}

// PAST: the rows are written past the caches, where they are larger than those.
constexpr int64_t kPastCachesBytes = (int64_t)256 << 20;
template <RowType T, int DIM, bool PAST>
__global__ __launch_bounds__(kThreads) void mx4_read_kernel(CacheRowsArgs p) {
  typedef typename Elem<T>::type E;
  typedef typename PairBytes<DIM>::type Word;
  constexpr int NB = DIM / 32, ROWS = kRowsPerGroup<T, DIM>;
  const int lane = threadIdx.x & 63;
  const uint32_t row = __builtin_amdgcn_readfirstlane(p.row0 + blockIdx.x * kWaves + (threadIdx.x >> 6));
  if (row >= (uint32_t)p.s.rows) return;  // unsigned: the last workgroup may pass 2^31
  const int t = (int)row;
  const int group = lane >> 4, j = lane & 15;
  const int nrows = 2 * p.c.heads;
  const int r0 = blockIdx.y * 4 * ROWS + group;
  const Place at = find_row(p.s, t, lane);
  if (!at.found) return;  // no sequence's row: left as it was
  int64_t base = -1;
  if (!at.seq.bad) base = token_row(p.c, p.s, at.b, at.seq.length - at.seq.n + at.index);
  const int inside = (int)(base & ((1 << p.c.page_shift) - 1));
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    const int r = r0 + 4 * q;
    if (r >= nrows) continue;
    Word codes = 0, scales = (Word)~0ull;  // no such token: NaN, never a wrong value
    if (base >= 0) {
      const int64_t page = (base - inside) + ((int64_t)(r >> 1) << p.c.page_shift);
      codes = *reinterpret_cast<const Word *>(reinterpret_cast<const uint8_t *>((r & 1) ? p.c.V : p.c.K) +
                                              page * (DIM / 2) + pair_place<DIM>(r & 1, inside, j));
      scales = *reinterpret_cast<const Word *>(reinterpret_cast<const uint8_t *>((r & 1) ? p.c.VS : p.c.KS) +
                                               (page + inside) * NB);
    }
    E *out = static_cast<E *>((r & 1) ? p.v : p.k) + (int64_t)t * ((r & 1) ? p.v_stride : p.k_stride) +
             (int64_t)(r >> 1) * DIM;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      typedef E Two __attribute__((ext_vector_type(2)));
      typedef Two Unaligned __attribute__((aligned(sizeof(E))));
      const float2 x = pair_values<Word>(codes, scales, b);
      const Two v = {Elem<T>::from_float(x.x), Elem<T>::from_float(x.y)};
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
__global__ __launch_bounds__(kThreads) void mx4_keep_kernel(CacheKeepArgs p) {
  typedef typename PairBytes<DIM>::type Word;
  constexpr int NB = DIM / 32;
  constexpr int kChunk = kThreads / 16;  // 16-lane groups: one kept token each
  const int b = p.seq0 + blockIdx.x;
  const int tid = threadIdx.x;
  const int group = tid >> 4, j = tid & 15;
  const Seq seq = seq_at(p.s, b);
  if (seq.n == 0 || seq.bad) return;
  const int first = seq.length - seq.n;
  const int *keep = p.keep + (int64_t)b * p.width;
  const int mask = (1 << p.c.page_shift) - 1;
  uint8_t *K = reinterpret_cast<uint8_t *>(p.c.K), *V = reinterpret_cast<uint8_t *>(p.c.V);
  uint8_t *KS = reinterpret_cast<uint8_t *>(p.c.KS), *VS = reinterpret_cast<uint8_t *>(p.c.VS);

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
    const int si = (int)(src & mask), di = (int)(dst & mask);
    for (int h = blockIdx.y; h < p.c.heads; h += gridDim.y) {
      const int64_t head = (int64_t)h << p.c.page_shift;
      const int64_t sp = (src - si + head) * (DIM / 2), dp = (dst - di + head) * (DIM / 2);
      Word kw = 0, vw = 0, ks = 0, vs = 0;
      if (move) {
        kw = *reinterpret_cast<const Word *>(K + sp + pair_place<DIM>(false, si, j));
        vw = *reinterpret_cast<const Word *>(V + sp + pair_place<DIM>(true, si, j));
        if (j == 0) {
          ks = *reinterpret_cast<const Word *>(KS + (src + head) * NB);
          vs = *reinterpret_cast<const Word *>(VS + (src + head) * NB);
        }
      }
      // Every wave's rows of this chunk have arrived before any is written.
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (move) {
        *reinterpret_cast<Word *>(K + dp + pair_place<DIM>(false, di, j)) = kw;
        *reinterpret_cast<Word *>(V + dp + pair_place<DIM>(true, di, j)) = vw;
        if (j == 0) {
          *reinterpret_cast<Word *>(KS + (dst + head) * NB) = ks;
          *reinterpret_cast<Word *>(VS + (dst + head) * NB) = vs;
        }
      }
    }
    if (count < kChunk) return;  // the same in every thread
    __syncthreads();             // `good` is written again
  }
}

template <RowType T>
hipError_t launch_rows(const CacheRowsArgs &a, int rows, bool write, hipStream_t stream) {
  const bool past = 2 * (int64_t)sizeof(typename Elem<T>::type) * a.s.rows * a.c.heads * a.c.dim > kPastCachesBytes;
#define Q8_LAUNCH(DIM)                                                                                 \
  case DIM: {                                                                                          \
    constexpr int kPerWave = 4 * kRowsPerGroup<T, DIM>;                                                \
    const dim3 grid((unsigned)((rows + kWaves - 1) / kWaves), (unsigned)((2 * a.c.heads + kPerWave - 1) / kPerWave)); \
    if (write)                                                                                         \
      hipLaunchKernelGGL((mx4_write_kernel<T, DIM>), grid, dim3(kThreads), 0, stream, a);              \
    else if (past)                                                                                     \
      hipLaunchKernelGGL((mx4_read_kernel<T, DIM, true>), grid, dim3(kThreads), 0, stream, a);         \
    else                                                                                               \
      hipLaunchKernelGGL((mx4_read_kernel<T, DIM, false>), grid, dim3(kThreads), 0, stream, a);        \
    return hipGetLastError();                                                                          \
  }
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

hipError_t launch_mx4_write(const CacheRowsArgs &a, RowType type, hipStream_t stream) {
  return launch_typed(a, type, true, stream);
}

hipError_t launch_mx4_read(const CacheRowsArgs &a, RowType type, hipStream_t stream) {
  return launch_typed(a, type, false, stream);
}

hipError_t launch_mx4_keep(const CacheKeepArgs &args, hipStream_t stream) {
  CacheKeepArgs a = args;
  hipError_t e = hipSuccess;
  for (int64_t seq0 = 0; seq0 < a.s.seqs && e == hipSuccess; seq0 += kMostGroups) {
    a.seq0 = (int)seq0;
    const dim3 grid((unsigned)std::min<int64_t>(a.s.seqs - seq0, kMostGroups), (unsigned)std::min(a.c.heads, 65535));
    switch (a.c.dim) {
      case 64: hipLaunchKernelGGL((mx4_keep_kernel<64>), grid, dim3(kThreads), 0, stream, a); break;
      case 128: hipLaunchKernelGGL((mx4_keep_kernel<128>), grid, dim3(kThreads), 0, stream, a); break;
      case 256: hipLaunchKernelGGL((mx4_keep_kernel<256>), grid, dim3(kThreads), 0, stream, a); break;
      default: return hipErrorInvalidValue;
    }
    e = hipGetLastError();
  }
  return e;
}

}  // namespace q8
