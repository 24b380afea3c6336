// Internal declarations of the Q8_0 cache: its layout, the description of the
// sequences that live in it, and the arguments of its kernels.
#pragma once

#include "q8_common.h"

namespace q8 {

// Element types of the rows outside the cache.
enum RowType { kRowF32 = 0, kRowBf16 = 1, kRowF16 = 2 };

// A cache of `pages` pages; a page holds page_size tokens of every head:
//   K, V    i8  [pages, heads, page_size, dim]       codes, in pair order
//   KS, VS  f32 [pages, heads, page_size, dim / 32]  scales, in block order
// Pair order: channel d = 32 b + 2 j + i (b < dim / 32, j < 16, i < 2) lies at
// byte j * (dim / 16) + 2 b + i of its row.  Lane j of a 16-lane group then
// finds one channel pair of every block in one load of dim / 16 bytes, which
// is what the matrix operands of the attention need of V (all 16 rows of an
// operand tile in one block, so that the block's scale is one factor), and a
// run of four pairs j holds eight neighbouring channels of every block, which
// is what they need of K.
struct Cache {
  int8_t *K;
  float *KS;
  int8_t *V;
  float *VS;
  uint32_t pages;
  int heads, dim;
  int page_shift;  // log2 of page_size
};

// Sequence b owns the pages table[b * table_stride + 0, 1, ...] and holds
// lengths[b] tokens.  Its newest offsets[b+1] - offsets[b] tokens are rows
// offsets[b] .. offsets[b+1] - 1 of the row tensors (`rows` rows).
struct Seqs {
  const int *table;
  const int *lengths;
  const int *offsets;
  int64_t table_stride;
  int64_t max_tokens;  // columns of the table, in tokens
  int seqs;
  int rows;
};

struct CacheRowsArgs {
  Cache c;
  Seqs s;
  void *k, *v;                 // rows of [heads, dim] elements (read: written)
  int64_t k_stride, v_stride;  // elements between rows
  int row0;                    // first row of the launch (set by the launcher)
};
hipError_t launch_cache_write(const CacheRowsArgs &a, RowType type, hipStream_t stream);
hipError_t launch_cache_read(const CacheRowsArgs &a, RowType type, hipStream_t stream);

struct CacheKeepArgs {
  Cache c;
  Seqs s;
  const int *keep;  // [seqs, width]
  int width;
  int seq0;  // first sequence of the launch (set by the launcher)
};
hipError_t launch_cache_keep(const CacheKeepArgs &a, hipStream_t stream);

#ifdef __HIPCC__
// One sequence, as its description says; n == 0 where its rows are none or
// do not lie within the row tensors.
struct Seq {
  int start, n, length;
  bool bad;  // the length does not hold the new rows, or is more than the table holds
};

__device__ __forceinline__ Seq seq_of(const Seqs &s, int start, int end, int length) {
  Seq q;
  const bool rows_ok = start >= 0 && end >= start && end <= s.rows;
  q.start = start;
  q.n = rows_ok ? end - start : 0;
  q.length = length;
  q.bad = length < q.n || (int64_t)length > s.max_tokens;
  return q;
}

// A word whose address is the same in all lanes, through the scalar cache.
__device__ __forceinline__ int uniform_load(const int *p) {
  return *(const __attribute__((address_space(4))) int *)p;
}
__device__ __forceinline__ Seq uniform_seq_at(const Seqs &s, int b) {
  return seq_of(s, uniform_load(s.offsets + b), uniform_load(s.offsets + b + 1), uniform_load(s.lengths + b));
}

__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ Seq seq_at(const Seqs &s, int b) {
  return seq_of(s, s.offsets[b], s.offsets[b + 1], s.lengths[b]);
}
#endif

}  // namespace q8
