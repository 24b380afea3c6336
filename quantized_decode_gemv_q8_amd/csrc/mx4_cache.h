// Internal declarations of the cache in 4-bit floats, and its attention.
#pragma once

#include "q8_attention.h"

namespace q8 {

// A cache of 4-bit floats: pages as those of the Q8_0 cache, u8 arrays
//   K, V    [pages, heads, page_size, dim / 2]   codes, two to a byte
//   KS, VS  [pages, heads, page_size, dim / 32]  scales, 2^(byte - 127)
// Channel d = 32 b + 2 j + i of a row is nibble i (low first) of byte
// j * (dim / 32) + b of the row in K.  In V four neighbouring tokens of a page
// share 2 * dim bytes, and the byte is (4 j + token % 4) * (dim / 32) + b of them.
// A lane of the attention then finds what it needs of a tile in one run of dim / 8
// bytes: of K the pairs 4 c .. 4 c + 3 of all blocks of one key, of V the pair j of
// all blocks of four keys.  A byte is what one conversion takes.
// The kernels' arguments are those of the Q8_0 cache with these arrays in them.
inline Cache mx4_cache(uint8_t *K, uint8_t *KS, uint8_t *V, uint8_t *VS) {
  Cache c;
  c.K = reinterpret_cast<int8_t *>(K);
  c.KS = reinterpret_cast<float *>(KS);
  c.V = reinterpret_cast<int8_t *>(V);
  c.VS = reinterpret_cast<float *>(VS);
  return c;
}

// Scale bytes: kMx4Least .. kMx4Most, and 255 for a block that holds an infinity
// or a NaN.  Half of the least scale, the smallest value, is a normal bf16;
// six times the largest is a finite one.
constexpr int kMx4Least = 2, kMx4Most = 252;

hipError_t launch_mx4_write(const CacheRowsArgs &a, RowType type, hipStream_t stream);
hipError_t launch_mx4_read(const CacheRowsArgs &a, RowType type, hipStream_t stream);
hipError_t launch_mx4_keep(const CacheKeepArgs &a, hipStream_t stream);

// Workgroups per CU of the kernel for 16 rows: as many as fit its registers, where more of
// them have more bytes in flight.  32 sequences of up to 32768 keys: dim 64 bf16 69 us with 4,
// 81 with 2; f16 71 and 84; f32 79 with 3, 89 with 2.  At dim 128 3 are no faster for bf16 and
// spill for f32.  At dim 256 2 spill: f32 420 us, 304 with 1; f16 265 and 268; bf16 (6 registers)
// 230, 256 with 1.
constexpr int mx4_direct_wgs(RowType type, int dim) {
  if (dim == 64) return type == kRowF32 ? 3 : 4;
  return dim == 128 || type == kRowBf16 ? kAttnWgsPerCu : 1;
}

// Rows of an item of the kernels whose waves share keys: 64 or 128, as far as half of a
// SIMD's registers hold, or 256 where all of them do.
constexpr int kMx4DeepRows = 256;
constexpr bool mx4_deep(RowType type, int dim) { return dim <= 64 || (dim == 128 && type != kRowF32); }

// Rows of an item, for `mean` rows of an average sequence's head.  us by the rows of an
// item, trees of drafts over 8 x 8192 keys (32 heads, 8 of keys), then 32 sequences of up to
// 32768 keys (4 heads of keys):
//   20 rows, dim 128, bf16   16: 36.9  32: 35.7  64: 46.2         16: 113  32:  88  64: 146
//   20 rows, dim 128, f32    16: 41.0  32: 45.3  64: 54.4         16: 127  32: 117  64: 180
//   20 rows, dim 256, bf16   16: 53.6            64: 68.7         16: 236           64: 235
//   20 rows, dim 256, f32    16: 76.9            64: 91.5         16: 319           64: 332
//   48 rows, dim 128, bf16   32: 47.8  64: 49.0  128: 51.7        32: 151  64: 154  128: 151
//   48 rows, dim 128, f32    16: 54.7  32: 63.8  64: 58.6         16: 197  32: 210  64: 189
//   48 rows, dim 256, bf16   16: 81.6            64: 73.7         16: 348           64: 253
//   96 rows, dim  64, f32    32: 57.4  64: 66.3  128: 63.7        32: 188  64: 234  128: 197
//   96 rows, dim 128, f16    32: 67.8  64: 78.9  128: 71.8
//   96 rows, dim 128, bf16   32: 63.9  64: 76.3  128: 67.3        32: 223  64: 272  128: 223
//  128 rows, dim 128, bf16   32: 72.9  64: 78.6  128: 71.5
// From 129 on 256: at 128 rows of dim 128 the two are alike (f16 78 us in items of 128, 77
// in those of 256, bf16 70 and 74).
constexpr int mx4_tile(RowType type, int dim, int64_t mean) {
  if (mean <= 16 || (mean <= 32 && dim == 256)) return 16;
  if (!mx4_deep(type, dim)) return mean <= 32 ? 32 : 64;
  return mean <= 96 ? 32 : mean <= 128 ? 128 : kMx4DeepRows;
}

constexpr int mx4_wgs(RowType type, int dim, int tile) {
  return tile == kMx4DeepRows ? 1 : tile <= 16 ? mx4_direct_wgs(type, dim) : kAttnWgsPerCu;
}

hipError_t launch_mx4_attention_f32(const AttnArgs &a, int rows, int wgs, hipStream_t stream);
hipError_t launch_mx4_attention_bf16(const AttnArgs &a, int rows, int wgs, hipStream_t stream);
hipError_t launch_mx4_attention_f16(const AttnArgs &a, int rows, int wgs, hipStream_t stream);

}  // namespace q8
