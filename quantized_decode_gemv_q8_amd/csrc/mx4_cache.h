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
// them have more bytes in flight (32 sequences of up to 32768 keys of dim 64: bf16 74 us
// with 4, 84 with 2; f32 81 with 3, 91 with 2; at dim 128 3 are no faster for bf16 and spill
// for f32).
constexpr int mx4_direct_wgs(RowType type, int dim) { return dim > 64 ? kAttnWgsPerCu : type == kRowF32 ? 3 : 4; }

// Rows of an item of the kernels whose waves share keys: 64 or 128, as far as half of a
// SIMD's registers hold, or 256 where all of them do.
constexpr int kMx4DeepRows = 256;
constexpr bool mx4_has_deep(RowType type, int dim) { return dim <= 64 || (dim == 128 && type != kRowF32); }
constexpr int mx4_max_rows(RowType type, int dim) { return dim <= 64 || (dim == 128 && type != kRowF32) ? 128 : 64; }
// For a mean of more than 64 rows.  At 128 rows of dim 128 the two are alike (f16 78 and 77
// us over 8 x 8192 keys, bf16 70 and 74), below it items of 128 are faster (68 rows 70 and 75).
constexpr int mx4_many_rows(RowType type, int dim, int64_t mean) {
  return mean > 128 && mx4_has_deep(type, dim) ? kMx4DeepRows : mx4_max_rows(type, dim);
}

constexpr int mx4_wgs(RowType type, int dim, int tile) {
  return tile == kMx4DeepRows ? 1 : tile <= 16 ? mx4_direct_wgs(type, dim) : kAttnWgsPerCu;
}

hipError_t launch_mx4_attention_f32(const AttnArgs &a, int rows, int wgs, hipStream_t stream);
hipError_t launch_mx4_attention_bf16(const AttnArgs &a, int rows, int wgs, hipStream_t stream);
hipError_t launch_mx4_attention_f16(const AttnArgs &a, int rows, int wgs, hipStream_t stream);

}  // namespace q8
