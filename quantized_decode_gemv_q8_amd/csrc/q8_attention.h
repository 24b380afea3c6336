// Internal declarations of the attention over the Q8_0 cache.
#pragma once

#include "q8_cache.h"

namespace q8 {

// Keys a workgroup takes at a time: one 32-key tile for each of its four waves.
constexpr int kAttnTile = 32;
constexpr int kAttnStep = kAttnTile * kWaves;

// One split item: rows whose keys several workgroups share.  Workgroup w is
// the first contributor of at most one, so the descriptors are indexed by it.
struct AttnItem {
  int valid;
  int last;    // last contributing workgroup
  int row0;    // first row of the row tensors
  int tokens;  // rows of the item
  int head0;   // first query head
  int heads;   // query heads per row
  int seq_new;            // new tokens of the sequence, for rows that see nothing
  int context;            // tokens before the new ones
};

struct AttnArgs {
  Cache c;
  Seqs s;
  const void *q;
  void *out;
  int64_t q_stride, out_stride;  // elements between rows
  const uint64_t *tree;          // [rows, tree_words] or null: causal
  int tree_words;
  int group;       // query heads per head of the cache
  int subs;        // a group's heads are taken in `subs` items of sub_heads
  int sub_heads;
  int tile_tokens;  // tokens (rows of q) per item
  float alpha;
  int unit_shift;    // log2 of the keys of a unit of work, a multiple of kAttnStep
  int half_rows;     // items of at most this many rows have units of twice the keys (0: none)
  int item_cost;     // units that an item is charged besides its keys
  int few_units;     // the units of all items are sure to stay below 2^31
  float *partial;    // 2 * gridDim.x slots of attn_slot_floats(rows, dim); null as items
  AttnItem *items;   // gridDim.x; null where every item is one unit
};

// Floats of one partial: rows x dim sums, then the rows' maxima and weights.
__host__ __device__ constexpr int64_t attn_slot_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }

// Rows of an item of the kernel whose waves take different keys (16, and 32
// where the sums and the query parts still leave room for a tile in flight).
constexpr int attn_direct_rows(int dim) { return dim <= 128 ? 32 : 16; }
// Rows of an item of the other kernel: 64 or 128, as far as a wave's registers hold.
constexpr int attn_max_rows(RowType type, int dim) { return dim <= 64 || (dim == 128 && type != kRowF32) ? 128 : 64; }

// Workgroups per CU: a wave then has half of a SIMD's registers.  With 3 or 4
// the kernel for 4 rows of f32 spills (26 and 93 registers at dim 128), and a
// batch of 32 sequences of 1 .. 8192 keys takes 81 and 134 us instead of 64
// (bf16 rows: 60, 60 and 93).
constexpr int kAttnWgsPerCu = 2;

hipError_t launch_attention_f32(const AttnArgs &a, int rows, int wgs, hipStream_t stream);
hipError_t launch_attention_bf16(const AttnArgs &a, int rows, int wgs, hipStream_t stream);
hipError_t launch_attention_f16(const AttnArgs &a, int rows, int wgs, hipStream_t stream);

}  // namespace q8
