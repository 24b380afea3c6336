// Attention over the Q8_0 cache for gfx950: for each row t and query head h
//   out[t, h] = sum_j p_j V_j / sum_j p_j,   p_j = exp(alpha q[t, h] . K_j - m)
// over the tokens j that the row sees, in one pass with a running maximum m
// and running sums.
//
// Arithmetic.  The k-slice of v_mfma_f32_16x16x32 is exactly one 32-channel
// block, and codes (|code| <= 128) are exact in f16 and bf16, so
//   * scores: q is cut into f16 parts (1 for bf16 and f16 rows, 2 for f32), each
//     row scaled by a power of two so that f16 holds it; a block's unscaled
//     partial comes out of the matrix core and is multiplied by the key's scale
//     once, in f32;
//   * output: the value scale depends on the key and the block, so it is
//     multiplied into the weight, p_j s_jb, which is cut into bf16 parts against
//     the exact codes (2 for bf16 and f16 rows: 2^-16; 3 for f32: exact).  bf16,
//     not f16: the product spans f32's range, and its size says nothing about
//     what it counts.  Where the keys with large weights hold values of zero, the
//     smallest weights make the output, and f16 has no bits left for them.
// Maxima, sums, weights and outputs are f32 throughout.
//
// Layout.  The scores are computed transposed, S^T = K Q^T, and so is the
// output, O^T = V^T P^T: lane l then holds, for its row (l % 16), the weights
// of keys 4 (l / 16) + 0..3 of each 16-key tile, which is what the second
// product needs from it when its k index is read as those keys.  Weights never
// leave their lane, a row's maximum is two cross-lane steps, and the cache's
// pair order lets K, V and their scales go from memory to registers with no
// shared memory between.
//
// Three kernels share this.  Attn (16 or 32 rows): every wave takes its own
// keys.  AttnFew (4 or 8 rows): the same, with the lanes that the missing rows
// leave idle put to the weights' work.  attention_wide_kernel (64 or 128 rows):
// the waves take the same keys and different rows, operands go through LDS.
//
// Work.  An item is a sequence's tile of rows for one head of the cache; its
// keys are cut into units (of 128, or one unit with all of a short sequence).
// The units of all items form one list that is dealt to the workgroups in equal
// contiguous runs, so sequences of all lengths load the device evenly.  A
// workgroup that has all of an item's units writes the rows; otherwise it
// leaves sums, maxima and weights, which a second kernel joins in key order (so
// results do not depend on timing).  Lengths and offsets are read on the
// device: a captured graph follows them.
//
// What bounds it.  Few rows: memory.  With 4 rows of f32 per head, dim 128, time
// grows by 1 us per 5.85 MB of cache.  A large copy moves 4.9 TB/s; a large read
// of contiguous runs 6.1, 7.1 with loads that leave no trace in the caches, which
// are not used here.  A batch of 32 ragged sequences (316 MB) takes 64 us and its
// join 5, two sequences of 131072 keys (604 MB) 112 and 7.  From 16 rows on:
// vector instructions, for the codes' conversion, the exponentials and the
// weights' parts.  68 GFLOP of bf16 trees take 169 us (0.40 PFLOP/s); of the 160
// of the main kernel vector instructions issue for 107 on every SIMD and the
// matrix cores are busy for 43, 9 of them at the same time.  16 GFLOP of f32
// pieces of prompts take 81 us (0.2 PFLOP/s, two parts of q and three of the
// weights): 42, 17 and 4 of 68.
#pragma once

#include <type_traits>

#include "q8_attention.h"

namespace q8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

template <RowType T>
struct AttnElem;
// kQParts f16 parts of a query, kPParts bf16 parts of a weight, each of what
// the ones before leave: two are to 2^-16, 2^-8 of a 16-bit output's half step or
// 2^-5, three are all of an f32.
template <>
struct AttnElem<kRowF32> {
  typedef float type;
  static constexpr int kQParts = 2, kPParts = 3;
};
template <>
struct AttnElem<kRowBf16> {
  typedef __bf16 type;
  static constexpr int kQParts = 1, kPParts = 2;
};
template <>
struct AttnElem<kRowF16> {
  typedef _Float16 type;
  static constexpr int kQParts = 1, kPParts = 2;
};

template <typename E, int N>
struct __attribute__((packed, aligned(sizeof(E)))) Run {
  E x[N];
};

__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }

// The upper halves of two floats, packed: exact where they fit bf16, cut otherwise.
__device__ __forceinline__ uint32_t pack_hi(float lo, float hi) {
  return __builtin_amdgcn_perm(bits(hi), bits(lo), 0x07060302u);
}

// The same rounded to bf16, to the nearest.
__device__ __forceinline__ uint32_t pack_near(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});
}

// Codes at byte pair `half` of a word as two f16: 1024 + (code + 128) by its
// bits, less 1152.
__device__ __forceinline__ uint32_t pair_f16(uint32_t w, int half) {
  const uint32_t u = __builtin_amdgcn_perm(0x64646464u, w ^ 0x80808080u, half ? 0x04030402u : 0x04010400u);
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, u) - v2h{(_Float16)1152.f, (_Float16)1152.f});
}
// The same as code + 128 in units of 2^-24, the f16 numbers whose bits are the
// biased code: one instruction, and the matrix cores take them as they are.
constexpr float kBiasedUnit = 1.f / 16777216.f;
__device__ __forceinline__ uint32_t pair_biased(uint32_t biased, int half) {
  return __builtin_amdgcn_perm(0u, biased, half ? 0x0c030c02u : 0x0c010c00u);
}

// x less half `half` of a packed pair of bf16, in one instruction: exact where
// that half is x cut to bf16.
template <int HALF>
__device__ __forceinline__ float less(uint32_t pair, float x) {
  // The pair (-1, 0) must not become the inline constant -1.0: the compiler
  // takes that for the lower half, the hardware for the upper one.
  uint32_t minus_one = 0xbf800000u;
  if constexpr (HALF == 0) asm("s_mov_b32 %0, 0xbf80" : "=s"(minus_one));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, pair), __builtin_bit_cast(v2bf, minus_one), x, false);
}

// Parts of eight floats as matrix operands, each the first 8 bits of what the
// ones before left; of two, the last is rounded (cut it would be off by twice
// as much, always downwards), of three it is all that is left.
template <int PARTS>
__device__ __forceinline__ void split8(const float (&x)[8], v4u (&out)[PARTS]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool rest = PARTS < 3 && p + 1 == PARTS;
      out[p][i] = rest ? pack_near(r[2 * i], r[2 * i + 1]) : pack_hi(r[2 * i], r[2 * i + 1]);
      if (p + 1 < PARTS) {
        r[2 * i] = less<0>(out[p][i], r[2 * i]);
        r[2 * i + 1] = less<1>(out[p][i], r[2 * i + 1]);
      }
    }
  }
}

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

__device__ __forceinline__ v4f mfma_f16(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Lane N of each 16-lane group, to all of them (row_newbcast).
template <int N>
__device__ __forceinline__ float bcast(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + N, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

__device__ __forceinline__ float across_groups_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float across_groups_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Channels 32 b + 8 c + 0..7 of every block of one row of q, as they come.
template <RowType T, int DIM>
struct QueryRow {
  Run<typename AttnElem<T>::type, 8> x[DIM / 32];
};
template <RowType T, int DIM>
__device__ __forceinline__ void fetch_query(const AttnArgs &p, int t, int head, int c, QueryRow<T, DIM> &to) {
  typedef typename AttnElem<T>::type E;
  const E *q = static_cast<const E *>(p.q) + (int64_t)t * p.q_stride + (int64_t)head * DIM + 8 * c;
#pragma unroll
  for (int b = 0; b < DIM / 32; ++b) to.x[b] = *reinterpret_cast<const Run<E, 8> *>(q + 32 * b);
}

// Its parts, scaled by a power of two that brings the row's largest channel to
// 2^14 .. 2^15 so that f16 holds them: one part is exact for bf16 and f16 rows
// (channels below 2^-32 of the largest lose bits that no f32 sum would keep), two
// are to 2^-23 for f32.  Returns what undoes the scaling.  A row that is not
// `in` is zeros.
template <RowType T, int DIM>
__device__ __forceinline__ float cut_query(const QueryRow<T, DIM> &from, bool in,
                                           v4u (&qf)[DIM / 32][AttnElem<T>::kQParts]) {
  constexpr int NB = DIM / 32;
  float x[NB][8], top = 0.f;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[b][i] = in ? (float)from.x[b].x[i] : 0.f;
      top = fmaxf(top, fabsf(x[b][i]));
    }
  top = across_groups_max(top);
  // No further than 2^126, so that what undoes it is no zero (which would make a
  // NaN of a masked score); even the smallest f32 is 2^-23 then, and kept.
  const int up = top > 0.f && top < INFINITY ? min(15 - __builtin_amdgcn_frexp_expf(top), 126) : 0;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0 = ldexpf(x[b][2 * i], up), y1 = ldexpf(x[b][2 * i + 1], up);
#pragma unroll
      for (int n = 0; n < AttnElem<T>::kQParts; ++n) {
        const v2h h = {(_Float16)y0, (_Float16)y1};
        qf[b][n][i] = __builtin_bit_cast(uint32_t, h);
        y0 -= (float)h.x;
        y1 -= (float)h.y;
      }
    }
  return ldexpf(1.f, -up);
}

// ---------------------------------------------------------------- the work list

// Keys an item's rows may see: all of the sequence's under a tree, those up to
// the item's last token otherwise.
__device__ __forceinline__ int item_keys(const AttnArgs &p, const Seq &q, int r) {
  if (p.tree != nullptr) return q.length;
  return q.length - q.n + min(q.n, (r + 1) * p.tile_tokens);
}
__device__ __forceinline__ int row_items(const AttnArgs &p, const Seq &q) {
  return (q.n + p.tile_tokens - 1) / p.tile_tokens;
}
// log2 of the keys of a unit: those of an item that leaves half of a wide
// kernel's row tiles empty are twice as long, so that units cost about the same.
__device__ __forceinline__ int item_shift(const AttnArgs &p, const Seq &q, int r) {
  return p.unit_shift + (p.half_rows > 0 && min(p.tile_tokens, q.n - r * p.tile_tokens) * p.sub_heads <= p.half_rows);
}
// Units of an item: those of its keys, after p.item_cost that stand for what an
// item costs whatever its length.
__device__ __forceinline__ int item_units(const AttnArgs &p, const Seq &q, int r) {
  if (q.bad) return 1 + p.item_cost;
  const int shift = item_shift(p, q, r);
  const int u = (item_keys(p, q, r) + (1 << shift) - 1) >> shift;
  return (u < 1 ? 1 : u) + p.item_cost;
}
// Units of a sequence's items for one head (and sub-group of heads).
__device__ __forceinline__ int64_t head_units(const AttnArgs &p, const Seq &q) {
  const int items = row_items(p, q);
  if (items == 0) return 0;
  if (items == 1 || p.tree != nullptr || q.bad)  // all items but the last are alike
    return (int64_t)(items - 1) * item_units(p, q, 0) + item_units(p, q, items - 1);
  int64_t u = 0;
  for (int r = 0; r < items; ++r) u += item_units(p, q, r);
  return u;
}

// a / b for a >= 0, b > 0 and quotients below 2^50: the double's quotient is off
// by at most one (a 64-bit integer division is over a hundred instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  const double d = (double)b;
  double x = __builtin_amdgcn_rcp(d);  // some 24 bits, doubled by each step
  x = fma(fma(-d, x, 1.0), x, x);
  x = fma(fma(-d, x, 1.0), x, x);
  int64_t q = (int64_t)((double)a * x);
  int64_t rest = a - q * b;
  if (rest < 0) {
    --q;
    rest += b;
  }
  return rest >= b ? q + 1 : q;
}

struct RunStart {  // where a workgroup's run begins
  int b;
  Seq seq;        // sequence b
  int64_t rest;   // units into sequence b
  int64_t begin, end, total;
  int wgs;        // workgroups with a run
};

// Every wave sums the sequences' units, a stretch of them per lane, and finds
// its workgroup's share.
__device__ __forceinline__ RunStart find_run(const AttnArgs &p, int wg, int wgs, int lane) {
  const int64_t heads = (int64_t)p.c.heads * p.subs;
  const int per = (p.s.seqs + 63) / 64;
  const int b0 = min(lane * per, p.s.seqs), b1 = min(b0 + per, p.s.seqs);
  int64_t mine = 0;
  Seq seq{0, 0, 0, false};
  for (int b = b0; b < b1; ++b) {
    seq = seq_at(p.s, b);
    mine += heads * head_units(p, seq);
  }
  int64_t upto;
  if (p.few_units) {  // the total fits 31 bits: a scan by DPP
    int x = (int)mine;
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);   // row_shr:1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
    upto = x;
  } else {
    upto = mine;
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t other = __shfl_up(upto, d);
      if (lane >= d) upto += other;
    }
  }
  RunStart r;
  r.total = (int64_t)((uint64_t)__builtin_amdgcn_readlane((uint32_t)((uint64_t)upto >> 32), 63) << 32 |
                      (uint32_t)__builtin_amdgcn_readlane((uint32_t)upto, 63));
  r.wgs = (int)(r.total < wgs ? r.total : wgs);
  if (wg >= r.wgs) return r;
  r.begin = quotient(r.total * wg, r.wgs);
  r.end = quotient(r.total * (wg + 1), r.wgs);
  int64_t at = upto - mine;
  const bool owner = r.begin >= at && r.begin < upto;
  int b = b0;
  if (owner && per > 1) {
    for (;; ++b) {
      seq = seq_at(p.s, b);
      const int64_t u = heads * head_units(p, seq);
      if (r.begin < at + u) break;  // before b1: the stretch holds the unit
      at += u;
    }
  }
  const int from = __builtin_ctzll(__ballot(owner));
  const int64_t rest = r.begin - at;
  r.b = __builtin_amdgcn_readlane(b, from);
  r.rest = (int64_t)((uint64_t)__builtin_amdgcn_readlane((uint32_t)((uint64_t)rest >> 32), from) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((uint32_t)rest, from));
  r.seq.start = __builtin_amdgcn_readlane(seq.start, from);
  r.seq.n = __builtin_amdgcn_readlane(seq.n, from);
  r.seq.length = __builtin_amdgcn_readlane(seq.length, from);
  r.seq.bad = __builtin_amdgcn_readlane((int)seq.bad, from) != 0;
  return r;
}

// The workgroup whose run holds unit u.
__device__ __forceinline__ int wg_of(int64_t u, const RunStart &r) {
  return (int)quotient((u + 1) * r.wgs - 1, r.total);
}

// Whether row `t` sees any key; only asked for rows without weight.
__device__ __forceinline__ bool sees_any(const uint64_t *tree, int words, int context, int n, int64_t t) {
  if (context > 0 || tree == nullptr) return true;
  for (int w = 0; w < words && 64 * w < n; ++w) {
    uint64_t x = tree[t * words + w];
    if (n - 64 * w < 64) x &= (1ull << (n - 64 * w)) - 1;
    if (x) return true;
  }
  return false;
}

template <typename E, int N>
__device__ __forceinline__ void store_run(E *to, const float (&x)[N]) {
  Run<E, N> o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.x[i] = (E)x[i];
  *reinterpret_cast<Run<E, N> *>(to) = o;
}

// ---------------------------------------------------------------- the main kernel

// A buffer of `bytes` bytes: loads past its end return zeros without touching
// memory, so a missing tile (0 bytes) needs no branch around its loads.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, 0x00020000);
}
template <int WORDS>
__device__ __forceinline__ void load_words(__amdgpu_buffer_rsrc_t rs, int offset, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 1) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, offset, 0, 0);
  } else if constexpr (WORDS == 2) {
    const v2u v = __builtin_amdgcn_raw_buffer_load_b64(rs, offset, 0, 0);
    w[0] = v[0];
    w[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const v4u v = __builtin_amdgcn_raw_buffer_load_b128(rs, offset + 16 * i, 0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
    }
  }
}
__device__ __forceinline__ float load_scale(__amdgpu_buffer_rsrc_t rs, int offset) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, offset, 0, 0));
}

// 16 keys of a sequence, on the way to their address: the page is read ahead.
struct Keys16 {
  int page, in;  // the table's entry, and the first token within the page
};
// The 16 keys at `pos`, or those of the last key where they lie past it.
__device__ __forceinline__ Keys16 keys_at(const AttnArgs &p, const int *pages, int pos, int last) {
  const int at = min(pos, last);
  // 16 keys lie within a page (pages hold 16 tokens or more).
  return Keys16{uniform_load(pages + (at >> p.c.page_shift)), at & ((1 << p.c.page_shift) - 1) & ~15};
}
// The token row, of head kvh, where they begin.  poison: NaN, to be added to
// the scales, where the table holds no page of the cache.
__device__ __forceinline__ int64_t token_row(const AttnArgs &p, const Keys16 &k, int kvh, float &poison) {
  const bool ok = (uint32_t)k.page < p.c.pages;
  poison = ok ? 0.f : NAN;
  return (((int64_t)(ok ? k.page : 0) * p.c.heads + kvh) << p.c.page_shift) + k.in;
}

// How much larger (as a power of two) a score may be than the maximum its row
// keeps before the row's sums are scaled down to it: weights stay below 2^8, and
// most tiles leave the sums as they are.
constexpr float kMaxSlack = 8.f;

// The largest of a row's values over the lanes that hold its keys: four groups
// of 16 lanes, and PACK places within each.
template <int PACK>
__device__ __forceinline__ float row_max(float x) {
  if constexpr (PACK == 4) x = fmaxf(x, dpp<0x124>(x));  // row_ror:4
  if constexpr (PACK >= 2) x = fmaxf(x, dpp<0x128>(x));  // row_ror:8
  return across_groups_max(x);
}
template <int PACK>
__device__ __forceinline__ float row_sum(float x) {
  if constexpr (PACK == 4) x += dpp<0x124>(x);
  if constexpr (PACK >= 2) x += dpp<0x128>(x);
  return across_groups_sum(x);
}

// Scores, up to the row's factor undo[rt], to weights against the rows' kept maxima.
template <int NRT, int NK, int NB, int PACK>
__device__ __forceinline__ void weigh(float (&s)[NRT][NK], const float *undo, float *m, float *l, v4f (*acc)[NB][2]) {
  float top[NRT];
  bool above = false;
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt) {
    top[rt] = s[rt][0];
#pragma unroll
    for (int k = 1; k < NK; ++k) top[rt] = fmaxf(top[rt], s[rt][k]);
    top[rt] = row_max<PACK>(top[rt]) * undo[rt];
    above |= top[rt] > m[rt] + kMaxSlack;  // the first key that is seen, too
  }
  if (__ballot(above) != 0) {
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      const float to = fmaxf(m[rt], top[rt]);
      const float f = __builtin_amdgcn_exp2f(m[rt] - (to == -INFINITY ? 0.f : to));
      m[rt] = to;
      l[rt] *= f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[rt][b][i] *= f;
    }
  }
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt) {
    // Nothing seen yet: weights are exp2(-inf) = 0.
    const float from = m[rt] == -INFINITY ? 0.f : m[rt];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      s[rt][k] = __builtin_amdgcn_exp2f(fmaf(s[rt][k], undo[rt], -from));
      sum += s[rt][k];
    }
    l[rt] += sum;
  }
}

// Keeps the arithmetic behind x on this side of what follows: otherwise the
// compiler spreads one step's operands over all steps and runs out of registers.
__device__ __forceinline__ void pin(float &x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void pin(v4f &x) { asm volatile("" : "+v"(x)); }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

template <RowType T, int DIM, int RT_>
struct Attn {
  typedef typename AttnElem<T>::type E;
  static constexpr int RT = RT_;
  static constexpr int NB = DIM / 32;             // blocks
  static constexpr int QP = AttnElem<T>::kQParts;
  static constexpr int PP = AttnElem<T>::kPParts;
  static constexpr int PACK = 1, NK = 8;          // keys of a tile per lane
  static constexpr int KW = DIM / 16;             // words of a lane's quarter row of K
  static constexpr int VW = DIM / 64;             // words of a lane's pairs of V
  static constexpr int SW = (4 * NB + 15) / 16;   // scale words per lane for 4 keys
  static constexpr int ROWS = 16 * RT;
  static constexpr int PITCH = DIM + 4;           // LDS row of sums; 16 rows then start 4 banks apart

  // Codes and scales of one 32-key tile: 16-key half h in kw[h] / ks[h]; keys
  // 16 h + 4 c + i in vw[4 h + i], vs[h] (c the lane's group).
  struct Tile {
    uint32_t kw[2][KW];
    float ks[2][SW];
    uint32_t vw[8][VW];
    float vs[2][SW];
    float poison[2];  // as token_row gives it
  };
  v4u qf[RT][NB][QP];
  v4f acc[RT][NB][2];
  float m[RT], l[RT], undo[RT];

  const AttnArgs *p;
  float scale;       // alpha log2 e, multiplied into the key scales
  int row, c;        // lane % 16 and lane / 16

  __device__ __forceinline__ int row_of(int rt) const { return 16 * rt + row; }  // of the item
  __device__ __forceinline__ bool holds_row() const { return true; }             // in its sums
  __device__ __forceinline__ void start() {}

  // live: 0 for a tile that does not exist (nothing is read), 1 otherwise.
  // Scales are left as they come: arithmetic here would wait for them.
  __device__ __forceinline__ void load_k(Tile &t, const int64_t (&base)[2], const float (&poison)[2], int live) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t.poison[h] = poison[h];
      load_words<KW>(buffer_of(p->c.K + base[h] * DIM, 16 * DIM * live), row * DIM + c * (DIM / 4), t.kw[h]);
      const __amdgpu_buffer_rsrc_t rs = buffer_of(p->c.KS + base[h] * NB, 64 * NB * live);
#pragma unroll
      for (int w = 0; w < SW; ++w)
        t.ks[h][w] = load_scale(rs, 4 * (4 * c * NB + (16 * w + row) % (4 * NB)));
    }
  }
  __device__ __forceinline__ void load_v(Tile &t, const int64_t (&base)[2], int live) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __amdgpu_buffer_rsrc_t codes = buffer_of(p->c.V + base[h] * DIM, 16 * DIM * live);
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words<VW>(codes, (4 * c + i) * DIM + row * (DIM / 16), t.vw[4 * h + i]);
      const __amdgpu_buffer_rsrc_t rs = buffer_of(p->c.VS + base[h] * NB, 64 * NB * live);
#pragma unroll
      for (int w = 0; w < SW; ++w)
        t.vs[h][w] = load_scale(rs, 4 * (4 * c * NB + (16 * w + row) % (4 * NB)));
    }
  }

  // Once the key scales are used: marks the value scales of a missing page.
  __device__ __forceinline__ void add_poison(Tile &t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < SW; ++w) t.vs[h][w] += t.poison[h];
  }

  // Scores of the tile: s[rt][4 h + i] for key 16 h + 4 c + i and row `row` of row tile rt.
  __device__ __forceinline__ void scores(Tile &t, float (&s)[RT][8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < SW; ++w) t.ks[h][w] = fmaf(t.ks[h][w], scale, t.poison[h]);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[rt][k] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      static_for<0, NB>([&](auto b_) {
        constexpr int b = decltype(b_)::value;
        v4u a;
#pragma unroll
        for (int jl = 0; jl < 4; ++jl) {
          constexpr int byte = 2 * b;  // within the pair's NB * 2 bytes
          a[jl] = pair_f16(t.kw[h][jl * VW + byte / 4], (byte / 2) % 2);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = QP - 1; q >= 0; --q) x = mfma_f16(a, qf[rt][b][q], x);  // small parts first
          static_for<0, 4>([&](auto i_) {
            constexpr int i = decltype(i_)::value;
            constexpr int e = i * NB + b;
            s[rt][4 * h + i] += bcast<e % 16>(t.ks[h][e / 16]) * x[i];
            pin(s[rt][4 * h + i]);
          });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  }

  // sees[rt]: bit k for key k of the tile.  Keys a row does not see get the
  // score of no weight.  Their value scales may be anything: a scale that is
  // not finite is taken out, and the rows that do see it are remembered in
  // lost[rt], bit b for block b.  Returns whether there is any such scale.
  __device__ __forceinline__ bool mask(Tile &t, float (&s)[RT][8], const uint32_t (&sees)[RT], uint32_t (&lost)[RT]) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (!((sees[rt] >> (16 * (k / 4) + 4 * c + k % 4)) & 1)) s[rt][k] = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < SW; ++w) bad |= !finite(t.vs[h][w]);
    if (__ballot(bad) == 0) return false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) lost[rt] = 0;
    static_for<0, 8>([&](auto k_) {
      static_for<0, NB>([&](auto b_) {
        constexpr int k = decltype(k_)::value, b = decltype(b_)::value, e = (k % 4) * NB + b;
        const bool gone = !finite(bcast<e % 16>(t.vs[k / 4][e / 16]));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (gone && ((sees[rt] >> (16 * (k / 4) + 4 * c + k % 4)) & 1)) lost[rt] |= 1u << b;
      });
    });
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      lost[rt] |= __shfl_xor(lost[rt], 16);
      lost[rt] |= __shfl_xor(lost[rt], 32);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < SW; ++w) t.vs[h][w] = finite(t.vs[h][w]) ? t.vs[h][w] : 0.f;
    return true;
  }

  __device__ __forceinline__ void values(const Tile &t, const float (&s)[RT][8]) {
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      // Lane: codes of keys (k index 4 h + i) at channels 32 b + 2 row + 0, 1.
      v4u a[2];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint32_t w0 = t.vw[2 * kk][b / 2], w1 = t.vw[2 * kk + 1][b / 2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x0 = (float)(int8_t)(w0 >> (16 * (b % 2) + 8 * i));
          const float x1 = (float)(int8_t)(w1 >> (16 * (b % 2) + 8 * i));
          a[i][kk] = pack_hi(x0, x1);
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float w[8];
        static_for<0, 8>([&](auto k_) {
          constexpr int k = decltype(k_)::value;
          constexpr int e = (k % 4) * NB + b;
          w[k] = bcast<e % 16>(t.vs[k / 4][e / 16]) * s[rt][k];
        });
        v4u parts[PP];
        split8<PP>(w, parts);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = PP - 1; q >= 0; --q) acc[rt][b][i] = mfma(a[i], parts[q], acc[rt][b][i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) pin(acc[rt][b][i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
};

// The same for items of at most 16 / PACK rows (one new token of a small group;
// 24 sequences of 4096 keys, dim 64, 4 rows of f32: 41.6 us, 45.1 with 16-row
// items; one sequence of 1000 keys, dim 128: 15.9 and 16.6):
// the query's columns repeat PACK times across the matrix operand, so that the
// lanes of a row's repeats hold the same scores, and each keeps a PACK-th of the
// keys (KPL).  Exponentials, weights and their parts, most of the other
// kernel's instructions, are then made once instead of PACK times; the parts
// return to the lanes of the first columns by DPP as matrix operands.  Scores
// take biased codes (one instruction a pair); what the bias adds, 128 times the
// sum of the query's block, is taken off the packed products.
template <RowType T, int DIM, int PACK_>
struct AttnFew {
  typedef typename AttnElem<T>::type E;
  static constexpr int RT = 1, PACK = PACK_, NK = 8 / PACK;
  static constexpr int NB = DIM / 32;
  static constexpr int QP = AttnElem<T>::kQParts;
  static constexpr int PP = AttnElem<T>::kPParts;
  static constexpr int KW = DIM / 16, VW = DIM / 64;
  static constexpr int ROWS = 16 / PACK;
  static constexpr int PITCH = DIM + 4;

  // As in the other kernel, but for the scales: those of the lane's NK keys,
  // key by key.
  struct Tile {
    uint32_t kw[2][KW];
    uint32_t vw[8][VW];
    Run<float, NK * NB> ks, vs;
    float poison;
  };
  v4u qf[1][NB][QP];
  v4f acc[1][NB][2];
  float m[1], l[1], undo[1];
  float bias[NB];

  const AttnArgs *p;
  float scale;
  int row, c;

  __device__ __forceinline__ int row_of(int) const { return row % ROWS; }
  __device__ __forceinline__ bool holds_row() const { return row < ROWS; }
  __device__ __forceinline__ int part() const { return row / ROWS; }
  // The lane's first key within the tile: the others follow it.
  __device__ __forceinline__ int first_key() const {
    return PACK == 4 ? 16 * (part() / 2) + 4 * c + 2 * (part() % 2) : 16 * part() + 4 * c;
  }
  __device__ __forceinline__ bool upper_half() const { return part() >= PACK / 2; }

  // After the query: its blocks' sums.
  __device__ __forceinline__ void start() {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float x = 0.f;
#pragma unroll
      for (int q = QP - 1; q >= 0; --q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v2h h = __builtin_bit_cast(v2h, (uint32_t)qf[0][b][q][i]);
          x += (float)h.x + (float)h.y;
        }
      bias[b] = across_groups_sum(x) * (128.f * kBiasedUnit);
    }
  }

  __device__ __forceinline__ void load_scales(const float *from, const int64_t (&base)[2], Run<float, NK * NB> &to) {
    to = *reinterpret_cast<const Run<float, NK * NB> *>(from + ((upper_half() ? base[1] : base[0]) + first_key() % 16) * NB);
  }
  __device__ __forceinline__ void load_k(Tile &t, const int64_t (&base)[2], const float (&poison)[2], int live) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load_words<KW>(buffer_of(p->c.K + base[h] * DIM, 16 * DIM * live), row * DIM + c * (DIM / 4), t.kw[h]);
    load_scales(p->c.KS, base, t.ks);
    t.poison = upper_half() ? poison[1] : poison[0];
  }
  __device__ __forceinline__ void load_v(Tile &t, const int64_t (&base)[2], int live) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __amdgpu_buffer_rsrc_t codes = buffer_of(p->c.V + base[h] * DIM, 16 * DIM * live);
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words<VW>(codes, (4 * c + i) * DIM + row * (DIM / 16), t.vw[4 * h + i]);
    }
    load_scales(p->c.VS, base, t.vs);
  }

  __device__ __forceinline__ void add_poison(Tile &t) {
#pragma unroll
    for (int e = 0; e < NK * NB; ++e) t.vs.x[e] += t.poison;
  }

  // s[k]: the lane's k-th key.
  __device__ __forceinline__ void scores(Tile &t, float (&s)[1][NK]) {
    const float unit = scale * (1.f / kBiasedUnit);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < KW; ++w) t.kw[h][w] ^= 0x80808080u;
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      v4f x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4u a;
#pragma unroll
        for (int jl = 0; jl < 4; ++jl) a[jl] = pair_biased(t.kw[h][jl * VW + b / 2], b % 2);
        x[h] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = QP - 1; q >= 0; --q) x[h] = mfma_f16(a, qf[0][b][q], x[h]);
      }
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        float y;
        if constexpr (PACK == 4) {
          y = in_bank<1>(x[0][k], x[0][2 + k]);
          y = in_bank<2>(y, x[1][k]);
          y = in_bank<3>(y, x[1][2 + k]);
        } else {
          y = in_bank<2>(x[0][k], x[1][k]);
          y = in_bank<3>(y, x[1][k]);
        }
        const float ks = fmaf(t.ks.x[k * NB + b], unit, t.poison);
        s[0][k] = b == 0 ? ks * (y - bias[b]) : fmaf(ks, y - bias[b], s[0][k]);
        pin(s[0][k]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  // other, in lanes 4 BANK .. 4 BANK + 3 of each 16.
  template <int BANK>
  static __device__ __forceinline__ float in_bank(float x, float other) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(__float_as_int(x), __float_as_int(other), 0xe4, 0xf, 1 << BANK, false));
  }

  __device__ __forceinline__ bool mask(Tile &t, float (&s)[1][NK], const uint32_t (&sees)[1], uint32_t (&lost)[1]) {
    const uint32_t mine = sees[0] >> first_key();
    bool bad = false;
#pragma unroll
    for (int k = 0; k < NK; ++k)
      if (!((mine >> k) & 1)) s[0][k] = -INFINITY;
#pragma unroll
    for (int e = 0; e < NK * NB; ++e) bad |= !finite(t.vs.x[e]);
    if (__ballot(bad) == 0) return false;
    uint32_t gone = 0;
#pragma unroll
    for (int e = 0; e < NK * NB; ++e)
      if (!finite(t.vs.x[e])) {
        gone |= ((mine >> (e / NB)) & 1) << (e % NB);
        t.vs.x[e] = 0.f;
      }
    if constexpr (PACK == 4) gone |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)gone, 0x124, 0xf, 0xf, true);
    gone |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)gone, 0x128, 0xf, 0xf, true);
    gone |= __shfl_xor(gone, 16);
    gone |= __shfl_xor(gone, 32);
    lost[0] = gone;
    return true;
  }

  __device__ __forceinline__ void values(const Tile &t, const float (&s)[1][NK]) {
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      v4u a[2];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint32_t w0 = t.vw[2 * kk][b / 2], w1 = t.vw[2 * kk + 1][b / 2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x0 = (float)(int8_t)(w0 >> (16 * (b % 2) + 8 * i));
          const float x1 = (float)(int8_t)(w1 >> (16 * (b % 2) + 8 * i));
          a[i][kk] = pack_hi(x0, x1);
        }
      }
      float w[NK];
#pragma unroll
      for (int k = 0; k < NK; ++k) w[k] = t.vs.x[k * NB + b] * s[0][k];
      v4u parts[PP];
#pragma unroll
      for (int q = 0; q < PP; ++q)
#pragma unroll
        for (int d = 0; d < NK / 2; ++d) {
          const bool rest = PP < 3 && q + 1 == PP;
          const uint32_t pair = rest ? pack_near(w[2 * d], w[2 * d + 1]) : pack_hi(w[2 * d], w[2 * d + 1]);
          if (q + 1 < PP) {
            w[2 * d] = less<0>(pair, w[2 * d]);
            w[2 * d + 1] = less<1>(pair, w[2 * d + 1]);
          }
          parts[q][d] = pair;
          if constexpr (PACK == 4) {  // keys 2 m, 2 m + 1 of the operand are those of part m's lanes
            parts[q][1] = shifted<4>(pair);
            parts[q][2] = shifted<8>(pair);
            parts[q][3] = shifted<12>(pair);
          } else {
            parts[q][2 + d] = shifted<8>(pair);
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int q = PP - 1; q >= 0; --q) acc[0][b][i] = mfma(a[i], parts[q], acc[0][b][i]);
        pin(acc[0][b][i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  template <int BY>
  static __device__ __forceinline__ uint32_t shifted(uint32_t x) {  // from BY lanes above (row_shl)
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x100 + BY, 0xf, 0xf, true);
  }
};

// Bit k: whether the row at index `i` among its sequence's new tokens (row t
// of q) sees key base + k.
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs &p, int base, int context, int length, int i, int64_t t) {
  const int left = length - base;  // keys that exist; more than 0
  uint32_t seen = left >= 32 ? 0xffffffffu : (1u << left) - 1;
  if (p.tree == nullptr) {
    const int upto = context + i + 1 - base;
    return upto >= 32 ? seen : upto <= 0 ? 0u : seen & ((1u << upto) - 1);
  }
  const int before = context - base;  // keys before the new tokens
  if (before >= 32) return seen;
  const uint64_t *words = p.tree + t * p.tree_words;
  uint32_t tree;
  if (before > 0) {
    tree = (p.tree_words > 0 ? (uint32_t)words[0] << before : 0u) | ((1u << before) - 1);
  } else {
    const int j = -before, w = j >> 6, off = j & 63;
    uint64_t x = w < p.tree_words ? words[w] >> off : 0;
    if (off > 32 && w + 1 < p.tree_words) x |= words[w + 1] << (64 - off);
    tree = (uint32_t)x;
  }
  return seen & tree;
}

// One workgroup's share of one item: units k0 .. k1 - 1 of its keys.
struct Share {
  Seq seq;
  const int *pages;  // the sequence's table row
  int kvh, head0, sub_heads;
  int i0, tokens, rows;  // the item's first token among the new ones, its tokens, tokens x heads
  int context;           // tokens before the new ones
  int keys;              // keys the item's rows may see
  int all;               // keys that all of its rows see
  int k0, k1;
  int shift;             // log2 of the keys of a unit
  bool whole;            // all of the item's units
  float *slot;           // where the sums go otherwise
};

// Walks through the shares of this workgroup's run.  slot_rows: rows of a slot.
template <int DIM, typename F>
__device__ __forceinline__ void walk_shares(const AttnArgs &p, int slot_rows, int tid, F work) {
  // Neighbouring runs, which may share keys or an item, on one XCD.
  const int per_xcd = gridDim.x / kXcds;
  const int wg = gridDim.x % kXcds == 0 ? (int)(blockIdx.x % kXcds) * per_xcd + (int)blockIdx.x / kXcds : (int)blockIdx.x;
  const RunStart run = find_run(p, wg, gridDim.x, tid & 63);
  if (tid == 0 && p.items != nullptr) p.items[wg].valid = 0;
  if (wg >= run.wgs) return;

  // Where the run begins: sequence b, head vh (with its sub-group), row item r, unit k0.
  Share h;
  int b = run.b;
  h.seq = run.seq;
  int vh, r;
  {
    const int64_t per_head = head_units(p, h.seq);
    vh = (int)quotient(run.rest, per_head);
    int64_t rest = run.rest - vh * per_head;
    if (p.tree != nullptr || h.seq.bad) {
      const int u = item_units(p, h.seq, 0);
      r = min((int)quotient(rest, u), row_items(p, h.seq) - 1);
      h.k0 = (int)(rest - (int64_t)r * u);
    } else {
      r = 0;
      while (rest >= item_units(p, h.seq, r)) rest -= item_units(p, h.seq, r++);
      h.k0 = (int)rest;
    }
  }

  int v0 = h.k0;  // units into the item, its cost included
  for (int64_t unit = run.begin;;) {
    const int units = item_units(p, h.seq, r);
    const int64_t left = run.end - unit;
    const int v1 = left < units - v0 ? v0 + (int)left : units;
    h.k0 = max(v0 - p.item_cost, 0);
    h.k1 = max(v1 - p.item_cost, 0);
    h.whole = h.k0 == 0 && v1 == units;
    h.shift = item_shift(p, h.seq, r);
    h.kvh = vh / p.subs;
    const int sub = vh - h.kvh * p.subs;
    h.sub_heads = min(p.sub_heads, p.group - sub * p.sub_heads);
    h.head0 = h.kvh * p.group + sub * p.sub_heads;
    h.i0 = r * p.tile_tokens;
    h.tokens = min(p.tile_tokens, h.seq.n - h.i0);
    h.rows = h.tokens * h.sub_heads;
    h.context = h.seq.length - h.seq.n;
    h.keys = item_keys(p, h.seq, r);
    h.all = p.tree != nullptr ? h.context : h.context + h.i0 + 1;
    h.pages = p.s.table + (int64_t)b * p.s.table_stride;
    // Slot 1 holds the run's last item, cut short at its end; slot 0 an item
    // that an earlier run began.
    h.slot = p.partial + (2 * (int64_t)wg + (h.k0 == 0 ? 1 : 0)) * attn_slot_floats(slot_rows, DIM);
    if (h.k1 > 0) work(h);
    if (tid == 0 && h.k0 == 0 && h.k1 > 0 && !h.whole) {
      AttnItem it;
      it.valid = 1;
      it.last = wg_of(unit - v0 + units - 1, run);
      it.row0 = h.seq.start + h.i0;
      it.tokens = h.tokens;
      it.head0 = h.head0;
      it.heads = h.sub_heads;
      it.seq_new = h.seq.n;
      it.context = h.context;
      p.items[wg] = it;
    }
    unit += v1 - v0;
    if (unit >= run.end) return;
    // The next item.
    v0 = 0;
    if (++r == row_items(p, h.seq)) {
      r = 0;
      if (++vh == p.c.heads * p.subs) {
        vh = 0;
        do {
          h.seq = uniform_seq_at(p.s, ++b);
        } while (h.seq.n == 0);
      }
    }
  }
}

// Channels of one finished row: sums over weight; zeros for a row that sees
// nothing, NaN for one of a sequence that is described wrongly.
template <int N>
__device__ __forceinline__ void finish_row(const AttnArgs &p, const Share &h, int64_t t, float weight, float (&x)[N]) {
  const float scale = h.seq.bad ? NAN : 1.f / weight;
  bool nothing = false;
  if (weight == 0.f && !h.seq.bad) nothing = !sees_any(p.tree, p.tree_words, h.context, h.seq.n, t);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = nothing ? 0.f : x[i] * scale;
}

template <RowType T, int DIM, int ROWS_>
struct AttnOf {
  typedef Attn<T, DIM, ROWS_ / 16> type;
};
template <RowType T, int DIM>
struct AttnOf<T, DIM, 4> {
  typedef AttnFew<T, DIM, 4> type;
};
template <RowType T, int DIM>
struct AttnOf<T, DIM, 8> {
  typedef AttnFew<T, DIM, 2> type;
};

// WAVES: 4, or 8 where a workgroup takes all keys of its items.
template <RowType T, int DIM, int ROWS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 ? kAttnWgsPerCu : 1) void attention_kernel(AttnArgs p) {
  typedef typename AttnOf<T, DIM, ROWS>::type A;
  typedef typename A::E E;
  constexpr int NB = A::NB, RT = A::RT, PITCH = A::PITCH, STEP = kAttnTile * WAVES;
  __shared__ __attribute__((aligned(16))) float sums[WAVES][ROWS][PITCH];
  __shared__ float tops[WAVES][ROWS], weights[WAVES][ROWS];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  A a;
  a.p = &p;
  a.scale = p.alpha * 1.4426950408889634f;
  a.row = tid & 15;
  a.c = (tid & 63) >> 4;

  walk_shares<DIM>(p, ROWS, tid, [&](const Share &h) {
    // The query's rows, the first tile and the second one's pages are asked
    // for before the first of them is needed.
    int index[RT];
    bool in[RT];
    QueryRow<T, DIM> q[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rho = a.row_of(rt);
      const int tok = rho / h.sub_heads;
      in[rt] = rho < h.rows;
      index[rt] = h.i0 + min(tok, h.tokens - 1);
      fetch_query<T, DIM>(p, h.seq.start + index[rt], in[rt] ? h.head0 + rho - tok * h.sub_heads : h.head0, a.c, q[rt]);
    }
    const int last = h.keys - 1;
    const int begin = (h.k0 << h.shift) + wave * kAttnTile;
    const int end = h.seq.bad ? 0 : min(h.k1 << h.shift, h.keys);
    Keys16 keys[2];  // a page's number is read one tile before the page
    int64_t base[2];
    float poison[2];
    auto ahead = [&](int at) {
#pragma unroll
      for (int k = 0; k < 2; ++k) keys[k] = keys_at(p, h.pages, at + 16 * k, last);
    };
    auto place = [&]() {
#pragma unroll
      for (int k = 0; k < 2; ++k) base[k] = token_row(p, keys[k], h.kvh, poison[k]);
    };
    typename A::Tile t;
    if (begin < end) {
      ahead(begin);
      place();
      ahead(begin + STEP);
      a.load_k(t, base, poison, 1);
      a.load_v(t, base, 1);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      a.undo[rt] = cut_query<T, DIM>(q[rt], in[rt], a.qf[rt]);
      a.m[rt] = -INFINITY;
      a.l[rt] = 0.f;
#pragma unroll
      for (int bb = 0; bb < NB; ++bb) a.acc[rt][bb][0] = a.acc[rt][bb][1] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    a.start();

    for (int at = begin; at < end; at += STEP) {
      // The next tile's parts are loaded as this one's are used up.
      const int more = at + STEP < end;
      place();
      ahead(at + 2 * STEP);
      float s[RT][A::NK];
      a.scores(t, s);
      a.add_poison(t);
      a.load_k(t, base, poison, more);
      bool some_lost = false;
      uint32_t lost[RT];
      if (at + kAttnTile > h.all) {
        uint32_t sees[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          sees[rt] = seen_bits(p, at, h.context, h.seq.length, index[rt], h.seq.start + index[rt]);
        some_lost = a.mask(t, s, sees, lost);
      }
      weigh<RT, A::NK, NB, A::PACK>(s, a.undo, a.m, a.l, a.acc);
      a.values(t, s);
      if (some_lost) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int bb = 0; bb < NB; ++bb)
            if (lost[rt] >> bb & 1) a.acc[rt][bb][0] = a.acc[rt][bb][1] = v4f{NAN, NAN, NAN, NAN};
      }
      a.load_v(t, base, more);
    }

    // The waves' sums, through LDS.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float l = row_sum<A::PACK>(a.l[rt]);
      if (!a.holds_row()) continue;
      if (a.c == 0) {
        tops[wave][a.row_of(rt)] = a.m[rt];
        weights[wave][a.row_of(rt)] = l;
      }
#pragma unroll
      for (int bb = 0; bb < NB; ++bb) {
        float *to = &sums[wave][a.row_of(rt)][32 * bb + 8 * a.c];
        const v4f x = a.acc[rt][bb][0], y = a.acc[rt][bb][1];  // channels 2 i and 2 i + 1 of the lane's eight
        *reinterpret_cast<v4f *>(to) = v4f{x[0], y[0], x[1], y[1]};
        *reinterpret_cast<v4f *>(to + 4) = v4f{x[2], y[2], x[3], y[3]};
      }
    }
    __syncthreads();
    for (int e = tid; e < h.rows * (DIM / 8); e += 64 * WAVES) {
      const int rho = e / (DIM / 8), d = 8 * (e % (DIM / 8));
      float top = tops[0][rho];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) top = fmaxf(top, tops[w][rho]);
      const float from = top == -INFINITY ? 0.f : top;
      float weight = 0.f, x[8] = {};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float f = __builtin_amdgcn_exp2f(tops[w][rho] - from);
        weight += f * weights[w][rho];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += f * sums[w][rho][d + i];
      }
      if (h.whole) {
        const int tok = rho / h.sub_heads;
        const int64_t t = h.seq.start + h.i0 + tok;
        finish_row(p, h, t, weight, x);
        store_run<E, 8>(static_cast<E *>(p.out) + t * p.out_stride + (int64_t)(h.head0 + rho - tok * h.sub_heads) * DIM + d, x);
      } else {
        v4f *to = reinterpret_cast<v4f *>(h.slot + (int64_t)rho * DIM + d);
        to[0] = v4f{x[0], x[1], x[2], x[3]};
        to[1] = v4f{x[4], x[5], x[6], x[7]};
        if (d == 0) {
          h.slot[(int64_t)ROWS * DIM + rho] = top;
          h.slot[(int64_t)ROWS * (DIM + 1) + rho] = weight;
        }
      }
    }
    __syncthreads();  // the sums are read before the next item's are written
  });
}

// ---------------------------------------------------------------- many rows

// The same for items of more rows (trees, prompts; 24 sequences of 4096 keys, 72
// rows of bf16, dim 128: 118 us, 130 with 32-row items): up to 64 * RT rows, 16 * RT
// for each wave, and all four waves take the same keys.  Converting the codes
// costs as much as the rest of the work on 32 rows, so a workgroup does it
// once: per step of 64 keys each wave loads 16 keys' codes, converts them and
// lays them into LDS as the matrix operands that all waves read (16 bytes per
// lane, conflict-free).  The next step's codes are in flight meanwhile.  Row
// tiles are dealt to the waves in turn, so a short item still uses all four.
constexpr int kWideKeys = 64;

template <int DIM>
struct WideLds {
  static constexpr int NB = DIM / 32;
  static constexpr int BUFS = DIM == 256 ? 1 : 2;  // two workgroups must fit a CU
  v4u k[BUFS][4][NB][64];     // 16-key tile, block, lane
  v2u v[BUFS][2][NB][2][64][2];  // 32-key group, block, pair element, lane, half
  float ks[BUFS][4][NB][16], vs[BUFS][4][NB][16];  // 16-key tile, block, key: a lane reads its four keys at once
  // Value scales that are not finite are zeros in vs; bit e % 64 of word e / 64
  // marks the one of key e / NB and block e % NB of a 16-key tile.
  uint64_t gone[BUFS][4][(16 * NB + 63) / 64];
};

template <RowType T, int DIM, int RT>
__global__ __launch_bounds__(kThreads, kAttnWgsPerCu) void attention_wide_kernel(AttnArgs p) {
  typedef typename AttnElem<T>::type E;
  constexpr int NB = DIM / 32, QP = AttnElem<T>::kQParts, PP = AttnElem<T>::kPParts;
  constexpr int KW = DIM / 16, VW = DIM / 64, SW = (4 * NB + 15) / 16;
  constexpr int ROWS = 64 * RT, BUFS = DIM == 256 ? 1 : 2;
  constexpr int SPL = (16 * NB + 63) / 64;  // scale words a lane stages
  __shared__ WideLds<DIM> lds;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, row = lane & 15, c = lane >> 4;

  const float scale = p.alpha * 1.4426950408889634f;  // multiplied into the key scales

  // This wave's 16 keys of a step, on their way to LDS.
  uint32_t kw[KW], vw[4][VW];
  float ksw[SPL], vsw[SPL];
  float poison = 0.f;
  // Offsets are made anew from the lane at each step: kept, they would be
  // spilled, and waiting for one to come back waits for all loads before it.
  auto load = [&](int64_t base) {
    int own = lane;
    asm volatile("" : "+v"(own));
    const int row = own & 15, c = own >> 4;
    load_words<KW>(buffer_of(p.c.K + base * DIM, 16 * DIM), row * DIM + c * (DIM / 4), kw);
    const __amdgpu_buffer_rsrc_t codes = buffer_of(p.c.V + base * DIM, 16 * DIM);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_words<VW>(codes, (4 * c + i) * DIM + row * (DIM / 16), vw[i]);
#pragma unroll
    for (int w = 0; w < SPL; ++w) {
      const int e = (64 * w + own) % (16 * NB);
      ksw[w] = p.c.KS[base * NB + e];
      vsw[w] = p.c.VS[base * NB + e];
    }
  };
  auto lay = [&](int buf) {
    int own = lane;
    asm volatile("" : "+v"(own));
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      v4u x;
#pragma unroll
      for (int jl = 0; jl < 4; ++jl) x[jl] = pair_f16(kw[jl * VW + b / 2], b % 2);
      lds.k[buf][wave][b][own] = x;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = (float)(int8_t)(vw[k][b / 2] >> (16 * (b % 2) + 8 * i));
        lds.v[buf][wave / 2][b][i][own][wave % 2] = v2u{pack_hi(y[0], y[1]), pack_hi(y[2], y[3])};
      }
    });
#pragma unroll
    for (int w = 0; w < SPL; ++w) {
      ksw[w] = fmaf(ksw[w], scale, poison);
      vsw[w] += poison;
      const uint64_t gone = __ballot(64 * w + own < 16 * NB && !finite(vsw[w]));
      if (own == 0) lds.gone[buf][wave][w] = gone;
      if (64 * w + own < 16 * NB) {
        const int e = 64 * w + own;  // key e / NB, block e % NB
        lds.ks[buf][wave][e % NB][e / NB] = ksw[w];
        lds.vs[buf][wave][e % NB][e / NB] = finite(vsw[w]) ? vsw[w] : 0.f;
      }
    }
  };

  walk_shares<DIM>(p, ROWS, tid, [&](const Share &h) {
    // The first step's codes are asked for before the query's rows are needed.
    const int last = h.keys - 1;
    const int begin = h.k0 << h.shift;
    const int end = h.seq.bad ? begin : min(h.k1 << h.shift, h.keys);
    auto load_at = [&](int at) {
      load(token_row(p, keys_at(p, h.pages, at + 16 * wave, last), h.kvh, poison));
    };
    // Row tile rt of this wave: rows 16 (4 rt + wave) .. of the item.
    v4u qf[RT][NB][QP];
    v4f acc[RT][NB][2];
    float m[RT], l[RT], undo[RT];
    int index[RT];
    bool in[RT];
    QueryRow<T, DIM> q[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rho = 16 * (4 * rt + wave) + row;
      const int tok = rho / h.sub_heads;
      in[rt] = rho < h.rows;
      index[rt] = h.i0 + min(tok, h.tokens - 1);
      fetch_query<T, DIM>(p, h.seq.start + index[rt], in[rt] ? h.head0 + rho - tok * h.sub_heads : h.head0, c, q[rt]);
    }
    if (begin < end) load_at(begin);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      undo[rt] = cut_query<T, DIM>(q[rt], in[rt], qf[rt]);
      m[rt] = -INFINITY;
      l[rt] = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[rt][b][0] = acc[rt][b][1] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    const int tiles = (h.rows + 15) / 16;
    const int mine = tiles <= wave ? 0 : (tiles - wave + 3) / 4;  // row tiles this wave has

    // One step over the 64 keys from `at` on, for the wave's first NRT row tiles.
    auto compute = [&](auto nrt_, int at, int buf) {
      constexpr int NRT = decltype(nrt_)::value;
      float s[NRT][16];
      {
        // Operands of product n + 1 are on their way while product n runs.
        v4u a[2];
        v4f ks[2];
        a[0] = lds.k[buf][0][0][lane];
        ks[0] = *reinterpret_cast<const v4f *>(&lds.ks[buf][0][0][4 * c]);
        static_for<0, 4 * NB>([&](auto n_) {
          constexpr int n = decltype(n_)::value, kt = n / NB, b = n % NB;
          if constexpr (n + 1 < 4 * NB) {
            a[(n + 1) % 2] = lds.k[buf][(n + 1) / NB][(n + 1) % NB][lane];
            ks[(n + 1) % 2] = *reinterpret_cast<const v4f *>(&lds.ks[buf][(n + 1) / NB][(n + 1) % NB][4 * c]);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt) {
            v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = QP - 1; q >= 0; --q) x = mfma_f16(a[n % 2], qf[rt][b][q], x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[rt][4 * kt + i] = b == 0 ? ks[n % 2][i] * x[i] : fmaf(ks[n % 2][i], x[i], s[rt][4 * kt + i]);
          }
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) pin(s[rt][4 * kt + i]);
        });
      }

      uint64_t sees[NRT];  // shifted: bit 16 kt + i is this lane's key i of tile kt
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) sees[rt] = ~0ull;
      if (at + kWideKeys > h.all) {
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) {
          const int64_t t = h.seq.start + index[rt];
          sees[rt] = seen_bits(p, at, h.context, h.seq.length, index[rt], t);
          if (at + 32 < h.seq.length)
            sees[rt] |= (uint64_t)seen_bits(p, at + 32, h.context, h.seq.length, index[rt], t) << 32;
          sees[rt] >>= 4 * c;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (!((sees[rt] >> (16 * (k / 4) + k % 4)) & 1)) s[rt][k] = -INFINITY;
        }
      }
      weigh<NRT, 16, NB, 1>(s, undo, m, l, acc);
      {
        v4u a[2][2];
        v4f vs[2][2];
        auto fetch = [&](auto n_) {
          constexpr int n = decltype(n_)::value, g = n / NB, b = n % NB;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[n % 2][i] = *reinterpret_cast<const v4u *>(&lds.v[buf][g][b][i][lane][0]);
            vs[n % 2][i] = *reinterpret_cast<const v4f *>(&lds.vs[buf][2 * g + i][b][4 * c]);
          }
        };
        fetch(std::integral_constant<int, 0>{});
        static_for<0, 2 * NB>([&](auto n_) {
          constexpr int n = decltype(n_)::value, g = n / NB, b = n % NB;
          if constexpr (n + 1 < 2 * NB) fetch(std::integral_constant<int, n + 1>{});
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt) {
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = vs[n % 2][k / 4][k % 4] * s[rt][8 * g + k];
            v4u parts[PP];
            split8<PP>(w, parts);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int q = PP - 1; q >= 0; --q) acc[rt][b][i] = mfma(a[n % 2][i], parts[q], acc[rt][b][i]);
          }
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int i = 0; i < 2; ++i) pin(acc[rt][b][i]);
        });
      }
      // Blocks of rows that see a value scale that is not finite are lost.
      uint64_t any = 0;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt)
#pragma unroll
        for (int w = 0; w < SPL; ++w) any |= lds.gone[buf][kt][w];
      if (uniform((int64_t)any) != 0) {
        uint32_t lost[NRT] = {};
#pragma unroll 1
        for (int kt = 0; kt < 4; ++kt)
#pragma unroll 1
          for (int e = 0; e < 4 * NB; ++e) {
            const int at_e = 4 * NB * c + e;  // key 4 c + e / NB, block e % NB
            if (lds.gone[buf][kt][at_e / 64] >> (at_e % 64) & 1)
#pragma unroll
              for (int rt = 0; rt < NRT; ++rt) lost[rt] |= (uint32_t)(sees[rt] >> (16 * kt + e / NB) & 1) << (e % NB);
          }
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) {
          lost[rt] |= __shfl_xor(lost[rt], 16);
          lost[rt] |= __shfl_xor(lost[rt], 32);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            if (lost[rt] >> b & 1) acc[rt][b][0] = acc[rt][b][1] = v4f{NAN, NAN, NAN, NAN};
        }
      }
    };

    if (begin < end) {
      lay(0);
      if (begin + kWideKeys < end) load_at(begin + kWideKeys);
      __syncthreads();
      auto steps = [&](auto nrt_) {
        for (int at = begin; at < end; at += kWideKeys) {
          const int buf = BUFS == 2 ? (at - begin) / kWideKeys % 2 : 0;
          if constexpr (decltype(nrt_)::value > 0) compute(nrt_, at, buf);
          if constexpr (BUFS == 1) __syncthreads();
          if (at + kWideKeys < end) {
            lay(BUFS == 2 ? buf ^ 1 : 0);
            if (at + 2 * kWideKeys < end) load_at(at + 2 * kWideKeys);
          }
          __syncthreads();
        }
      };
      if (RT == 2 && mine == 2)
        steps(std::integral_constant<int, RT>{});
      else if (mine >= 1)
        steps(std::integral_constant<int, 1>{});
      else
        steps(std::integral_constant<int, 0>{});
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rho = 16 * (4 * rt + wave) + row;
      const float weight = across_groups_sum(l[rt]);
      if (rho >= h.rows) continue;
      const int tok = rho / h.sub_heads;
      const int64_t t = h.seq.start + h.i0 + tok;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const v4f u = acc[rt][b][0], v = acc[rt][b][1];
        float x[8] = {u[0], v[0], u[1], v[1], u[2], v[2], u[3], v[3]};
        const int d = 32 * b + 8 * c;
        if (h.whole) {
          finish_row(p, h, t, weight, x);
          store_run<E, 8>(static_cast<E *>(p.out) + t * p.out_stride + (int64_t)(h.head0 + rho - tok * h.sub_heads) * DIM + d, x);
        } else {
          v4f *to = reinterpret_cast<v4f *>(h.slot + (int64_t)rho * DIM + d);
          to[0] = v4f{x[0], x[1], x[2], x[3]};
          to[1] = v4f{x[4], x[5], x[6], x[7]};
        }
      }
      if (!h.whole && c == 0) {
        h.slot[(int64_t)ROWS * DIM + rho] = m[rt];
        h.slot[(int64_t)ROWS * (DIM + 1) + rho] = weight;
      }
    }
  });
}

// ---------------------------------------------------------------- joining the parts

// Rows that a wave of the join takes: four channels of a row per lane.  One row
// per wave took twice as long for 128-row items of dim 64 (whose join takes 8.6 us
// for the pieces of prompts above).
constexpr int join_rows(int dim) { return 256 / dim; }

// Workgroup (y, w): the split item that workgroup w began, and its y-th run of
// kWaves * join_rows rows; parts are taken in key order.  Runs come first in the
// grid: split items often begin every 2nd, 4th ... workgroup, and with w first
// they would all land on a few of the XCDs and take twice as long (512 slots of
// 128 rows of dim 128, 34 MB: 10 us as it is).
template <RowType T, int DIM>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnArgs p, int slot_rows) {
  typedef typename AttnElem<T>::type E;
  const int first = blockIdx.y;
  const AttnItem it = p.items[first];
  if (!it.valid) return;
  constexpr int LANES = 64 / join_rows(DIM);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = lane & (LANES - 1);
  const int live = it.tokens * it.heads, rho0 = (blockIdx.x * kWaves + wave) * join_rows(DIM);
  if (rho0 >= live) return;
  const bool mine = rho0 + lane / LANES < live;
  const int rho = mine ? rho0 + lane / LANES : rho0;
  const int64_t size = attn_slot_floats(slot_rows, DIM);
  const int parts = __builtin_amdgcn_readfirstlane(it.last) - first + 1;
  // Contributor k: the first one's slot 1, then slot 0 of the following ones.
  const float *base = p.partial + (2 * (int64_t)first + 1) * size;
  auto part = [&](int k) { return k == 0 ? base : p.partial + 2 * (int64_t)(first + k) * size; };
  // Eight parts' rows in flight, where there are more than two (32 parts: 7 us,
  // 8 with four); past the last one the last one again, unused.
  constexpr int AHEAD = 8;
  v4f y[AHEAD];
  auto load = [&](int k) {
    auto some = [&](auto from, auto to) {
#pragma unroll
      for (int u = decltype(from)::value; u < decltype(to)::value; ++u)
        y[u] = *reinterpret_cast<const v4f *>(part(min(k + u, parts - 1)) + (int64_t)rho * DIM + c * 4);
    };
    some(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{});
    if (k + 2 < parts) some(std::integral_constant<int, 2>{}, std::integral_constant<int, AHEAD>{});
  };
  load(0);
  // The largest maximum, then the parts' factors, a lane per part.
  float top = -INFINITY;
  for (int k = c; k < parts; k += LANES) top = fmaxf(top, part(k)[(int64_t)slot_rows * DIM + rho]);
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float from = top == -INFINITY ? 0.f : top;
  float weight = 0.f, f = 0.f, wt = 0.f;
  float x[4] = {};
  for (int k = 0;;) {
    if ((k & (LANES - 1)) == 0) {
      f = wt = 0.f;
      if (k + c < parts) {
        const float *s = part(k + c) + (int64_t)slot_rows * DIM + rho;
        f = __builtin_amdgcn_exp2f(s[0] - from);
        wt = f * s[slot_rows];
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (k + u >= parts) break;
      const int from_lane = (k + u) & (LANES - 1);
      const float g = __shfl(f, from_lane, LANES);
      weight += __shfl(wt, from_lane, LANES);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += g * y[u][i];
    }
    k += AHEAD;
    if (k >= parts) break;
    load(k);
  }
  if (!mine) return;
  const int tok = rho / it.heads;
  const int64_t t = it.row0 + tok;
  bool nothing = false;
  if (weight == 0.f) nothing = !sees_any(p.tree, p.tree_words, it.context, it.seq_new, t);
  const float scale = 1.f / weight;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = nothing ? 0.f : x[i] * scale;
  store_run<E, 4>(static_cast<E *>(p.out) + t * p.out_stride + (int64_t)(it.head0 + rho - tok * it.heads) * DIM + c * 4, x);
}

template <RowType T, int DIM, int ROWS>
hipError_t launch_instance(const AttnArgs &a, int wgs, hipStream_t stream) {
  if constexpr (ROWS >= 64)
    hipLaunchKernelGGL((attention_wide_kernel<T, DIM, ROWS / 64>), dim3((unsigned)wgs), dim3(kThreads), 0, stream, a);
  else if (ROWS <= 16 && a.items == nullptr)
    hipLaunchKernelGGL((attention_kernel<T, DIM, ROWS, ROWS <= 16 ? 8 : 4>), dim3((unsigned)wgs), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((attention_kernel<T, DIM, ROWS, 4>), dim3((unsigned)wgs), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.items == nullptr) return e;  // without items none is split
  hipLaunchKernelGGL((attention_join_kernel<T, DIM>), dim3((ROWS + kWaves * join_rows(DIM) - 1) / (kWaves * join_rows(DIM)), (unsigned)wgs),
                     dim3(kThreads), 0, stream, a, ROWS);
  return hipGetLastError();
}

template <RowType T, int DIM>
hipError_t launch_rows(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  if constexpr (DIM <= 128) {
    if (rows == 4) return launch_instance<T, DIM, 4>(a, wgs, stream);
    if (rows == 8) return launch_instance<T, DIM, 8>(a, wgs, stream);
  }
  if (rows == 16) return launch_instance<T, DIM, 16>(a, wgs, stream);
  if constexpr (attn_direct_rows(DIM) == 32)
    if (rows == 32) return launch_instance<T, DIM, 32>(a, wgs, stream);
  if (rows == 64) return launch_instance<T, DIM, 64>(a, wgs, stream);
  if constexpr (attn_max_rows(T, DIM) == 128)
    if (rows == 128) return launch_instance<T, DIM, 128>(a, wgs, stream);
  return hipErrorInvalidValue;
}

// rows: of an item, a power of two from 4 to 128.
template <RowType T>
hipError_t launch_attention(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  switch (a.c.dim) {
    case 64: return launch_rows<T, 64>(a, rows, wgs, stream);
    case 128: return launch_rows<T, 128>(a, rows, wgs, stream);
    case 256: return launch_rows<T, 256>(a, rows, wgs, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace q8
