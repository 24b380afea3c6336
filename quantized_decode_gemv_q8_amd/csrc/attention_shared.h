// What the attentions over the caches share, whatever the cache holds: the work
// list, the masks, the running softmax, the kernel whose waves take different
// keys, and the join of split items.
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

// The same of the lanes 16 and 32 apart, by swaps of rows and halves of the wave:
// no trip through LDS, whose latency the running softmax would wait for.
__device__ __forceinline__ float across_groups_max(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float across_groups_sum(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
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

// ---------------------------------------------------------------- keys and weights

// A buffer of `bytes` bytes: loads past its end return zeros without touching
// memory, so a missing tile (0 bytes) needs no branch around its loads.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, 0x00020000);
}
template <int WORDS, int AUX = 0>
__device__ __forceinline__ void load_words(__amdgpu_buffer_rsrc_t rs, int offset, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 1) {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, offset, 0, AUX);
  } else if constexpr (WORDS == 2) {
    const v2u v = __builtin_amdgcn_raw_buffer_load_b64(rs, offset, 0, AUX);
    w[0] = v[0];
    w[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const v4u v = __builtin_amdgcn_raw_buffer_load_b128(rs, offset + 16 * i, 0, AUX);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
    }
  }
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

// Raises the rows' kept maxima where a score, up to the row's factor undo[rt], passes
// one by kMaxSlack, and scales the rows' sums down to the new ones.  Every lane looks at
// its own keys; the row's largest is only made where one of them passes.
template <int NRT, int NK, int NB, int PACK>
__device__ __forceinline__ void settle(const float (&s)[NRT][NK], const float *undo, float *m, float *l, v4f (*acc)[NB][2]) {
  float top[NRT];
  bool above = false;
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt) {
    top[rt] = s[rt][0];
#pragma unroll
    for (int k = 1; k < NK; ++k) top[rt] = fmaxf(top[rt], s[rt][k]);
    above |= top[rt] * undo[rt] > m[rt] + kMaxSlack;  // the first key that is seen, too
  }
  if (__ballot(above) != 0) {
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      const float to = fmaxf(m[rt], row_max<PACK>(top[rt]) * undo[rt]);
      const float f = __builtin_amdgcn_exp2f(m[rt] - (to == -INFINITY ? 0.f : to));
      m[rt] = to;
      l[rt] *= f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[rt][b][i] *= f;
    }
  }
}

// What a row's scores are taken against: its kept maximum.  Nothing seen yet: weights
// are exp2(-inf) = 0.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

// Scores, up to the row's factor undo[rt], a power of two, to weights against the rows'
// kept maxima.
template <int NRT, int NK, int NB, int PACK>
__device__ __forceinline__ void weigh(float (&s)[NRT][NK], const float *undo, float *m, float *l, v4f (*acc)[NB][2]) {
  settle<NRT, NK, NB, PACK>(s, undo, m, l, acc);
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt) {
    const float from = base_of(m[rt]);
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
__device__ __forceinline__ void pin(v4u &x) { asm volatile("" : "+v"(x)); }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

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

// A: how a wave takes a tile of 32 keys from a cache's codes to scores and sums
// (loads, scores, masks, weights, values).  WAVES: 4, or 8 where a workgroup takes all
// keys of its items.
template <class A, RowType T, int DIM, int ROWS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 ? A::WGS : 1) void attention_kernel(AttnArgs p) {
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
      a.cut(rt, q[rt], in[rt]);
      a.no_top(rt);
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
      a.weights(s);
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
        tops[wave][a.row_of(rt)] = a.top(rt);
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

}  // namespace
}  // namespace q8
