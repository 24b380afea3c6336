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
// are not used here.  A batch of 32 ragged sequences (316 MB) takes 62 to 67 us and its
// join 5, two sequences of 131072 keys (604 MB) 112 and 7.  From 16 rows on:
// vector instructions, for the codes' conversion, the exponentials and the
// weights' parts.  68 GFLOP of bf16 trees take 167 us (0.41 PFLOP/s); of the 156
// of the main kernel vector instructions issue for 107 on every SIMD and the
// matrix cores are busy for 43, 11 of them at the same time.  16 GFLOP of f32
// pieces of prompts take 78 us (0.2 PFLOP/s, two parts of q and three of the
// weights): 41, 17 and 4 of 66.
#pragma once

#include "attention_shared.h"

namespace q8 {
namespace {

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

// A query row's parts, scaled by a power of two that brings its largest channel to
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

// ---------------------------------------------------------------- the main kernel

__device__ __forceinline__ float load_scale(__amdgpu_buffer_rsrc_t rs, int offset) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, offset, 0, 0));
}

template <RowType T, int DIM, int RT_>
struct Attn {
  typedef typename AttnElem<T>::type E;
  static constexpr int RT = RT_;
  static constexpr int NB = DIM / 32;             // blocks
  static constexpr int QP = AttnElem<T>::kQParts;
  static constexpr int PP = AttnElem<T>::kPParts;
  static constexpr int PACK = 1, NK = 8;          // keys of a tile per lane
  static constexpr int WGS = kAttnWgsPerCu;
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
  __device__ __forceinline__ void cut(int rt, const QueryRow<T, DIM> &from, bool in) {
    undo[rt] = cut_query<T, DIM>(from, in, qf[rt]);
  }
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

  __device__ __forceinline__ void no_top(int rt) { m[rt] = -INFINITY; }
  __device__ __forceinline__ float top(int rt) const { return m[rt]; }
  __device__ __forceinline__ void weights(float (&s)[RT][NK]) { weigh<RT, NK, NB, PACK>(s, undo, m, l, acc); }

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
// 24 sequences of 4096 keys, dim 64, 4 rows of f32: 27.9 us, 28.9 with 16-row
// items; one sequence of 1000 keys, dim 128: 16.7 and 17.5):
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
  static constexpr int WGS = kAttnWgsPerCu;
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

  __device__ __forceinline__ void cut(int rt, const QueryRow<T, DIM> &from, bool in) {
    undo[rt] = cut_query<T, DIM>(from, in, qf[rt]);
  }

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

  __device__ __forceinline__ void no_top(int rt) { m[rt] = -INFINITY; }
  __device__ __forceinline__ float top(int rt) const { return m[rt]; }
  __device__ __forceinline__ void weights(float (&s)[1][NK]) { weigh<1, NK, NB, PACK>(s, undo, m, l, acc); }

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

// ---------------------------------------------------------------- many rows

// The same for items of more rows (trees, prompts; 24 sequences of 4096 keys, 72
// rows of bf16, dim 128: 115 us, 128 with 32-row items): up to 64 * RT rows, 16 * RT
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

template <RowType T, int DIM, int ROWS>
hipError_t launch_instance(const AttnArgs &a, int wgs, hipStream_t stream) {
  typedef typename AttnOf<T, DIM, ROWS>::type A;
  if constexpr (ROWS >= 64)
    hipLaunchKernelGGL((attention_wide_kernel<T, DIM, ROWS / 64>), dim3((unsigned)wgs), dim3(kThreads), 0, stream, a);
  else if (ROWS <= 16 && a.items == nullptr)
    hipLaunchKernelGGL((attention_kernel<A, T, DIM, ROWS, ROWS <= 16 ? 8 : 4>), dim3((unsigned)wgs), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((attention_kernel<A, T, DIM, ROWS, 4>), dim3((unsigned)wgs), dim3(kThreads), 0, stream, a);
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
