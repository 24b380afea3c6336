// Attention over the cache in 4-bit floats for gfx950, on the work list, masks
// and running softmax of the attentions over caches.
//
// Arithmetic.  A code times its power-of-two scale is exact in bf16, so the matrix
// cores take keys and values themselves, from one conversion per pair of codes:
// a score is one chain of products over all channels, with no block to rescale,
// and the weights enter the second product as they are.
//   * scores: q is cut into bf16 parts (1 for bf16 rows, 2 for f16, 3 for f32: all
//     of it);
//   * output: weights are cut into bf16 parts (2 for bf16 and f16 rows: 2^-16 of
//     the weight; 3 for f32: all of it).
// Maxima, sums, weights and outputs are f32 throughout.
//
// Layout.  As over the Q8_0 cache, S^T = K Q^T and O^T = V^T P^T, so that weights
// never leave their lane.  K's operand wants pairs 4 c .. 4 c + 3 of a block of key
// l % 16 in lane l = 16 c + l % 16: neighbouring bytes of its row, all blocks of them one
// run of dim / 8 bytes.  V's wants channels 2 (l % 16) + 0, 1 of a block of keys 4 c ..
// 4 c + 3: in V's own order, where four tokens share 2 dim bytes, one run of dim / 8
// bytes again.  V's conversions take a key's pair of channels, since its two keys
// would have two scales, and a permutation sorts the pairs by channel.
#pragma once

#include "attention_shared.h"
#include "mx4_cache.h"

namespace q8 {
namespace {

template <RowType T>
constexpr int kMx4QParts = T == kRowF32 ? 3 : T == kRowF16 ? 2 : 1;

// The pair of byte BYTE of `codes` as bf16, times 2^(byte SCALE of `scales` - 127);
// of the scale only the exponent counts, and 255 gives NaN.
template <int BYTE, int SCALE>
__device__ __forceinline__ uint32_t pair_bf16(uint32_t codes, uint32_t scales) {
  const uint32_t e = SCALE < 3 ? scales << (23 - 8 * SCALE) : scales >> 1;
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, __uint_as_float(e), BYTE));
}
// Bit 7 of every byte of x that stands for no number (253 .. 255; 253 and 254 are no scales).
__device__ __forceinline__ uint32_t no_numbers(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x03030303u) & x & 0x80808080u; }

// split8 by vector instructions alone: v_dot2_f32_bf16, of which it takes one per
// part and weight, runs on the matrix pipe, in the way of the products.
template <int PARTS>
__device__ __forceinline__ void cut8(const float (&x)[8], v4u (&out)[PARTS]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    const bool rest = PARTS < 3 && p + 1 == PARTS;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[p][i] = rest ? pack_near(r[2 * i], r[2 * i + 1]) : pack_hi(r[2 * i], r[2 * i + 1]);
    if (p + 1 < PARTS)
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] -= __uint_as_float(bits(r[i]) & 0xffff0000u);
  }
}

template <int BYTES>
__device__ __forceinline__ void load_bytes(__amdgpu_buffer_rsrc_t rs, int offset, uint32_t (&w)[(BYTES + 3) / 4]) {
  if constexpr (BYTES == 2)
    w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, offset, 0, 0);
  else
    load_words<BYTES / 4>(rs, offset, w);
}

// A query row's bf16 parts; sign: of alpha, 0 for alpha = 0.  A row that is not
// `in` is zeros.
template <RowType T, int DIM>
__device__ __forceinline__ void cut_bf16(const QueryRow<T, DIM> &from, bool in, float sign,
                                         v4u (&qf)[DIM / 32][kMx4QParts<T>]) {
#pragma unroll
  for (int b = 0; b < DIM / 32; ++b) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = in ? (float)from.x[b].x[i] * sign : 0.f;
    if constexpr (kMx4QParts<T> == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[b][0][i] = pack_hi(x[2 * i], x[2 * i + 1]);
    } else {
      cut8<kMx4QParts<T>>(x, qf[b]);
    }
  }
}

// A row's kept maximum, as its scores meet it: what they are taken against, 0 before any
// is seen, and from where on a score raises it: everything does before any is seen.
struct Top {
  float from, limit;
  __device__ __forceinline__ void none() {
    from = 0.f;
    limit = -INFINITY;
  }
  __device__ __forceinline__ float value() const { return limit == -INFINITY ? -INFINITY : from; }
};

// Scores, up to the factor undo, to the exponents of their weights, against the row's
// kept maximum, which is raised first where one passes it by kMaxSlack (as in settle).
// scale_sums(rt, f) scales what grows with the weights.  A score is rounded once, against
// the new maximum: against the one before, a row whose first keys score far below the
// others would lose what those differ by.
// undo is no power of two, so a maximum is rounded where a score is not, and its own weight
// is 2^r with r up to half a step of the maximum.  That cancels, but where the step is large
// 2^r passes f32.  For maxima from kCoarse on (r up to a half) every step's scores pass the
// limit, and are rounded as the maximum is.
constexpr float kCoarse = 1 << 24, kLeast = -3.4028234663852886e38f;
// Scores times undo must keep the order of their sizes, and masked ones -inf; the sign is
// the query's.
__device__ __forceinline__ float undo_of(float scale) { return scale == 0.f ? 1.f : fabsf(scale); }
template <int NRT, int NK, typename F>
__device__ __forceinline__ void exponents(float (&s)[NRT][NK], float undo, Top *m, F scale_sums) {
  float top[NRT], factor = undo;
  bool above = false;
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt) {
    top[rt] = s[rt][0];
#pragma unroll
    for (int k = 1; k < NK; ++k) top[rt] = fmaxf(top[rt], s[rt][k]);
    above |= top[rt] * undo > m[rt].limit;
  }
  if (__ballot(above) != 0) {
    bool coarse = false;
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      const float before = m[rt].value(), to = fmaxf(before, row_max<1>(top[rt]) * undo);
      const bool far = finite(to) && fabsf(to) >= kCoarse;
      m[rt].from = base_of(to);
      m[rt].limit = far ? kLeast : to + kMaxSlack;
      scale_sums(rt, __builtin_amdgcn_exp2f(before - m[rt].from));
      coarse |= far;
    }
    if (__ballot(coarse) != 0) {
      factor = 1.f;
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          s[rt][k] *= undo;
          pin(s[rt][k]);  // a branch, no selection among both in every step
        }
    }
  }
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
    for (int k = 0; k < NK; ++k) s[rt][k] = fmaf(s[rt][k], factor, -m[rt].from);
}

// Cache policy of loads that are not to stay in the caches (nt).
constexpr int kPastCaches = 2;

// PAST: codes are read past the caches: they leave the Infinity Cache anyway where
// they are larger than it (596 MB of bf16 rows' keys: 117 us, 122 through the caches; 150 MB,
// read again and again: 41 and 39).
template <RowType T, int DIM, int RT_, bool PAST>
struct Mx4Attn {
  typedef typename AttnElem<T>::type E;
  static constexpr int RT = RT_;
  static constexpr int NB = DIM / 32;             // blocks, and bytes of a lane's pairs and of a key's scales
  static constexpr int QP = kMx4QParts<T>;
  static constexpr int PP = AttnElem<T>::kPParts;
  static constexpr int PACK = 1, NK = 8;          // keys of a tile per lane
  static constexpr int WGS = RT == 1 ? mx4_direct_wgs(T, DIM) : kAttnWgsPerCu;
  static constexpr int KS = (NB + 3) / 4;         // words of a key's scales
  static constexpr int ROWS = 16 * RT;
  static constexpr int PITCH = DIM + 4;           // LDS row of sums; 16 rows then start 4 banks apart

  // Codes and scales of one 32-key tile: of 16-key half h the pairs 4 c .. of key
  // `row` and its scales, and the pair `row` of keys 4 c .. 4 c + 3 and theirs.
  struct Tile {
    uint32_t kw[2][NB], ks[2][KS];
    uint32_t vw[2][NB], vs[2][NB];
    uint32_t lost[2];  // all ones where there is no such page
  };
  v4u qf[RT][NB][QP];
  v4f acc[RT][NB][2];
  Top m[RT];
  float l[RT];

  const AttnArgs *p;
  float scale;       // alpha log2 e
  int row, c;        // lane % 16 and lane / 16

  __device__ __forceinline__ int row_of(int rt) const { return 16 * rt + row; }  // of the item
  __device__ __forceinline__ bool holds_row() const { return true; }             // in its sums
  __device__ __forceinline__ void cut(int rt, const QueryRow<T, DIM> &from, bool in) {
    cut_bf16<T, DIM>(from, in, scale == 0.f ? 0.f : scale < 0.f ? -1.f : 1.f, qf[rt]);
  }
  __device__ __forceinline__ void start() {}

  // live: 0 for a tile that does not exist (nothing is read), 1 otherwise.
  __device__ __forceinline__ void load_k(Tile &t, const int64_t (&base)[2], const float (&poison)[2], int live) {
    const uint8_t *K = reinterpret_cast<const uint8_t *>(p->c.K), *S = reinterpret_cast<const uint8_t *>(p->c.KS);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t.lost[h] = poison[h] == 0.f ? 0u : ~0u;
      load_words<NB, PAST ? kPastCaches : 0>(buffer_of(K + base[h] * (DIM / 2), 8 * DIM * live), row * (DIM / 2) + c * (4 * NB), t.kw[h]);
      load_bytes<NB>(buffer_of(S + base[h] * NB, 16 * NB * live), row * NB, t.ks[h]);
    }
  }
  __device__ __forceinline__ void load_v(Tile &t, const int64_t (&base)[2], int live) {
    const uint8_t *V = reinterpret_cast<const uint8_t *>(p->c.V), *S = reinterpret_cast<const uint8_t *>(p->c.VS);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_words<NB, PAST ? kPastCaches : 0>(buffer_of(V + base[h] * (DIM / 2), 8 * DIM * live), c * (2 * DIM) + row * (4 * NB), t.vw[h]);
      load_words<NB>(buffer_of(S + base[h] * NB, 16 * NB * live), c * (4 * NB), t.vs[h]);
    }
  }

  // Marks the value scales of a missing page.
  __device__ __forceinline__ void add_poison(Tile &t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < NB; ++w) t.vs[h][w] |= t.lost[h];
  }

  // Scores of the tile: s[rt][4 h + i] for key 16 h + 4 c + i and row `row` of row tile rt.
  __device__ __forceinline__ void scores(Tile &t, float (&s)[RT][8]) {
    v4f x[RT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int w = 0; w < KS; ++w) t.ks[h][w] |= t.lost[h];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) x[rt][h] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      static_for<0, 2>([&](auto h_) {
        constexpr int h = decltype(h_)::value;
        v4u a;
        static_for<0, 4>([&](auto j_) {
          constexpr int j = decltype(j_)::value, e = j * NB + b;
          a[j] = pair_bf16<e % 4, b % 4>(t.kw[h][e / 4], t.ks[h][b / 4]);
        });
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int q = QP - 1; q >= 0; --q) x[rt][h] = mfma(a, qf[rt][b][q], x[rt][h]);  // small parts first
      });
    });
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[rt][k] = x[rt][k / 4][k % 4];
  }

  // sees[rt]: bit k for key k of the tile.  Keys a row does not see get the
  // score of no weight.  Their value scales may be anything: one that is no
  // number is taken out, and the rows that do see it are remembered in
  // lost[rt], bit b for block b.  Returns whether there is any such scale.
  __device__ __forceinline__ bool mask(Tile &t, float (&s)[RT][8], const uint32_t (&sees)[RT], uint32_t (&lost)[RT]) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (!((sees[rt] >> (16 * (k / 4) + 4 * c + k % 4)) & 1)) s[rt][k] = -INFINITY;
    uint32_t bad = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < NB; ++w) bad |= no_numbers(t.vs[h][w]);
    if (__ballot(bad != 0) == 0) return false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) lost[rt] = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int w = 0; w < NB; ++w) {
        const uint32_t gone = no_numbers(t.vs[h][w]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int i = (4 * w + y) / NB, b = (4 * w + y) % NB;  // key 4 c + i of the half, block b
          if (gone >> (8 * y + 7) & 1) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) lost[rt] |= ((sees[rt] >> (16 * h + 4 * c + i)) & 1) << b;
            t.vs[h][w] &= ~(0xffu << (8 * y));
          }
        }
      }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      lost[rt] |= __shfl_xor(lost[rt], 16);
      lost[rt] |= __shfl_xor(lost[rt], 32);
    }
    return true;
  }

  __device__ __forceinline__ void no_top(int rt) { m[rt].none(); }
  __device__ __forceinline__ float top(int rt) const { return m[rt].value(); }
  __device__ __forceinline__ void weights(float (&s)[RT][8]) {
    exponents<RT, 8>(s, undo_of(scale), m, [&](int rt, float f) {
      l[rt] *= f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[rt][b][i] *= f;
    });
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[rt][k] = __builtin_amdgcn_exp2f(s[rt][k]);
        sum += s[rt][k];
      }
      l[rt] += sum;
    }
  }

  __device__ __forceinline__ void values(const Tile &t, const float (&s)[RT][8]) {
    v4u parts[RT][PP];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) cut8<PP>(s[rt], parts[rt]);
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      // Lane: values of keys (k index 4 h + i) at channels 32 b + 2 row + 0, 1.
      v4u a[2];
      static_for<0, 4>([&](auto k_) {
        constexpr int k = decltype(k_)::value, h = k / 2, e = 2 * (k % 2) * NB + b, f = e + NB;
        const uint32_t u = pair_bf16<e % 4, e % 4>(t.vw[h][e / 4], t.vs[h][e / 4]);
        const uint32_t v = pair_bf16<f % 4, f % 4>(t.vw[h][f / 4], t.vs[h][f / 4]);
        a[0][k] = __builtin_amdgcn_perm(v, u, 0x05040100u);
        a[1][k] = __builtin_amdgcn_perm(v, u, 0x07060302u);
      });
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int q = PP - 1; q >= 0; --q) acc[rt][b][i] = mfma(a[i], parts[rt][q], acc[rt][b][i]);
          pin(acc[rt][b][i]);
        }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
};

// ---------------------------------------------------------------- many rows

// The same for items of more rows (trees, prompts), up to 64 * RT: all four waves
// take the same keys.  Bound by the issue of vector instructions.  Per step of 64 keys each wave loads 16 keys' codes, converts
// them and lays them into LDS as the matrix operands that all waves read (16 bytes
// per lane, conflict-free); the next step's codes are in flight meanwhile.  Row
// tiles are dealt to the waves in turn, so a short item still uses all four.
constexpr int kMx4WideKeys = 64;
// Operands that are on their way from LDS ahead of the product that takes them.
constexpr int kAhead = 2;

// The order of what lies before it back to the last one: products with VALU vector
// instructions behind each.
template <int PRODUCTS, int VALU>
__device__ __forceinline__ void mix() {
  static_for<0, PRODUCTS>([](auto) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
  });
  __builtin_amdgcn_sched_barrier(0);
}

template <int DIM>
struct Mx4WideLds {
  static constexpr int NB = DIM / 32;
  static constexpr int BUFS = DIM == 256 ? 1 : 2;  // two workgroups must fit a CU
  v4u k[BUFS][4][NB][64];        // 16-key tile, block, lane
  v2u v[BUFS][2][NB][2][64][2];  // 32-key group, block, channel of the pair, lane, half
  // Value scales that are no numbers are taken as the least one; `gone` says
  // whether a 16-key tile has any, and `vs` then holds its scales, of keys 4 c ..
  uint32_t gone[BUFS][4];
  uint32_t vs[BUFS][4][4][NB];
};

template <RowType T, int DIM, int RT>
__global__ __launch_bounds__(kThreads, kAttnWgsPerCu) void mx4_wide_kernel(AttnArgs p) {
  typedef typename AttnElem<T>::type E;
  constexpr int NB = DIM / 32, QP = kMx4QParts<T>, PP = AttnElem<T>::kPParts;
  constexpr int KS = (NB + 3) / 4;
  constexpr int ROWS = 64 * RT, BUFS = Mx4WideLds<DIM>::BUFS;
  __shared__ Mx4WideLds<DIM> lds;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, row = lane & 15, c = lane >> 4;
  const uint8_t *Kc = reinterpret_cast<const uint8_t *>(p.c.K), *Ks = reinterpret_cast<const uint8_t *>(p.c.KS);
  const uint8_t *Vc = reinterpret_cast<const uint8_t *>(p.c.V), *Vs = reinterpret_cast<const uint8_t *>(p.c.VS);
  const float scale = p.alpha * 1.4426950408889634f;
  const float undo = undo_of(scale);

  // This wave's 16 keys of a step, on their way to LDS.
  uint32_t kw[NB], ksw[KS], vw[NB], vsw[NB];
  float poison = 0.f;
  auto load = [&](int64_t base) {
    load_words<NB>(buffer_of(Kc + base * (DIM / 2), 8 * DIM), row * (DIM / 2) + c * (4 * NB), kw);
    load_bytes<NB>(buffer_of(Ks + base * NB, 16 * NB), row * NB, ksw);
    load_words<NB>(buffer_of(Vc + base * (DIM / 2), 8 * DIM), c * (2 * DIM) + row * (4 * NB), vw);
    load_words<NB>(buffer_of(Vs + base * NB, 16 * NB), c * (4 * NB), vsw);
  };
  // Into LDS: scales that are no numbers first, then, for each block, its keys and
  // its values.
  auto lay_scales = [&](int buf) {
    const uint32_t lost = poison == 0.f ? 0u : ~0u;
    uint32_t bad = 0;
#pragma unroll
    for (int w = 0; w < KS; ++w) ksw[w] |= lost;
#pragma unroll
    for (int w = 0; w < NB; ++w) {
      vsw[w] |= lost;
      bad |= no_numbers(vsw[w]);
    }
    const bool any = __ballot(bad != 0) != 0;
    if (any) {
#pragma unroll
      for (int w = 0; w < NB; ++w) {
        if (row == 0) lds.vs[buf][wave][c][w] = vsw[w];
        vsw[w] &= ~((no_numbers(vsw[w]) >> 7) * 0xffu);
      }
    }
    if (lane == 0) lds.gone[buf][wave] = any;
  };
  auto lay_keys = [&](auto b_, int buf) {
    constexpr int b = decltype(b_)::value;
    v4u x;
    static_for<0, 4>([&](auto j_) {
      constexpr int j = decltype(j_)::value, e = j * NB + b;
      x[j] = pair_bf16<e % 4, b % 4>(kw[e / 4], ksw[b / 4]);
    });
    lds.k[buf][wave][b][lane] = x;
  };
  auto lay_values = [&](auto b_, int buf) {
    constexpr int b = decltype(b_)::value;
    uint32_t u[4];
    static_for<0, 4>([&](auto k_) {
      constexpr int e = decltype(k_)::value * NB + b;
      u[decltype(k_)::value] = pair_bf16<e % 4, e % 4>(vw[e / 4], vsw[e / 4]);
    });
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t sel = i ? 0x07060302u : 0x05040100u;
      lds.v[buf][wave / 2][b][i][lane][wave % 2] =
          v2u{__builtin_amdgcn_perm(u[1], u[0], sel), __builtin_amdgcn_perm(u[3], u[2], sel)};
    }
  };
  auto lay = [&](int buf) {
    lay_scales(buf);
    static_for<0, NB>([&](auto b_) {
      lay_keys(b_, buf);
      lay_values(b_, buf);
    });
  };

  walk_shares<DIM>(p, ROWS, tid, [&](const Share &h) {
    // The first step's codes are asked for before the query's rows are needed.
    const int last = h.keys - 1;
    const int begin = h.k0 << h.shift;
    const int end = h.seq.bad ? begin : min(h.k1 << h.shift, h.keys);
    // A page's number is read one step before the page.
    Keys16 ahead;
    auto load_at = [&](int at) {
      load(token_row(p, ahead, h.kvh, poison));
      ahead = keys_at(p, h.pages, at + kMx4WideKeys + 16 * wave, last);
    };
    // Row tile rt of this wave: rows 16 (4 rt + wave) .. of the item.
    v4u qf[RT][NB][QP];
    v4f acc[RT][2 * NB];
    Top m[RT];
  float l[RT];
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
    if (begin < end) {
      ahead = keys_at(p, h.pages, begin + 16 * wave, last);
      load_at(begin);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      cut_bf16<T, DIM>(q[rt], in[rt], scale == 0.f ? 0.f : scale < 0.f ? -1.f : 1.f, qf[rt]);
      m[rt].none();
      l[rt] = 0.f;
#pragma unroll
      for (int n = 0; n < 2 * NB; ++n) acc[rt][n] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    const int tiles = (h.rows + 15) / 16;
    const int mine = tiles <= wave ? 0 : (tiles - wave + 3) / 4;  // row tiles this wave has

    // One step over the 64 keys from `at` on, for the wave's first NRT row tiles.  With two
    // buffers the next step's codes (more: there is one) are converted meanwhile, in the
    // shadow of the products.
    auto compute = [&](auto nrt_, int at, int buf, bool more) {
      constexpr int NRT = decltype(nrt_)::value;
      float s[NRT][16];
      if (BUFS == 2 && more) lay_scales(buf ^ 1);
      {
        v4f x[NRT][4];
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) x[rt][kt] = v4f{0.f, 0.f, 0.f, 0.f};
        v4u a[kAhead + 1];
        auto fetch = [&](auto n_) {
          constexpr int n = decltype(n_)::value;
          if constexpr (n < 4 * NB) a[n % (kAhead + 1)] = lds.k[buf][n % 4][n / 4][lane];
        };
        // Products first: what another wave of the SIMD does meanwhile fits between them
        // (256 rows of bf16 a sequence over 8 x 8192 keys 124 us, 129 without).
        __builtin_amdgcn_s_setprio(1);
        static_for<0, kAhead>(fetch);
        auto products = [&](auto lays_) {
          static_for<0, 4 * NB>([&](auto n_) {
            constexpr int n = decltype(n_)::value, kt = n % 4, b = n / 4;
            fetch(std::integral_constant<int, n + kAhead>{});
            if constexpr (decltype(lays_)::value && n % 4 == 1) lay_keys(std::integral_constant<int, b>{}, buf ^ 1);
            if constexpr (decltype(lays_)::value && n % 4 == 3) lay_values(std::integral_constant<int, b>{}, buf ^ 1);
#pragma unroll
            for (int q = QP - 1; q >= 0; --q)
#pragma unroll
              for (int rt = 0; rt < NRT; ++rt) x[rt][kt] = mfma(a[n % (kAhead + 1)], qf[rt][b][q], x[rt][kt]);
            mix<QP * NRT, 6>();
          });
        };
        if (BUFS == 2 && more)
          products(std::true_type{});
        else
          products(std::false_type{});
        __builtin_amdgcn_s_setprio(0);
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
          for (int k = 0; k < 16; ++k) s[rt][k] = x[rt][k / 4][k % 4];
      }

      uint64_t sees[NRT];  // shifted: bit 16 kt + i is this lane's key i of tile kt
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) sees[rt] = ~0ull;
      if (at + kMx4WideKeys > h.all) {
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
      exponents<NRT, 16>(s, undo, m, [&](int rt, float f) {
        l[rt] *= f;
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n) acc[rt][n] *= f;
      });
      {
        constexpr int RING = kAhead + 1;
        v4u a[RING][2];
        auto fetch = [&](auto n_) {
          constexpr int n = decltype(n_)::value, g = n / NB, b = n % NB;
          if constexpr (n < 2 * NB)
#pragma unroll
            for (int i = 0; i < 2; ++i) a[n % RING][i] = *reinterpret_cast<const v4u *>(&lds.v[buf][g][b][i][lane][0]);
        };
        auto weight = [&](int rt, int k) {
          s[rt][k] = __builtin_amdgcn_exp2f(s[rt][k]);
          l[rt] += s[rt][k];
        };
        // Sums are made here: later, the weights would have to be kept for them.
        auto summed = [&]() {
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt) pin(l[rt]);
        };
        v4u parts[NRT][PP];
        auto cut = [&](int g) {
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt) {
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = s[rt][8 * g + k];
            cut8<PP>(w, parts[rt]);
          }
        };
        static_for<0, kAhead>(fetch);
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
          for (int k = 0; k < 8; ++k) weight(rt, k);
        summed();
        cut(0);
        __builtin_amdgcn_s_setprio(1);
        __builtin_amdgcn_sched_barrier(0);
        static_for<0, 2 * NB>([&](auto n_) {
          constexpr int n = decltype(n_)::value, g = n / NB, b = n % NB;
          fetch(std::integral_constant<int, n + kAhead>{});
          // The second half's weights in the shadow of the first one's products.
          if constexpr (g == 0)
#pragma unroll
            for (int e = b * NRT * 8 / NB; e < (b + 1) * NRT * 8 / NB; ++e) weight(e / 8, 8 + e % 8);
#pragma unroll
          for (int q = PP - 1; q >= 0; --q)
#pragma unroll
            for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
              for (int i = 0; i < 2; ++i) acc[rt][2 * b + i] = mfma(a[n % RING][i], parts[rt][q], acc[rt][2 * b + i]);
          mix<2 * PP * NRT, 2>();
          if constexpr (n == NB - 1) {
            summed();
            cut(1);
            __builtin_amdgcn_sched_barrier(0);
          }
        });
        __builtin_amdgcn_s_setprio(0);
      }
      // Blocks of rows that see a value scale that is no number are lost.
      uint32_t any = 0;
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) any |= lds.gone[buf][kt];
      if (__builtin_amdgcn_readfirstlane(any) != 0) {
        uint32_t lost[NRT] = {};
#pragma unroll 1
        for (int kt = 0; kt < 4; ++kt) {
          if (lds.gone[buf][kt] == 0) continue;
#pragma unroll 1
          for (int e = 0; e < 4 * NB; ++e)  // key 4 c + e / NB, block e % NB
            if (no_numbers(lds.vs[buf][kt][c][e / 4]) >> (8 * (e % 4) + 7) & 1)
#pragma unroll
              for (int rt = 0; rt < NRT; ++rt) lost[rt] |= (uint32_t)(sees[rt] >> (16 * kt + e / NB) & 1) << (e % NB);
        }
#pragma unroll
        for (int rt = 0; rt < NRT; ++rt) {
          lost[rt] |= __shfl_xor(lost[rt], 16);
          lost[rt] |= __shfl_xor(lost[rt], 32);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            if (lost[rt] >> b & 1) acc[rt][2 * b] = acc[rt][2 * b + 1] = v4f{NAN, NAN, NAN, NAN};
        }
      }
    };

    if (begin < end) {
      lay(0);
      if (begin + kMx4WideKeys < end) load_at(begin + kMx4WideKeys);
      __syncthreads();
      auto steps = [&](auto nrt_) {
        for (int at = begin; at < end; at += kMx4WideKeys) {
          const int buf = BUFS == 2 ? (at - begin) / kMx4WideKeys % 2 : 0;
          const bool more = at + kMx4WideKeys < end;
          if constexpr (decltype(nrt_)::value > 0) compute(nrt_, at, buf, more);
          if constexpr (BUFS == 1) __syncthreads();
          if (more) {
            if constexpr (BUFS == 1 || decltype(nrt_)::value == 0) lay(BUFS == 2 ? buf ^ 1 : 0);
            if (at + 2 * kMx4WideKeys < end) load_at(at + 2 * kMx4WideKeys);
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
        const v4f u = acc[rt][2 * b], v = acc[rt][2 * b + 1];
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
        h.slot[(int64_t)ROWS * DIM + rho] = m[rt].value();
        h.slot[(int64_t)ROWS * (DIM + 1) + rho] = weight;
      }
    }
  });
}

// ---------------------------------------------------------------- very many rows

// The same for items of up to 256 rows, by eight waves of 32 that share the keys' codes.
// Matrix and vector instructions of two waves overlap on a SIMD only where one wave is
// at the first while the other is at the second; left to themselves, the two waves of a
// SIMD do the same at the same time.  So the waves work in two groups of four, one on each
// SIMD, half a step apart: between two barriers one group multiplies (the values of
// its last 64 keys, the scores of the next) while the other makes its scores weights and
// converts codes, keys in the first group, values in the second.
//   slot 2 t:      first group PV(t - 1), S(t)       second group weights(t - 1), V(t) to LDS
//   slot 2 t + 1:  first group weights(t), K(t + 1)  second group PV(t - 1), S(t)
// Two buffers of each are enough: K(t + 1) replaces K(t - 1), last read in slot 2 t - 1, V(t)
// replaces V(t - 2), last read there too.
// Trees of 64 drafts over 8 x 8192 keys (32 heads, 8 of keys, of 128): bf16 103 us, 124 by the
// kernel above; f16 116, 133.  A slot takes some 3100 cycles, 1660 of matrix instructions
// (bf16): the wave that makes weights issues an instruction in five cycles, and loses about
// six to each product of the SIMD's other wave.  Products of 32 x 32 x 16, half as many, made
// dim 64 5 % faster and dim 128 4 % slower.
template <int DIM>
struct Mx4DeepLds {
  static constexpr int NB = DIM / 32;
  v4u k[2][4][NB][64];        // 16-key tile, block, lane
  v2u v[2][2][NB][2][64][2];  // 32-key group, block, channel of the pair, lane, half
  uint32_t gone[2][4];        // as in the kernel above
  uint32_t vs[2][4][4][NB];
};

template <RowType T, int DIM>
__global__ __launch_bounds__(2 * kThreads, 1) void mx4_deep_kernel(AttnArgs p) {
  typedef typename AttnElem<T>::type E;
  constexpr int NB = DIM / 32, QP = kMx4QParts<T>, PP = AttnElem<T>::kPParts;
  constexpr int KS = (NB + 3) / 4;
  constexpr int ROWS = kMx4DeepRows, RT = ROWS / 128, RING = kAhead + 1;
  __shared__ Mx4DeepLds<DIM> lds;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = wave >> 2, quarter = wave & 3;  // of the keys of a step
  const int lane = tid & 63, row = lane & 15, c = lane >> 4;
  const float scale = p.alpha * 1.4426950408889634f;
  const float undo = undo_of(scale);
  const v4u ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};

  // 16 keys of a step, on their way to LDS: keys in the first group, values in the second.
  const uint8_t *codes = reinterpret_cast<const uint8_t *>(group == 0 ? p.c.K : p.c.V);
  const uint8_t *scales = reinterpret_cast<const uint8_t *>(group == 0 ? p.c.KS : p.c.VS);
  uint32_t cw[NB], sw[NB];
  float poison = 0.f;
  auto load = [&](int64_t base) {
    const __amdgpu_buffer_rsrc_t cs = buffer_of(codes + base * (DIM / 2), 8 * DIM), ss = buffer_of(scales + base * NB, 16 * NB);
    if (group == 0) {
      load_words<NB>(cs, row * (DIM / 2) + c * (4 * NB), cw);
      uint32_t s[KS];
      load_bytes<NB>(ss, row * NB, s);
#pragma unroll
      for (int w = 0; w < KS; ++w) sw[w] = s[w];
    } else {
      load_words<NB>(cs, c * (2 * DIM) + row * (4 * NB), cw);
      load_words<NB>(ss, c * (4 * NB), sw);
    }
  };
  auto lay_keys = [&](int buf) {
    const uint32_t lost = poison == 0.f ? 0u : ~0u;
#pragma unroll
    for (int w = 0; w < KS; ++w) sw[w] |= lost;
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      v4u x;
      static_for<0, 4>([&](auto j_) {
        constexpr int j = decltype(j_)::value, e = j * NB + b;
        x[j] = pair_bf16<e % 4, b % 4>(cw[e / 4], sw[b / 4]);
      });
      lds.k[buf][quarter][b][lane] = x;
    });
  };
  auto lay_values = [&](int buf) {
    const uint32_t lost = poison == 0.f ? 0u : ~0u;
    uint32_t bad = 0;
#pragma unroll
    for (int w = 0; w < NB; ++w) {
      sw[w] |= lost;
      bad |= no_numbers(sw[w]);
    }
    const bool any = __ballot(bad != 0) != 0;
    if (any) {
#pragma unroll
      for (int w = 0; w < NB; ++w) {
        if (row == 0) lds.vs[buf][quarter][c][w] = sw[w];
        sw[w] &= ~((no_numbers(sw[w]) >> 7) * 0xffu);
      }
    }
    if (lane == 0) lds.gone[buf][quarter] = any;
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      uint32_t u[4];
      static_for<0, 4>([&](auto k_) {
        constexpr int e = decltype(k_)::value * NB + b;
        u[decltype(k_)::value] = pair_bf16<e % 4, e % 4>(cw[e / 4], sw[e / 4]);
      });
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t sel = i ? 0x07060302u : 0x05040100u;
        lds.v[buf][quarter / 2][b][i][lane][quarter % 2] =
            v2u{__builtin_amdgcn_perm(u[1], u[0], sel), __builtin_amdgcn_perm(u[3], u[2], sel)};
      }
    });
  };

  walk_shares<DIM>(p, ROWS, tid, [&](const Share &h) {
    const int last = h.keys - 1;
    const int begin = h.k0 << h.shift;
    const int end = h.seq.bad ? begin : min(h.k1 << h.shift, h.keys);
    const int steps = (end - begin + kMx4WideKeys - 1) / kMx4WideKeys;
    // A page's number is read one step before the page.
    auto find_step = [&](int t) { return keys_at(p, h.pages, begin + t * kMx4WideKeys + 16 * quarter, last); };
    Keys16 ahead;
    int64_t place;
    float place_poison;
    auto place_step = [&](int t) {
      place = token_row(p, ahead, h.kvh, place_poison);
      ahead = find_step(t + 1);
    };
    auto load_placed = [&]() {
      load(place);
      poison = place_poison;
    };
    if (steps > 0) {
      ahead = find_step(0);
      place_step(0);
      load_placed();
      place_step(1);
    }
    // Row tile rt of this wave: rows 16 (8 rt + wave) .. of the item.
    v4u qf[RT][NB][QP];
    // Sums over a row tile: of block b's channels at 2 b, 2 b + 1, of the weights at 2 NB.
    v4f acc[RT][2 * NB + 1];
    Top m[RT];
    {
      QueryRow<T, DIM> q[RT];
      bool in[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int rho = 16 * (8 * rt + wave) + row;
        const int tok = rho / h.sub_heads;
        in[rt] = rho < h.rows;
        fetch_query<T, DIM>(p, h.seq.start + h.i0 + min(tok, h.tokens - 1), in[rt] ? h.head0 + rho - tok * h.sub_heads : h.head0, c, q[rt]);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        cut_bf16<T, DIM>(q[rt], in[rt], scale == 0.f ? 0.f : scale < 0.f ? -1.f : 1.f, qf[rt]);
        m[rt].none();
#pragma unroll
        for (int n = 0; n <= 2 * NB; ++n) acc[rt][n] = v4f{0.f, 0.f, 0.f, 0.f};
      }
    }
    const int tiles = (h.rows + 15) / 16;
    const int mine = tiles <= wave ? 0 : (tiles - wave + 7) / 8;  // row tiles this wave has

    // What the row of tile rt sees of the 64 keys at `at`, shifted: bit 16 kt + i is this lane's key i of tile kt.
    auto seen = [&](int rt, int at) -> uint64_t {
      if (at + kMx4WideKeys <= h.all) return ~0ull;
      const int i = h.i0 + min((16 * (8 * rt + wave) + row) / h.sub_heads, h.tokens - 1);
      const int64_t t = h.seq.start + i;
      uint64_t x = seen_bits(p, at, h.context, h.seq.length, i, t);
      if (at + 32 < h.seq.length) x |= (uint64_t)seen_bits(p, at + 32, h.context, h.seq.length, i, t) << 32;
      return x >> 4 * c;
    };

    auto work = [&](auto nrt_) {
      constexpr int NRT = decltype(nrt_)::value;
      float s[NRT > 0 ? NRT : 1][16];
      v4u parts[NRT > 0 ? NRT : 1][2][PP];
      v4u va[RING][2];
      auto fetch_v = [&](auto n_, int buf) {
        constexpr int n = decltype(n_)::value, g = n / NB, b = n % NB;
        if constexpr (n < 2 * NB)
#pragma unroll
          for (int i = 0; i < 2; ++i) va[n % RING][i] = *reinterpret_cast<const v4u *>(&lds.v[buf][g][b][i][lane][0]);
      };
      v4u ka[RING];
      auto fetch_k = [&](auto n_, int buf) {
        constexpr int n = decltype(n_)::value;
        if constexpr (n < 4 * NB) ka[n % RING] = lds.k[buf][n % 4][n / 4][lane];
      };
      // The values of step t, its first operands on their way; then those of the next
      // step's scores are (more: there is one).
      auto values = [&](int t, auto more_) {
        if constexpr (NRT == 0) {
          if constexpr (decltype(more_)::value) place_step(t + 3);
        } else {
          const int buf = t & 1;
          __builtin_amdgcn_s_setprio(1);
          static_for<0, 2 * NB>([&](auto n_) {
            constexpr int n = decltype(n_)::value, g = n / NB, b = n % NB;
            fetch_v(std::integral_constant<int, n + kAhead>{}, buf);
            if constexpr (decltype(more_)::value && n + 1 == 2 * NB)
              static_for<0, kAhead>([&](auto i_) { fetch_k(i_, buf ^ 1); });
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = PP - 1; q >= 0; --q)
#pragma unroll
              for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[rt][2 * b + i] = mfma(va[n % RING][i], parts[rt][g][q], acc[rt][2 * b + i]);
            if constexpr (b == 0)  // the weights' sums: times ones
#pragma unroll
              for (int q = PP - 1; q >= 0; --q)
#pragma unroll
                for (int rt = 0; rt < NRT; ++rt) acc[rt][2 * NB] = mfma(ones, parts[rt][g][q], acc[rt][2 * NB]);
            __builtin_amdgcn_sched_barrier(0);
            // Where the codes after the next ones lie: scalar work, in the products' shadow.
            if constexpr (decltype(more_)::value && n == 0) place_step(t + 3);
          });
          // Blocks of rows that see a value scale that is no number are lost.
          uint32_t any = 0;
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) any |= lds.gone[buf][kt];
          if (__builtin_amdgcn_readfirstlane(any) != 0) {
#pragma unroll
            for (int rt = 0; rt < NRT; ++rt) {
              const uint64_t sees = seen(rt, begin + t * kMx4WideKeys);
              uint32_t lost = 0;
#pragma unroll 1
              for (int kt = 0; kt < 4; ++kt) {
                if (lds.gone[buf][kt] == 0) continue;
#pragma unroll 1
                for (int e = 0; e < 4 * NB; ++e)  // key 4 c + e / NB, block e % NB
                  if (no_numbers(lds.vs[buf][kt][c][e / 4]) >> (8 * (e % 4) + 7) & 1)
                    lost |= (uint32_t)(sees >> (16 * kt + e / NB) & 1) << (e % NB);
              }
              lost |= __shfl_xor(lost, 16);
              lost |= __shfl_xor(lost, 32);
#pragma unroll
              for (int b = 0; b < NB; ++b)
                if (lost >> b & 1) acc[rt][2 * b] = acc[rt][2 * b + 1] = v4f{NAN, NAN, NAN, NAN};
            }
          }
          __builtin_amdgcn_s_setprio(0);
        }
      };
      auto scores = [&](int t) {
        if constexpr (NRT > 0) {
          v4f x[NRT][4];
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) x[rt][kt] = v4f{0.f, 0.f, 0.f, 0.f};
          __builtin_amdgcn_s_setprio(1);
          static_for<0, 4 * NB>([&](auto n_) {
            constexpr int n = decltype(n_)::value, kt = n % 4, b = n / 4;
            fetch_k(std::integral_constant<int, n + kAhead>{}, t & 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = QP - 1; q >= 0; --q)
#pragma unroll
              for (int rt = 0; rt < NRT; ++rt) x[rt][kt] = mfma(ka[n % RING], qf[rt][b][q], x[rt][kt]);
            __builtin_amdgcn_sched_barrier(0);
          });
          __builtin_amdgcn_s_setprio(0);
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
            for (int k = 0; k < 16; ++k) s[rt][k] = x[rt][k / 4][k % 4];
        }
      };
      // The scores of step t to weights and their parts.
      auto weights = [&](int t) {
        if constexpr (NRT > 0) {
          const int at = begin + t * kMx4WideKeys;
          if (at + kMx4WideKeys > h.all) {
#pragma unroll
            for (int rt = 0; rt < NRT; ++rt) {
              const uint64_t sees = seen(rt, at);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (!((sees >> (16 * (k / 4) + k % 4)) & 1)) s[rt][k] = -INFINITY;
            }
          }
          exponents<NRT, 16>(s, undo, m, [&](int rt, float f) {
#pragma unroll
            for (int n = 0; n <= 2 * NB; ++n) acc[rt][n] *= f;
          });
#pragma unroll
          for (int rt = 0; rt < NRT; ++rt) {
#pragma unroll
            for (int k = 0; k < 16; ++k) s[rt][k] = __builtin_amdgcn_exp2f(s[rt][k]);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = s[rt][8 * g + k];
              cut8<PP>(w, parts[rt][g]);
#pragma unroll
              for (int q = 0; q < PP; ++q) pin(parts[rt][g][q]);
            }
          }
        }
      };
      auto ready = [&](int t) {  // for values(t)
        if constexpr (NRT > 0) static_for<0, kAhead>([&](auto n_) { fetch_v(n_, t & 1); });
      };
      auto first_scores = [&]() {
        if constexpr (NRT > 0) static_for<0, kAhead>([&](auto n_) { fetch_k(n_, 0); });
        place_step(2);
        scores(0);
      };
      auto keys_on = [&](int t) {  // those of step t, and the next ones asked for
        if (t < steps) {
          lay_keys(t & 1);
          if (t + 1 < steps) load_placed();
        }
      };
      auto values_on = [&](int t) {
        if (t < steps) {
          lay_values(t & 1);
          if (t + 1 < steps) load_placed();
        }
      };

      // Both groups pass the same barriers.
      if (group == 0) {
        keys_on(0);
        __syncthreads();
        first_scores();
        __syncthreads();
        weights(0);
        keys_on(1);
        ready(0);
        __syncthreads();
        for (int t = 1; t < steps; ++t) {
          values(t - 1, std::true_type{});
          scores(t);
          __syncthreads();
          weights(t);
          keys_on(t + 1);
          ready(t);
          __syncthreads();
        }
        values(steps - 1, std::false_type{});
        __syncthreads();
        __syncthreads();
      } else {
        __syncthreads();
        values_on(0);
        __syncthreads();
        first_scores();
        __syncthreads();
        for (int t = 1; t < steps; ++t) {
          weights(t - 1);
          values_on(t);
          ready(t - 1);
          __syncthreads();
          values(t - 1, std::true_type{});
          scores(t);
          __syncthreads();
        }
        weights(steps - 1);
        ready(steps - 1);
        __syncthreads();
        values(steps - 1, std::false_type{});
        __syncthreads();
      }
    };
    if (steps > 0) {
      if (mine == 2)
        work(std::integral_constant<int, 2>{});
      else if (mine == 1)
        work(std::integral_constant<int, 1>{});
      else
        work(std::integral_constant<int, 0>{});
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rho = 16 * (8 * rt + wave) + row;
      const float weight = acc[rt][2 * NB][0];
      if (rho >= h.rows) continue;
      const int tok = rho / h.sub_heads;
      const int64_t t = h.seq.start + h.i0 + tok;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const v4f u = acc[rt][2 * b], v = acc[rt][2 * b + 1];
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
        h.slot[(int64_t)ROWS * DIM + rho] = m[rt].value();
        h.slot[(int64_t)ROWS * (DIM + 1) + rho] = weight;
      }
    }
  });
}

template <class A, RowType T, int DIM, int ROWS, int WAVES = kWaves>
void launch_direct(const AttnArgs &a, int wgs, hipStream_t stream) {
  hipLaunchKernelGGL((attention_kernel<A, T, DIM, ROWS, WAVES>), dim3((unsigned)wgs), dim3(64 * WAVES), 0, stream, a);
}

// Workgroups of eight waves where each takes all keys of its items (tables of up to 1024 tokens)
// and there are few of them: 1 and 8 sequences of 1023 keys take 11.2 and 11.5 us, 11.8 and
// 12.0 with four waves; but 32 of them 21.4 and 16.3, 128 of 200 keys 25.1 and 15.7 (bf16, 8 heads
// of keys of 128).  At dim 256 they spill or are no faster.
constexpr int kFewWorkgroups = 128;
template <RowType T, int DIM, int ROWS>
hipError_t launch_instance(const AttnArgs &a, int wgs, hipStream_t stream) {
  if constexpr (ROWS == kMx4DeepRows)
    hipLaunchKernelGGL((mx4_deep_kernel<T, DIM>), dim3((unsigned)wgs), dim3(2 * kThreads), 0, stream, a);
  else if constexpr (ROWS >= 64)
    hipLaunchKernelGGL((mx4_wide_kernel<T, DIM, ROWS / 64>), dim3((unsigned)wgs), dim3(kThreads), 0, stream, a);
  else if constexpr (ROWS > 16)
    launch_direct<Mx4Attn<T, DIM, ROWS / 16, false>, T, DIM, ROWS>(a, wgs, stream);
  else if (DIM <= 128 && a.items == nullptr && wgs <= kFewWorkgroups)
    launch_direct<Mx4Attn<T, DIM, 1, false>, T, DIM, ROWS, DIM <= 128 ? 2 * kWaves : kWaves>(a, wgs, stream);
  else if (a.past_caches)
    launch_direct<Mx4Attn<T, DIM, 1, true>, T, DIM, ROWS>(a, wgs, stream);
  else
    launch_direct<Mx4Attn<T, DIM, 1, false>, T, DIM, ROWS>(a, wgs, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.items == nullptr) return e;  // without items none is split
  hipLaunchKernelGGL((attention_join_kernel<T, DIM>), dim3((ROWS + kWaves * join_rows(DIM) - 1) / (kWaves * join_rows(DIM)), (unsigned)wgs),
                     dim3(kThreads), 0, stream, a, ROWS);
  return hipGetLastError();
}

template <RowType T, int DIM>
hipError_t launch_rows(const AttnArgs &a, int rows, int wgs, hipStream_t stream) {
  if (rows == 16) return launch_instance<T, DIM, 16>(a, wgs, stream);
  if constexpr (DIM <= 128)
    if (rows == 32) return launch_instance<T, DIM, 32>(a, wgs, stream);
  if constexpr (mx4_deep(T, DIM)) {
    if (rows == 128) return launch_instance<T, DIM, 128>(a, wgs, stream);
    if (rows == kMx4DeepRows) return launch_instance<T, DIM, kMx4DeepRows>(a, wgs, stream);
  } else {
    if (rows == 64) return launch_instance<T, DIM, 64>(a, wgs, stream);
  }
  return hipErrorInvalidValue;
}

// rows: of an item (mx4_tile).
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
