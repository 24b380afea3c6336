// Attention over the Q8_0 cache for gfx950: for each row t and query head h
//   out[t, h] = sum_j p_j V_j / sum_j p_j,   p_j = exp(alpha q[t, h] . K_j - m)
// over the tokens j that the row sees, in one pass with a running maximum m
// and running sums.
//
// Arithmetic.  Codes are exact in bf16 (|code| <= 128 has at most 8 bits), and
// the k-slice of v_mfma_f32_16x16x32_bf16 is exactly one 32-channel block, so
//   * scores: q is cut into bf16 parts that add up to it exactly (1 part for
//     bf16, 2 for f16, 3 for f32; cut by truncation, so no part overflows); a
//     block's unscaled partial comes out of the matrix core and is multiplied
//     by the key's scale once, in f32;
//   * output: the value scale depends on the key and the block, so it is
//     multiplied into the weight, p_j s_jb, which is cut into bf16 parts (2:
//     exact to 2^-16, for bf16 and f16 outputs; 3: exact, for f32) against the
//     exact codes.
// Maxima, sums and outputs are f32 throughout; the only rounding beyond f32 is
// the last one to the output's type.
//
// Layout.  The scores are computed transposed, S^T = K Q^T, and so is the
// output, O^T = V^T P^T: lane l then holds, for its row (l % 16), the weights
// of keys 4 (l / 16) + 0..3 of each 16-key tile, which is what the second
// product needs from it when its k index is read as those keys.  Weights never
// leave their lane, a row's maximum is two cross-lane steps, and the cache's
// pair order lets K, V and their scales go from memory to registers with no
// shared memory between.  Scales arrive one per lane and are broadcast within
// the 16-lane group by DPP.
//
// Work.  An item is a sequence's tile of rows for one head of the cache; its
// keys are cut into units of 128 (32 for each wave).  The units of all items
// form one list that is dealt to the workgroups in equal contiguous runs, so
// sequences of all lengths load the device evenly.  A workgroup that has all
// of an item's units writes the rows; otherwise it leaves sums, maxima and
// weights, which a second kernel joins in key order (so results do not depend
// on timing).  Lengths and offsets are read on the device: a captured graph
// follows them.
#pragma once

#include <type_traits>

#include "q8_attention.h"

namespace q8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

template <RowType T>
struct AttnElem;
template <>
struct AttnElem<kRowF32> {
  typedef float type;
  static constexpr int kQParts = 3, kPParts = 3;
};
template <>
struct AttnElem<kRowBf16> {
  typedef __bf16 type;
  static constexpr int kQParts = 1, kPParts = 2;
};
template <>
struct AttnElem<kRowF16> {
  typedef _Float16 type;
  static constexpr int kQParts = 2, kPParts = 2;
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
__device__ __forceinline__ float cut_bf16(float x) { return __uint_as_float(bits(x) & 0xffff0000u); }

// Codes at byte pair `half` of a word, as two bf16.
__device__ __forceinline__ uint32_t pair_bf16(uint32_t w, int half) {
  const float a = (float)(int8_t)(w >> (16 * half));
  const float b = (float)(int8_t)(w >> (16 * half + 8));
  return pack_hi(a, b);
}

// Parts of eight floats as matrix operands.
template <int PARTS>
__device__ __forceinline__ void split8(const float (&x)[8], v4u (&out)[PARTS]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[p][i] = pack_hi(r[2 * i], r[2 * i + 1]);
    if (p + 1 < PARTS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] -= cut_bf16(r[i]);
    }
  }
}

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Lane N of each 16-lane group, to all of them (row_newbcast).
template <int N>
__device__ __forceinline__ float bcast(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + N, 0xf, 0xf, true));
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

// ---------------------------------------------------------------- the work list

// Keys an item's rows may see: all of the sequence's under a tree, those up to
// the item's last token otherwise.
__device__ __forceinline__ int item_keys(const AttnArgs &p, const Seq &q, int r) {
  if (p.tree != nullptr) return q.length;
  return q.length - q.n + min(q.n, (r + 1) * p.tile_tokens);
}
__device__ __forceinline__ int item_units(const AttnArgs &p, const Seq &q, int r) {
  if (q.bad) return 1;
  const int u = (item_keys(p, q, r) + kAttnUnit - 1) / kAttnUnit;
  return u < 1 ? 1 : u;
}
__device__ __forceinline__ int row_items(const AttnArgs &p, const Seq &q) {
  return (q.n + p.tile_tokens - 1) / p.tile_tokens;
}
// Units of a sequence's items for one head (and sub-group of heads).
__device__ __forceinline__ int64_t head_units(const AttnArgs &p, const Seq &q) {
  const int items = row_items(p, q);
  if (items <= 1 || p.tree != nullptr || q.bad) return items == 0 ? 0 : (int64_t)items * item_units(p, q, items - 1);
  int64_t u = 0;
  for (int r = 0; r < items; ++r) u += item_units(p, q, r);
  return u;
}

struct Run0 {  // where a workgroup's run begins
  int b;
  int64_t rest;   // units into sequence b
  int64_t begin, end, total;
  int wgs;        // workgroups with a run
};

// Every workgroup sums the sequences' units and finds its share of them.
__device__ __forceinline__ Run0 find_run(const AttnArgs &p, int wg, int wgs, int tid) {
  __shared__ int64_t sums[kThreads];
  __shared__ int64_t found_rest;
  __shared__ int found_b;
  const int64_t heads = (int64_t)p.c.heads * p.subs;
  const int per = (p.s.seqs + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.s.seqs), b1 = min(b0 + per, p.s.seqs);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += heads * head_units(p, seq_at(p.s, b));
  sums[tid] = mine;
  __syncthreads();
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < kThreads; d <<= 1) {
    const int64_t other = tid >= d ? sums[tid - d] : 0;
    __syncthreads();
    incl += other;
    sums[tid] = incl;
    __syncthreads();
  }
  Run0 r;
  r.total = uniform(sums[kThreads - 1]);
  r.wgs = (int)(r.total < wgs ? r.total : wgs);
  r.begin = r.end = r.rest = 0;
  r.b = 0;
  if (wg < r.wgs) {
    r.begin = r.total * wg / r.wgs;
    r.end = r.total * (wg + 1) / r.wgs;
    int64_t at = incl - mine;
    if (r.begin >= at && r.begin < incl) {
      int b = b0;
      for (; b < b1 - 1; ++b) {
        const int64_t u = heads * head_units(p, seq_at(p.s, b));
        if (r.begin < at + u) break;
        at += u;
      }
      found_b = b;
      found_rest = r.begin - at;
    }
    __syncthreads();
    r.b = __builtin_amdgcn_readfirstlane(found_b);
    r.rest = uniform(found_rest);
  }
  return r;
}

// The workgroup whose run holds unit u.
__device__ __forceinline__ int wg_of(int64_t u, const Run0 &r) {
  return (int)(((u + 1) * r.wgs - 1) / r.total);
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

// VB-byte pieces of codes.
template <int WORDS>
__device__ __forceinline__ void load_words(const int8_t *p, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 1) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (WORDS == 2) {
    const v2u v = *reinterpret_cast<const v2u *>(p);
    w[0] = v[0];
    w[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const v4u v = reinterpret_cast<const v4u *>(p)[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
    }
  }
}

template <RowType T, int DIM, int RT>
struct Attn {
  typedef typename AttnElem<T>::type E;
  static constexpr int NB = DIM / 32;             // blocks
  static constexpr int QP = AttnElem<T>::kQParts;
  static constexpr int PP = AttnElem<T>::kPParts;
  static constexpr int KW = DIM / 16;             // words of a lane's quarter row of K
  static constexpr int VW = DIM / 64;             // words of a lane's pairs of V
  static constexpr int SW = (4 * NB + 15) / 16;   // scale words per lane for 4 keys
  static constexpr int ROWS = 16 * RT;
  static constexpr int PITCH = DIM + 4;           // LDS row of sums; 16 rows then start 4 banks apart

  // Codes and scales of one 32-key tile: 16-key half h in kw[h] / ks[h]; keys
  // 16 h + 4 c + i in vw[4 h + i], vs[h] (c the lane's group).
  uint32_t kw[2][KW];
  float ks[2][SW];
  uint32_t vw[8][VW];
  float vs[2][SW];
  v4u qf[RT][NB][QP];
  v4f acc[RT][NB][2];
  float m[RT], l[RT];

  const AttnArgs *p;
  int lane, row, c;  // row = lane % 16, c = lane / 16

  // The token row, of head kvh, where the 16 keys at `pos` begin.  poison: NaN,
  // to be added to the scales, where the table holds no page of the cache.
  __device__ __forceinline__ int64_t half_base(const int *pages, int pos, int last, int kvh, float &poison) const {
    const int at = min(pos, last);
    int page = uniform_load(pages + (at >> p->c.page_shift));
    const bool ok = (uint32_t)page < p->c.pages;
    page = ok ? page : 0;
    poison = ok ? 0.f : NAN;
    // 16-key halves lie within a page (pages hold 16 tokens or more); one past
    // the last key reads the last key's half instead.
    const int in = at & ((1 << p->c.page_shift) - 1) & ~15;
    return ((((int64_t)page * p->c.heads + kvh) << p->c.page_shift)) + in;
  }

  __device__ __forceinline__ void load_k(const int64_t (&base)[2], const float (&poison)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_words<KW>(p->c.K + base[h] * DIM + row * DIM + c * (DIM / 4), kw[h]);
      const float *s = p->c.KS + (base[h] + 4 * c) * NB;
#pragma unroll
      for (int w = 0; w < SW; ++w) ks[h][w] = s[(16 * w + row) % (4 * NB)] + poison[h];
    }
  }
  __device__ __forceinline__ void load_v(const int64_t (&base)[2], const float (&poison)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words<VW>(p->c.V + (base[h] + 4 * c + i) * DIM + row * (DIM / 16), vw[4 * h + i]);
      const float *s = p->c.VS + (base[h] + 4 * c) * NB;
#pragma unroll
      for (int w = 0; w < SW; ++w) vs[h][w] = s[(16 * w + row) % (4 * NB)] + poison[h];
    }
  }

  // Scores of the tile: s[rt][4 h + i] for key 16 h + 4 c + i and row `row` of row tile rt.
  __device__ __forceinline__ void scores(float (&s)[RT][8]) {
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
          a[jl] = pair_bf16(kw[h][jl * VW + byte / 4], (byte / 2) % 2);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = QP - 1; q >= 0; --q) x = mfma(a, qf[rt][b][q], x);  // small parts first
          static_for<0, 4>([&](auto i_) {
            constexpr int i = decltype(i_)::value;
            constexpr int e = i * NB + b;
            s[rt][4 * h + i] += bcast<e % 16>(ks[h][e / 16]) * x[i];
          });
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Weights of the tile (running maximum, sums), then the second product.
  // sees[rt]: bit k of it for key k of the tile (MASKED only).
  template <bool MASKED>
  __device__ __forceinline__ void softmax(float (&s)[RT][8], const uint32_t (&sees)[RT]) {
    const float scale = p->alpha * 1.4426950408889634f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[rt][k] *= scale;
        if constexpr (MASKED)
          if (!((sees[rt] >> (16 * (k / 4) + 4 * c + k % 4)) & 1)) s[rt][k] = -INFINITY;
      }
      float top = s[rt][0];
#pragma unroll
      for (int k = 1; k < 8; ++k) top = fmaxf(top, s[rt][k]);
      top = across_groups_max(top);
      const float to = fmaxf(m[rt], top);
      const float from = to == -INFINITY ? 0.f : to;  // nothing seen yet: all weights are exp2(-inf) = 0
      const float f = __builtin_amdgcn_exp2f(m[rt] - from);
      m[rt] = to;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s[rt][k] = __builtin_amdgcn_exp2f(s[rt][k] - from);
        sum += s[rt][k];
      }
      l[rt] = l[rt] * f + sum;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[rt][b][i] *= f;
    }
  }

  template <bool MASKED>
  __device__ __forceinline__ void values(const float (&s)[RT][8], const uint32_t (&sees)[RT]) {
    static_for<0, NB>([&](auto b_) {
      constexpr int b = decltype(b_)::value;
      // Lane: codes of keys (k index 4 h + i) at channels 32 b + 2 row + 0, 1.
      v4u a[2];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint32_t w0 = vw[2 * kk][b / 2], w1 = vw[2 * kk + 1][b / 2];
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
          w[k] = bcast<e % 16>(vs[k / 4][e / 16]) * s[rt][k];
          // A key the row does not see may hold anything, a NaN scale too.
          if constexpr (MASKED)
            if (!((sees[rt] >> (16 * (k / 4) + 4 * c + k % 4)) & 1)) w[k] = 0.f;
        });
        v4u parts[PP];
        split8<PP>(w, parts);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = PP - 1; q >= 0; --q) acc[rt][b][i] = mfma(a[i], parts[q], acc[rt][b][i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
};

// Bit k: whether the row at index `i` among its sequence's new tokens (row t
// of q) sees key base + k.
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs &p, int base, int context, int n, int length, int i,
                                              int64_t t) {
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

template <RowType T, int DIM, int RT>
__global__ __launch_bounds__(kThreads, kAttnWgsPerCu) void attention_kernel(AttnArgs p) {
  typedef Attn<T, DIM, RT> A;
  typedef typename A::E E;
  constexpr int NB = A::NB, ROWS = A::ROWS, PITCH = A::PITCH;
  __shared__ __attribute__((aligned(16))) float sums[kWaves][ROWS][PITCH];
  __shared__ float tops[kWaves][ROWS], weights[kWaves][ROWS];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Neighbouring runs, which may share keys or an item, on one XCD.
  const int per_xcd = gridDim.x / kXcds;
  const int wg = gridDim.x % kXcds == 0 ? (int)(blockIdx.x % kXcds) * per_xcd + (int)blockIdx.x / kXcds : (int)blockIdx.x;
  const Run0 run = find_run(p, wg, gridDim.x, tid);
  if (tid == 0) p.items[wg].valid = 0;
  if (wg >= run.wgs) return;

  A a;
  a.p = &p;
  a.lane = tid & 63;
  a.row = a.lane & 15;
  a.c = a.lane >> 4;

  // Where the run begins: sequence b, head vh (with its sub-group), row item r, unit k0.
  int b = run.b;
  Seq seq = uniform_seq_at(p.s, b);
  int vh, r, k0;
  {
    const int64_t per_head = head_units(p, seq);
    vh = (int)(run.rest / per_head);
    int64_t rest = run.rest - vh * per_head;
    if (p.tree != nullptr || seq.bad) {
      const int u = item_units(p, seq, 0);
      r = (int)(rest / u);
      k0 = (int)(rest - (int64_t)r * u);
    } else {
      r = 0;
      while (rest >= item_units(p, seq, r)) rest -= item_units(p, seq, r++);
      k0 = (int)rest;
    }
  }

  for (int64_t unit = run.begin; unit < run.end;) {
    const int units = item_units(p, seq, r);
    const int64_t left = run.end - unit;
    const int k1 = left < units - k0 ? k0 + (int)left : units;
    const int kvh = vh / p.subs, sub = vh - kvh * p.subs;
    const int sub_heads = min(p.sub_heads, p.group - sub * p.sub_heads);
    const int head0 = kvh * p.group + sub * p.sub_heads;
    const int i0 = r * p.tile_tokens;
    const int tokens = min(p.tile_tokens, seq.n - i0);
    const int context = seq.length - seq.n;
    const int rows = tokens * sub_heads;

    int index[RT], head[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int rho = 16 * rt + a.row;
      const int tok = rho / sub_heads;
      index[rt] = i0 + min(tok, tokens - 1);
      head[rt] = head0 + rho - tok * sub_heads;
      // the query's parts; rows past the item's are zeros
      const bool in = rho < rows;
      const E *q = static_cast<const E *>(p.q) + (int64_t)(seq.start + index[rt]) * p.q_stride +
                   (int64_t)(in ? head[rt] : head0) * DIM + 8 * a.c;
#pragma unroll
      for (int bb = 0; bb < NB; ++bb) {
        const Run<E, 8> v = *reinterpret_cast<const Run<E, 8> *>(q + 32 * bb);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = in ? (float)v.x[i] : 0.f;
        split8<A::QP>(x, a.qf[rt][bb]);
      }
      a.m[rt] = -INFINITY;
      a.l[rt] = 0.f;
#pragma unroll
      for (int bb = 0; bb < NB; ++bb) a.acc[rt][bb][0] = a.acc[rt][bb][1] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    if (!seq.bad) {
      const int keys = item_keys(p, seq, r);
      const int last = keys - 1;
      // Keys that every row of the item sees.
      const int all = p.tree != nullptr ? context : context + i0 + 1;
      const int *pages = p.s.table + (int64_t)b * p.s.table_stride;
      const int begin = k0 * kAttnUnit + wave * kAttnTile;
      const int end = min(k1 * kAttnUnit, keys);
      if (begin < end) {
        int64_t base[2];
        float poison[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) base[h] = a.half_base(pages, begin + 16 * h, last, kvh, poison[h]);
        a.load_k(base, poison);
        a.load_v(base, poison);
        // Two loops, not a branch in one: the compiler would move what both
        // sides begin with (128 conversions) above the branch and run out of registers.
        auto step = [&](auto masked_, int at) {
          constexpr bool MASKED = decltype(masked_)::value;
          const int next = at + kAttnUnit;
          const bool more = next < end;
          if (more) {
#pragma unroll
            for (int h = 0; h < 2; ++h) base[h] = a.half_base(pages, next + 16 * h, last, kvh, poison[h]);
          }
          float s[RT][8];
          a.scores(s);
          if (more) a.load_k(base, poison);
          uint32_t sees[RT];
          if constexpr (MASKED) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              sees[rt] = seen_bits(p, at, context, seq.n, seq.length, index[rt], seq.start + index[rt]);
          }
          a.template softmax<MASKED>(s, sees);
          a.template values<MASKED>(s, sees);
          if (more) a.load_v(base, poison);
        };
        int at = begin;
        for (; at < end && at + kAttnTile <= all; at += kAttnUnit) step(std::false_type{}, at);
        for (; at < end; at += kAttnUnit) step(std::true_type{}, at);
      }
    }

    // The four waves' sums, through LDS.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float l = across_groups_sum(a.l[rt]);
      if (a.c == 0) {
        tops[wave][16 * rt + a.row] = a.m[rt];
        weights[wave][16 * rt + a.row] = l;
      }
#pragma unroll
      for (int bb = 0; bb < NB; ++bb) {
        float *to = &sums[wave][16 * rt + a.row][32 * bb + 8 * a.c];
        const v4f x = a.acc[rt][bb][0], y = a.acc[rt][bb][1];  // channels 2 i and 2 i + 1 of the lane's eight
        *reinterpret_cast<v4f *>(to) = v4f{x[0], y[0], x[1], y[1]};
        *reinterpret_cast<v4f *>(to + 4) = v4f{x[2], y[2], x[3], y[3]};
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == units;
    // Slot 1 holds the run's last item, cut short at its end; slot 0 an item
    // that an earlier run began.
    float *slot = p.partial + (2 * (int64_t)wg + (k0 == 0 ? 1 : 0)) * attn_slot_floats(ROWS, DIM);
    for (int e = tid; e < rows * (DIM / 8); e += kThreads) {
      const int rho = e / (DIM / 8), d = 8 * (e % (DIM / 8));
      float top = tops[0][rho];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, tops[w][rho]);
      const float from = top == -INFINITY ? 0.f : top;
      float weight = 0.f, x[8] = {};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(tops[w][rho] - from);
        weight += f * weights[w][rho];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += f * sums[w][rho][d + i];
      }
      if (whole) {
        const int tok = rho / sub_heads;
        const int64_t t = seq.start + i0 + tok;
        float scale = 1.f / weight;
        bool nothing = false;
        if (weight == 0.f) nothing = !sees_any(p.tree, p.tree_words, context, seq.n, t);
        if (seq.bad) {
          scale = NAN;
          nothing = false;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = nothing ? 0.f : seq.bad ? NAN : x[i] * scale;
        store_run<E, 8>(static_cast<E *>(p.out) + t * p.out_stride + (int64_t)(head0 + rho - tok * sub_heads) * DIM + d, x);
      } else {
        v4f *to = reinterpret_cast<v4f *>(slot + (int64_t)rho * DIM + d);
        to[0] = v4f{x[0], x[1], x[2], x[3]};
        to[1] = v4f{x[4], x[5], x[6], x[7]};
        if (d == 0) {
          slot[(int64_t)ROWS * DIM + rho] = top;
          slot[(int64_t)ROWS * (DIM + 1) + rho] = weight;
        }
      }
    }
    if (tid == 0 && k0 == 0 && !whole) {
      AttnItem it;
      it.valid = 1;
      it.last = wg_of(unit + units - 1, run);
      it.row0 = seq.start + i0;
      it.tokens = tokens;
      it.head0 = head0;
      it.heads = sub_heads;
      it.seq_row0 = seq.start;
      it.seq_new = seq.n;
      it.context = context;
      p.items[wg] = it;
    }
    __syncthreads();  // the sums are read before the next item's are written

    unit += k1 - k0;
    if (unit >= run.end) break;
    // The next item.
    k0 = 0;
    if (++r == row_items(p, seq)) {
      r = 0;
      if (++vh == p.c.heads * p.subs) {
        vh = 0;
        do {
          seq = uniform_seq_at(p.s, ++b);
        } while (seq.n == 0);
      }
    }
  }
}

// ---------------------------------------------------------------- joining the parts

// Workgroup (w, y): the split item that workgroup w began, rows 4 y .. 4 y + 3
// (one per wave); parts are taken in key order, several in flight.
template <RowType T, int DIM>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnArgs p, int slot_rows) {
  typedef typename AttnElem<T>::type E;
  const AttnItem it = p.items[blockIdx.x];
  if (!it.valid) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rho = blockIdx.y * kWaves + wave;
  if (rho >= it.tokens * it.heads) return;
  constexpr int PER = DIM / 64;  // channels per lane
  const int64_t size = attn_slot_floats(slot_rows, DIM);
  const int first = blockIdx.x, parts = it.last - first + 1;
  // Contributor k: the first one's slot 1, then slot 0 of the following ones.
  const float *base = p.partial + (2 * (int64_t)first + 1) * size;
  auto part = [&](int k) { return k == 0 ? base : p.partial + 2 * (int64_t)(first + k) * size; };
  // The largest maximum, then every part's factor, a lane per part.
  float top = -INFINITY;
  for (int k = lane; k < parts; k += 64) top = fmaxf(top, part(k)[(int64_t)slot_rows * DIM + rho]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float from = top == -INFINITY ? 0.f : top;
  float weight = 0.f, x[PER] = {};
  for (int k0 = 0; k0 < parts; k0 += 64) {
    float f = 0.f, wt = 0.f;
    if (k0 + lane < parts) {
      const float *s = part(k0 + lane) + (int64_t)slot_rows * DIM + rho;
      f = __builtin_amdgcn_exp2f(s[0] - from);
      wt = f * s[slot_rows];
    }
    const int n = min(64, parts - k0);
    for (int k = 0; k < n; ++k) {
      const float g = __shfl(f, k);
      weight += __shfl(wt, k);
      const float *s = part(k0 + k) + (int64_t)rho * DIM + lane * PER;
#pragma unroll
      for (int i = 0; i < PER; ++i) x[i] += g * s[i];
    }
  }
  const int tok = rho / it.heads;
  const int64_t t = it.row0 + tok;
  bool nothing = false;
  if (weight == 0.f) nothing = !sees_any(p.tree, p.tree_words, it.context, it.seq_new, t);
  const float scale = 1.f / weight;
#pragma unroll
  for (int i = 0; i < PER; ++i) x[i] = nothing ? 0.f : x[i] * scale;
  store_run<E, PER>(static_cast<E *>(p.out) + t * p.out_stride + (int64_t)(it.head0 + rho - tok * it.heads) * DIM + lane * PER, x);
}

template <RowType T, int DIM, int RT>
hipError_t launch_instance(const AttnArgs &a, int wgs, hipStream_t stream) {
  hipLaunchKernelGGL((attention_kernel<T, DIM, RT>), dim3((unsigned)wgs), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attention_join_kernel<T, DIM>), dim3((unsigned)wgs, 16 * RT / kWaves), dim3(kThreads), 0, stream,
                     a, 16 * RT);
  return hipGetLastError();
}

template <RowType T>
hipError_t launch_attention(const AttnArgs &a, int row_tiles, int wgs, hipStream_t stream) {
  if (row_tiles == 1) {
    if (a.c.dim == 64) return launch_instance<T, 64, 1>(a, wgs, stream);
    if (a.c.dim == 128) return launch_instance<T, 128, 1>(a, wgs, stream);
    if (a.c.dim == 256) return launch_instance<T, 256, 1>(a, wgs, stream);
  } else if (row_tiles == 2) {
    if (a.c.dim == 64) return launch_instance<T, 64, 2>(a, wgs, stream);
    if (a.c.dim == 128) return launch_instance<T, 128, 2>(a, wgs, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace q8
