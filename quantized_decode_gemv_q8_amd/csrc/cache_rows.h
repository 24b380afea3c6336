// What the kernels that move rows into and out of the caches share: the rows'
// elements, and where a row's token lives.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "q8_cache.h"

namespace q8 {
namespace {

template <RowType T>
struct Elem;
template <>
struct Elem<kRowF32> {
  typedef float type;
  static __device__ __forceinline__ float to_float(float x) { return x; }
  static __device__ __forceinline__ float from_float(float x) { return x; }
};
template <>
struct Elem<kRowBf16> {
  typedef __bf16 type;
  static __device__ __forceinline__ float to_float(__bf16 x) { return (float)x; }
  static __device__ __forceinline__ __bf16 from_float(float x) { return (__bf16)x; }
};
template <>
struct Elem<kRowF16> {
  typedef _Float16 type;
  static __device__ __forceinline__ float to_float(_Float16 x) { return (float)x; }
  static __device__ __forceinline__ _Float16 from_float(float x) { return (_Float16)x; }
};

// Two neighbouring elements, aligned as one: a row may start at any element.
template <typename E>
struct __attribute__((packed, aligned(sizeof(E)))) Pair {
  E x, y;
};

// Largest of a 16-lane group.  For |x| as bits: infinities above all numbers,
// NaN above them.
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xf, 0xf, true));  // row_ror:8, 4, 2, 1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xf, 0xf, true));
  return m;
}

// Where row t of the row tensors lives: found by the whole wave (t is the same
// in all lanes).  64 sequences are looked at per step, so up to 64 sequences
// take one round of loads, and 4096 take two.  A sequence whose offsets do not
// ascend within the rows has none, and may lead the steps astray: a row that
// they do not find (one of no sequence, too) is looked for among all sequences.
// A step of 256 sequences and as many rows of none is no slower for it (5.3 us),
// one of 4096 takes 28 us instead of 12.
struct Place {
  bool found;
  Seq seq;
  int index;  // among the sequence's new tokens
  int b;
};

__device__ __forceinline__ Place find_row(const Seqs &s, int t, int lane) {
  int lo = 0, n = s.seqs;
  while (n > 64) {
    const int step = (n + 63) / 64;
    const int at = lo + lane * step;
    const bool below = lane * step < n && s.offsets[at] <= t;
    int k = __popcll(__ballot(below)) - 1;
    if (k < 0) k = 0;  // rows before the first sequence
    lo += k * step;
    n = min(step, n - k * step);
  }
  const bool in = lane < n;
  const int b = lo + (in ? lane : 0);
  int start = s.offsets[b], end = s.offsets[b + 1], length = s.lengths[b];
  uint64_t hit = __ballot(in && start >= 0 && start <= t && t < end && end <= s.rows);
  if (hit == 0 && s.seqs > 64) {
    constexpr int kAhead = 8;  // of 64 sequences in flight
    for (int at = 0; at < s.seqs && hit == 0; at += 64 * kAhead) {
      int first[kAhead], past[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = min(at + 64 * u + lane, s.seqs - 1);  // the last one again, behind it
        first[u] = s.offsets[i];
        past[u] = s.offsets[i + 1];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const uint64_t some = __ballot(first[u] >= 0 && first[u] <= t && t < past[u] && past[u] <= s.rows);
        if (hit == 0 && some != 0) {
          hit = some;
          lo = at + 64 * u;
          start = first[u];
          end = past[u];
        }
      }
    }
    if (hit != 0) length = s.lengths[min(lo + lane, s.seqs - 1)];
  }
  Place p;
  p.found = hit != 0;
  const int from = p.found ? __builtin_ctzll(hit) : 0;
  p.b = __builtin_amdgcn_readfirstlane(lo + from);
  p.seq = seq_of(s, __builtin_amdgcn_readlane(start, from), __builtin_amdgcn_readlane(end, from),
                 __builtin_amdgcn_readlane(length, from));
  p.found = p.found && p.seq.n > 0;
  p.index = t - p.seq.start;
  return p;
}

// First element, among the page's token rows of head 0, of position `pos` of
// sequence b; -1 where the table holds no page of the cache.
__device__ __forceinline__ int64_t token_row(const Cache &c, const Seqs &s, int b, int pos) {
  const int page = s.table[(int64_t)b * s.table_stride + (pos >> c.page_shift)];
  if ((uint32_t)page >= c.pages) return -1;
  return (((int64_t)page * c.heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// Workgroups of one launch: a grid holds less than 2^32 threads in a direction.
constexpr int kMostGroups = 1 << 22;

}  // namespace
}  // namespace q8
