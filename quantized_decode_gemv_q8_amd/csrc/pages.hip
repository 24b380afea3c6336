// A pool of pages: forking, growing, freeing and compacting the page tables of
// sequences, and copying pages.
//
// refs[p] counts the table rows that own page p; a page is free where it is not
// above zero.  Everything is decided by order, never by timing: pages are given
// to the sequences in their order, the lowest free ones first, and compacting
// keeps the order of what it moves.
//
// resize and compact go through phases that each need all of the one before:
// counts of tiles of pages, their prefixes, what follows from them.  A large pool
// takes one launch each over the device, a small one is done by one workgroup.
#include <algorithm>

#include "pages.h"

namespace q8 {
namespace {

constexpr int kBig = 1024;  // threads of a workgroup of resize and compact
constexpr int kBigWaves = kBig / 64;

__device__ __forceinline__ bool is_page(int p, int pages) { return (uint32_t)p < (uint32_t)pages; }

// Pages of `tokens` tokens, for 0 <= tokens < 2^30.
__device__ __forceinline__ int pages_of(int tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

__device__ __forceinline__ bool fits(int tokens, const PageTable &t) { return tokens >= 0 && tokens <= t.max_tokens; }

template <typename X>
__device__ __forceinline__ X wave_sum_before(X x, int lane) {  // exclusive
  X upto = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const X other = __shfl_up(upto, d);
    if (lane >= d) upto += other;
  }
  return upto - x;
}

// Exclusive sum over the workgroup's threads, and the sum of all.
template <typename X>
__device__ __forceinline__ X block_sum_before(X x, X *all) {
  __shared__ X sums[kBigWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const X before = wave_sum_before(x, lane);
  if (lane == 63) sums[wave] = before + x;
  __syncthreads();
  X base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kBigWaves; ++w) {
    const X s = sums[w];
    if (w < wave) base += s;
    total += s;
  }
  __syncthreads();  // before `sums` is written again
  *all = total;
  return base + before;
}

// Sum of x[0 .. n - 1], by the whole workgroup.
template <typename X>
__device__ __forceinline__ int64_t block_total(const X *x, int64_t n) {
  int64_t mine = 0, all;
  for (int64_t i = threadIdx.x; i < n; i += kBig) mine += x[i];
  block_sum_before(mine, &all);
  return all;
}

// The counts of a thread's four neighbouring pages in tile t.  Bit k of `in` is set where
// the pool has page first + k, of used() where an owner has it.
struct Quad {
  int64_t first;
  int in, refs[4];
  __device__ __forceinline__ int used() const {
    int bits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) bits |= (refs[k] > 0) << k;
    return bits & in;
  }
};
__device__ __forceinline__ Quad load_quad(const int *refs, int pages, int64_t t) {
  Quad q;
  q.first = t * kPagesTile + 4 * (int64_t)threadIdx.x;
  if (q.first + 4 <= pages) {
    typedef int Four __attribute__((ext_vector_type(4), aligned(4)));
    const Four x = *reinterpret_cast<const Four *>(refs + q.first);
    q.in = 15;
#pragma unroll
    for (int k = 0; k < 4; ++k) q.refs[k] = x[k];
  } else {
    q.in = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool is = q.first + k < pages;
      q.refs[k] = is ? refs[q.first + k] : 0;
      q.in |= is << k;
    }
  }
  return q;
}

// A workgroup's share of `tiles` tiles.
struct Tiles {
  int64_t begin, end;
};
__device__ __forceinline__ Tiles share(int64_t tiles) {
  const int64_t per = (tiles + gridDim.x - 1) / gridDim.x;
  const int64_t begin = min(per * blockIdx.x, tiles);
  return Tiles{begin, min(begin + per, tiles)};
}

// ---------------------------------------------------------------- fork

// One wave per child.
__global__ __launch_bounds__(kThreads) void fork_kernel(ForkArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * kWaves;
  for (int64_t i = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6); i < a.to.seqs; i += waves) {
    const int parent = a.parent[i];
    int length = 0;
    if ((uint32_t)parent < (uint32_t)a.from.seqs) length = a.lengths[parent];
    if (!fits(length, a.from) || !fits(length, a.to)) length = 0;
    const int held = pages_of(length, a.page_shift);
    int *to = a.to.table + i * a.to.stride;
    const int *from = a.from.table + (int64_t)(held > 0 ? parent : 0) * a.from.stride;
    constexpr int kAtOnce = 4;
    for (int c0 = lane; c0 < a.to.max_pages; c0 += 64 * kAtOnce) {
      int page[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) page[k] = c0 + 64 * k < held ? from[c0 + 64 * k] : -1;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int c = c0 + 64 * k;
        if (is_page(page[k], a.pages))
          atomicAdd(a.refs + page[k], 1);
        else
          page[k] = -1;
        if (c < a.to.max_pages) to[c] = page[k];
      }
    }
    if (lane == 0) a.lengths_out[i] = length;
  }
}

// ---------------------------------------------------------------- resize

struct Change {
  int held, want;  // pages before and after
  bool ok;         // neither is outside of the table
  bool writes;     // into the last page that it holds
};
__device__ __forceinline__ Change change_of(const ResizeArgs &a, int64_t b) {
  const int before = a.before[b], after = a.after[b];
  Change c;
  c.ok = fits(before, a.t) && fits(after, a.t);
  c.held = c.ok ? pages_of(before, a.page_shift) : 0;
  c.want = c.ok ? pages_of(after, a.page_shift) : 0;
  c.writes = c.ok && after > before && (before & ((1 << a.page_shift) - 1)) != 0;
  return c;
}

// Phase 0: pages past what is wanted are released.  A lane takes its sequence's first
// ones, its wave the rest of one sequence after another (1000 sequences that take or
// give back one page each: 5.3 us, 20 with all by waves).
constexpr int kOwn = 4;
__device__ void resize_release(const ResizeArgs &a) {
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * kBigWaves;
  // A wave looks at up to 64 sequences at a time.
  const int64_t each = min((a.t.seqs + waves - 1) / waves, (int64_t)64);
  for (int64_t b0 = ((int64_t)blockIdx.x * kBigWaves + (threadIdx.x >> 6)) * each; b0 < a.t.seqs; b0 += waves * each) {
    Change c{};
    if (lane < each && b0 + lane < a.t.seqs) c = change_of(a, b0 + lane);
    int *own = a.t.table + (c.want < c.held ? b0 + lane : 0) * a.t.stride;
    int page[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) page[i] = c.want + i < c.held ? own[c.want + i] : -1;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (c.want + i < c.held) {
        if (is_page(page[i], a.pages)) atomicAdd(a.refs + page[i], -1);
        own[c.want + i] = -1;
      }
    uint64_t more = __ballot(c.want + kOwn < c.held);
    while (more != 0) {
      const int s = __builtin_ctzll(more);
      more &= more - 1;
      const int held = __shfl(c.held, s), want = __shfl(c.want, s) + kOwn;
      int *row = a.t.table + (b0 + s) * a.t.stride;
      for (int i = want + lane; i < held; i += 64) {
        const int page = row[i];
        if (is_page(page, a.pages)) atomicAdd(a.refs + page, -1);
        row[i] = -1;
      }
    }
  }
}

constexpr int64_t kReplaced = (int64_t)1 << 62;

// Phase 1: free pages of each tile; what each sequence wants, and that of the
// sequences before it in its tile.
__device__ void resize_count(const ResizeArgs &a) {
  const Tiles tiles = share(pages_tiles(a.pages));
  for (int64_t t = tiles.begin; t < tiles.end; ++t) {
    const Quad q = load_quad(a.refs, a.pages, t);
    int all;
    block_sum_before((int)__popc(q.in & ~q.used()), &all);
    if (threadIdx.x == 0) a.w.counts[t] = all;
  }
  const Tiles seqs = share(seqs_tiles(a.t.seqs));
  for (int64_t t = seqs.begin; t < seqs.end; ++t) {
    const int64_t b = t * kSeqsTile + threadIdx.x;
    int64_t need = 0, all;
    bool replaced = false;
    if (b < a.t.seqs) {
      const Change c = change_of(a, b);
      if (c.writes) {
        const int last = a.t.table[b * a.t.stride + c.held - 1];
        replaced = is_page(last, a.pages) && a.refs[last] > 1;
      }
      need = max(c.want - c.held, 0) + (replaced ? 1 : 0);
    }
    const int64_t before = block_sum_before(need, &all);
    if (b < a.t.seqs) a.w.start[b] = before | (replaced ? kReplaced : 0);
    if (threadIdx.x == 0) a.w.totals[t] = all;
  }
}

// Phase 2: the lowest free pages in order, as many as are wanted.
__device__ void resize_list(const ResizeArgs &a) {
  const Tiles tiles = share(pages_tiles(a.pages));
  if (tiles.begin >= tiles.end) return;
  const int64_t wanted = block_total(a.w.totals, seqs_tiles(a.t.seqs));
  int64_t rank = block_total(a.w.counts, tiles.begin);
  for (int64_t t = tiles.begin; t < tiles.end && rank < wanted; ++t) {
    const Quad q = load_quad(a.refs, a.pages, t);
    int all, free = q.in & ~q.used();
    int64_t r = rank + block_sum_before((int)__popc(free), &all);
    for (; free != 0; free &= free - 1, ++r)
      if (r < wanted) a.w.list[r] = (int)(q.first + __builtin_ctz(free));
    rank += all;
  }
}

// Phase 3: a thread gives a sequence its first pages, its wave the rest.
__device__ void resize_give(const ResizeArgs &a) {
  const Tiles seqs = share(seqs_tiles(a.t.seqs));
  if (seqs.begin >= seqs.end) return;
  const int lane = threadIdx.x & 63;
  const int64_t free = block_total(a.w.counts, pages_tiles(a.pages));
  int64_t base = block_total(a.w.totals, seqs.begin);
  for (int64_t t = seqs.begin; t < seqs.end; ++t) {
    const int64_t b = t * kSeqsTile + threadIdx.x;
    const bool in = b < a.t.seqs;
    Change c{};
    int64_t start = 0;
    bool replaced = false;
    if (in) {
      c = change_of(a, b);
      start = a.w.start[b];
      replaced = (start & kReplaced) != 0;
      start = base + (start & ~kReplaced);
    }
    int first = c.held - (replaced ? 1 : 0);  // column of the first page given
    const int need = max(c.want - c.held, 0) + (replaced ? 1 : 0);
    const bool served = start + need <= free;
    int given = served ? need : 0;
    int *row = a.t.table + (in ? b : 0) * a.t.stride;
    if (in) {
      int old = -1, fresh = -1;
      if (replaced && served) {
        old = row[first];
        fresh = a.w.list[start];
        atomicAdd(a.refs + old, -1);
      }
      a.moves[2 * b] = old;
      a.moves[2 * b + 1] = fresh;
      a.missing[b] = !c.ok ? -1 : served ? 0 : need;
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (i < given) {
        const int page = a.w.list[start + i];
        row[first + i] = page;
        a.refs[page] = 1;
      }
    uint64_t more = __ballot(given > kOwn);
    while (more != 0) {
      const int s = __builtin_ctzll(more);
      more &= more - 1;
      const int n = __shfl(given, s), column = __shfl(first, s);
      const int64_t from = __shfl(start, s);
      int *to = a.t.table + (b - lane + s) * a.t.stride;
      for (int i = kOwn + lane; i < n; i += 64) {
        const int page = a.w.list[from + i];
        to[column + i] = page;
        a.refs[page] = 1;
      }
    }
    base += a.w.totals[t];
  }
}

template <int PHASE>
__global__ __launch_bounds__(kBig) void resize_kernel(ResizeArgs a) {
  if constexpr (PHASE == 0) resize_release(a);
  if constexpr (PHASE == 1) resize_count(a);
  if constexpr (PHASE == 2) resize_list(a);
  if constexpr (PHASE == 3) resize_give(a);
}

// The same by one workgroup, a thread for each of up to 1024 sequences: what the phases
// keep in memory stays in registers, the free pages are looked at only as far as
// they are wanted, and a call that wants none (most decode steps) looks at none.
constexpr int kSmallSeqs = kBig;
template <bool RELEASE>
__global__ __launch_bounds__(kBig) void resize_small_kernel(ResizeArgs a) {
  constexpr int kListed = 4096;
  __shared__ int listed[kListed];  // the first ones; the others go through memory
  const int b = threadIdx.x, lane = b & 63;
  const bool in = b < a.t.seqs;
  Change c{};
  if (in) c = change_of(a, b);
  int *row = a.t.table + (in ? b : 0) * a.t.stride;
  int last = -1;
  if (c.writes) last = row[c.held - 1];
  if constexpr (RELEASE) {
    if (__syncthreads_or(c.want < c.held)) {
      resize_release(a);
      __syncthreads();
    }
  }
  const bool replaced = is_page(last, a.pages) && a.refs[last] > 1;
  const int need = max(c.want - c.held, 0) + (replaced ? 1 : 0);
  int64_t wanted;
  const int64_t start = block_sum_before((int64_t)need, &wanted);
  int64_t found = 0;
  Quad q;
  if (wanted > 0) q = load_quad(a.refs, a.pages, 0);
  for (int64_t t = 0; t < pages_tiles(a.pages) && found < wanted; ++t) {
    const Quad next = load_quad(a.refs, a.pages, t + 1);
    int all, free = q.in & ~q.used();
    int64_t r = found + block_sum_before((int)__popc(free), &all);
    for (; free != 0; free &= free - 1, ++r) {
      const int page = (int)(q.first + __builtin_ctz(free));
      if (r < kListed)
        listed[r] = page;
      else if (r < wanted)
        a.w.list[r] = page;
    }
    found += all;
    q = next;
  }
  __syncthreads();
  const bool served = start + need <= found;
  const int given = served ? need : 0, column = c.held - (replaced ? 1 : 0);
  auto page_of = [&](int64_t r) { return r < kListed ? listed[r] : a.w.list[r]; };
  if (in) {
    const bool moves = replaced && served;
    if (moves) atomicAdd(a.refs + last, -1);
    a.moves[2 * b] = moves ? last : -1;
    a.moves[2 * b + 1] = moves ? page_of(start) : -1;
    a.missing[b] = !c.ok ? -1 : served ? 0 : need;
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    if (i < given) {
      const int page = page_of(start + i);
      row[column + i] = page;
      a.refs[page] = 1;
    }
  uint64_t more = __ballot(given > kOwn);
  while (more != 0) {
    const int s = __builtin_ctzll(more);
    more &= more - 1;
    const int n = __shfl(given, s), at = __shfl(column, s);
    const int64_t from = __shfl(start, s);
    int *to = a.t.table + (b - lane + s) * a.t.stride;
    for (int i = kOwn + lane; i < n; i += 64) {
      const int page = page_of(from + i);
      to[at + i] = page;
      a.refs[page] = 1;
    }
  }
}

// ---------------------------------------------------------------- compact

// Phase 0: used pages of each tile.
__device__ void compact_count(const CompactArgs &a) {
  const Tiles tiles = share(pages_tiles(a.pages));
  for (int64_t t = tiles.begin; t < tiles.end; ++t) {
    int all;
    block_sum_before((int)__popc(load_quad(a.refs, a.pages, t).used()), &all);
    if (threadIdx.x == 0) a.w.counts[t] = all;
  }
}

// Phase 1: with U used pages, the r-th used page from U on goes to the r-th free
// page below U.  Both sides of the moves, and every page's rank r among its kind.
__device__ void compact_rank(const CompactArgs &a) {
  const int64_t all_tiles = pages_tiles(a.pages);
  const Tiles tiles = share(all_tiles);
  // All used pages, and those before this workgroup's tiles.
  int64_t U, before;
  {
    int64_t sum = 0, some = 0;
    for (int64_t i = threadIdx.x; i < all_tiles; i += kBig) {
      const int n = a.w.counts[i];
      sum += n;
      if (i < tiles.begin) some += n;
    }
    block_sum_before(sum, &U);
    block_sum_before(some, &before);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.used = (int)U;
  // Used pages below U: those that the ranks from U on do not count.
  int64_t below;
  {
    const int64_t tu = U / kPagesTile;  // the tile that U lies in, or the one past the last
    int64_t some = 0;
    for (int64_t i = threadIdx.x; i < tu; i += kBig) some += a.w.counts[i];
    if (tu < all_tiles) {
      const Quad q = load_quad(a.refs, a.pages, tu);
      int used = q.used();
      for (int k = 0; k < 4; ++k)
        if (q.first + k >= U) used &= ~(1 << k);
      some += __popc(used);
    }
    block_sum_before(some, &below);
  }
  for (int64_t t = tiles.begin; t < tiles.end; ++t) {
    const Quad q = load_quad(a.refs, a.pages, t);
    const int used = q.used();
    int all;
    int64_t u = before + block_sum_before((int)__popc(used), &all);  // used pages before this thread's
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!(q.in >> k & 1)) continue;
      const int64_t p = q.first + k;
      const bool is = used >> k & 1;
      if (is && p >= U) {
        const int64_t r = u - below;
        a.moves[2 * r] = (int)p;
        a.w.list[p] = (int)r;
      } else if (!is && p < U) {
        const int64_t r = p - u;
        a.moves[2 * r + 1] = (int)p;
        a.w.list[p] = (int)r;
      }
      u += is;
    }
    before += all;
  }
  // Places that no move takes.
  const int64_t moved = U - below;
  for (int64_t i = (int64_t)blockIdx.x * kBig + threadIdx.x; i < a.pages / 2; i += (int64_t)gridDim.x * kBig)
    if (i >= moved) a.moves[2 * i] = a.moves[2 * i + 1] = -1;
}

// Phase 2: counts and tables in the new order.
__device__ void compact_apply(const CompactArgs &a) {
  const int64_t U = *a.used;
  const int64_t threads = (int64_t)gridDim.x * kBig, me = (int64_t)blockIdx.x * kBig + threadIdx.x;
  for (int64_t p = me; p < a.pages; p += threads) {
    int r = 0;
    if (p < U) {
      r = a.refs[p];
      if (r <= 0) r = a.refs[a.moves[2 * (int64_t)a.w.list[p]]];
    }
    a.refs_out[p] = r;
  }
  // A thread per entry of the table: its page, then that page's count and rank, then
  // its place, are three loads that wait for each other.
  const int64_t columns = a.to.max_pages, entries = columns * a.to.seqs;
  for (int64_t i = me; i < entries; i += threads) {
    const int64_t b = i / columns, c = i - b * columns;
    const int length = a.lengths[b];
    const int from = a.from.table[b * a.from.stride + c];
    int page = -1;
    if (fits(length, a.from) && c < pages_of(length, a.page_shift) && is_page(from, a.pages) && a.refs[from] > 0)
      page = from < U ? from : a.moves[2 * (int64_t)a.w.list[from] + 1];
    a.to.table[b * a.to.stride + c] = page;
  }
}

// Between phases of one workgroup.  A barrier is enough: its threads share a cache.  (A
// fence for the device writes L2 back, and took most of a small call's 28 us.)
__device__ __forceinline__ void phase_end() { __syncthreads(); }

template <int PHASE>  // -1: all of them
__global__ __launch_bounds__(kBig) void compact_kernel(CompactArgs a) {
  if constexpr (PHASE < 0 || PHASE == 0) compact_count(a);
  if constexpr (PHASE < 0) phase_end();
  if constexpr (PHASE < 0 || PHASE == 1) compact_rank(a);
  if constexpr (PHASE < 0) phase_end();
  if constexpr (PHASE < 0 || PHASE == 2) compact_apply(a);
}

// ---------------------------------------------------------------- copying

// 16 bytes at any word: the Q8_0 cache's scales need no more.
typedef uint32_t Sixteen __attribute__((ext_vector_type(4), aligned(4)));
// Bytes of a page that a workgroup takes at a time, eight loads of 16 bytes in flight
// per thread.
constexpr int kCopyLoads = 8;
constexpr int kCopyPiece = 16 * kThreads * kCopyLoads;

// Workgroup (x, y): the x-th piece of pages moves[y], moves[y + gridDim.y], ...; a
// page's four arrays are taken as one after another.  The next move is asked for
// before this one's bytes are stored.
__global__ __launch_bounds__(kThreads) void copy_kernel(CopyArgs a) {
  const int64_t whole = a.bytes[0] + a.bytes[1] + a.bytes[2] + a.bytes[3];
  // Where this thread's bytes lie: array and offset, the same in every page.
  const char *base[kCopyLoads];
  int64_t step[kCopyLoads];
#pragma unroll
  for (int k = 0; k < kCopyLoads; ++k) {
    int64_t o = (int64_t)blockIdx.x * kCopyPiece + 16 * (kThreads * k + (int)threadIdx.x);
    base[k] = nullptr;
    step[k] = 0;
    if (o >= whole) continue;
    base[k] = a.base[0];
    step[k] = a.bytes[0];
    if (o >= a.bytes[0]) {
      o -= a.bytes[0];
      base[k] = a.base[1];
      step[k] = a.bytes[1];
      if (o >= a.bytes[1]) {
        o -= a.bytes[1];
        base[k] = a.base[2];
        step[k] = a.bytes[2];
        if (o >= a.bytes[2]) {
          o -= a.bytes[2];
          base[k] = a.base[3];
          step[k] = a.bytes[3];
        }
      }
    }
    base[k] += o;
  }
  int64_t i = blockIdx.y;
  int from = a.moves[2 * i], to = a.moves[2 * i + 1];
  while (true) {
    const int64_t next = i + gridDim.y;
    int next_from = -1, next_to = -1;
    if (next < a.n) {
      next_from = a.moves[2 * next];
      next_to = a.moves[2 * next + 1];
    }
    if ((uint32_t)from < (uint64_t)a.pages && (uint32_t)to < (uint64_t)a.pages && from != to) {
      Sixteen x[kCopyLoads];
#pragma unroll
      for (int k = 0; k < kCopyLoads; ++k)
        if (base[k] != nullptr) x[k] = *reinterpret_cast<const Sixteen *>(base[k] + from * step[k]);
#pragma unroll
      for (int k = 0; k < kCopyLoads; ++k)
        if (base[k] != nullptr) *reinterpret_cast<Sixteen *>(const_cast<char *>(base[k]) + to * step[k]) = x[k];
    }
    if (next >= a.n) return;
    i = next;
    from = next_from;
    to = next_to;
  }
}

// Up to these sizes one workgroup does all of it.
// Resize, pages: it looks at those in front of the last free one that it gives, 0.24 us per
// 1024.  16 to 1000 sequences that take one page each, us, by launches of their own in
// brackets: free pages early in the pool 4.5 to 5.5 (14 to 15) at any size, none wanted 4 (13);
// free ones last 7.2 (13.8) in a pool of 16384, 10.8 (13.8) of 32768, 18.5 (13.9) of
// 65536, 22.4 (14) of 81920, 34 (14.2) of 131072.  Where the free pages lie is known
// on the device only.  At the border the one side loses 8.5 where they come last, the other 9.5
// where they come early.
// Table entries: where all leave 64 x 256 take 8.4 us, 1000 x 32 25.7; with
// the release in a launch of its own 7, but 5.5 instead of 4.0 where nothing changes.
constexpr int64_t kResizePages = 81920, kResizeEntries = 16384;
// Compact, pages: 2048 take 9.9 us, by three launches 11.6; 4096 13.0 and 13.4, 8192 17.7 and
// 14.  Entries: 64 x 64 11.2 and 11.6, 128 x 128 19.4 and 11.9.
constexpr int64_t kCompactPages = 4096, kCompactEntries = 4096;

}  // namespace

hipError_t launch_pages_fork(const ForkArgs &a, hipStream_t stream) {
  const int64_t wgs = std::min<int64_t>(((int64_t)a.to.seqs + kWaves - 1) / kWaves, 1 << 20);
  hipLaunchKernelGGL(fork_kernel, dim3((unsigned)wgs), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_pages_resize(const ResizeArgs &a, int cus, hipStream_t stream) {
  const bool small = a.pages <= kResizePages && a.t.seqs <= kSmallSeqs;
  if (small && (int64_t)a.t.seqs * a.t.max_pages <= kResizeEntries) {
    hipLaunchKernelGGL((resize_small_kernel<true>), dim3(1), dim3(kBig), 0, stream, a);
    return hipGetLastError();
  }
  const unsigned by_waves = (unsigned)std::min<int64_t>(((int64_t)a.t.seqs + kBigWaves - 1) / kBigWaves, 2 * cus);
  hipLaunchKernelGGL((resize_kernel<0>), dim3(by_waves), dim3(kBig), 0, stream, a);
  if (small) {
    hipLaunchKernelGGL((resize_small_kernel<false>), dim3(1), dim3(kBig), 0, stream, a);
    return hipGetLastError();
  }
  const unsigned tiles = (unsigned)std::min<int64_t>(std::max(pages_tiles(a.pages), seqs_tiles(a.t.seqs)), 2 * cus);
  hipLaunchKernelGGL((resize_kernel<1>), dim3(tiles), dim3(kBig), 0, stream, a);
  hipLaunchKernelGGL((resize_kernel<2>), dim3(tiles), dim3(kBig), 0, stream, a);
  hipLaunchKernelGGL((resize_kernel<3>), dim3((unsigned)std::min<int64_t>(seqs_tiles(a.t.seqs), 2 * cus)), dim3(kBig), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const CompactArgs &a, int cus, hipStream_t stream) {
  if (a.pages <= kCompactPages && (int64_t)a.to.seqs * a.to.max_pages <= kCompactEntries) {
    hipLaunchKernelGGL((compact_kernel<-1>), dim3(1), dim3(kBig), 0, stream, a);
    return hipGetLastError();
  }
  const unsigned tiles = (unsigned)std::max<int64_t>(std::min<int64_t>(pages_tiles(a.pages), 2 * cus), 1);
  hipLaunchKernelGGL((compact_kernel<0>), dim3(tiles), dim3(kBig), 0, stream, a);
  hipLaunchKernelGGL((compact_kernel<1>), dim3(tiles), dim3(kBig), 0, stream, a);
  hipLaunchKernelGGL((compact_kernel<2>), dim3((unsigned)(2 * cus)), dim3(kBig), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_pages_copy(const CopyArgs &args, int cus, hipStream_t stream) {
  CopyArgs a = args;
  const int64_t whole = a.bytes[0] + a.bytes[1] + a.bytes[2] + a.bytes[3];
  const int64_t pieces = (whole + kCopyPiece - 1) / kCopyPiece;  // below 2^22: a page is below 2^37 bytes
  // Enough workgroups for the device; each takes moves that far apart.
  const int64_t rows = std::max<int64_t>(std::min<int64_t>((int64_t)cus * 8 / pieces, 65535), 1);
  hipLaunchKernelGGL(copy_kernel, dim3((unsigned)pieces, (unsigned)std::min(rows, a.n)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace q8
