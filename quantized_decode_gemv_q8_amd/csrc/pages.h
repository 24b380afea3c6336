// Internal declarations of the operators on a pool of pages and the tables that
// own them, and of the copying of pages.
#pragma once

#include "q8_common.h"

namespace q8 {

struct PageTable {
  int *table;  // [seqs, max_pages], rows `stride` apart
  int64_t stride;
  int64_t max_tokens;  // of a row
  int seqs, max_pages;
};

// Pages and sequences are taken in tiles of this many.
constexpr int kPagesTile = 4096;
constexpr int kSeqsTile = 1024;
constexpr int64_t pages_tiles(int64_t pages) { return (pages + kPagesTile - 1) / kPagesTile; }
constexpr int64_t seqs_tiles(int64_t seqs) { return (seqs + kSeqsTile - 1) / kSeqsTile; }

// Parts of the workspace of resize and compact, in 8-byte words.
//   totals  per tile of sequences: pages they want
//   start   per sequence: pages wanted before it in its tile, and whether its last page is replaced (bit 62)
//   counts  per tile of pages: free (resize) or used (compact) ones
//   list    per page: the free pages in order (resize), ranks (compact)
struct PagesWork {
  int64_t *totals;
  int64_t *start;
  int *counts;
  int *list;
};
constexpr int64_t pages_work_bytes(int64_t pages, int64_t seqs) {
  return 8 * (seqs_tiles(seqs) + seqs) + 4 * (pages_tiles(pages) + pages);
}

struct ForkArgs {
  PageTable from, to;
  const int *lengths, *parent;
  int *lengths_out;
  int *refs;
  int pages, page_shift;
};
hipError_t launch_pages_fork(const ForkArgs &a, hipStream_t stream);

struct ResizeArgs {
  PageTable t;
  const int *before, *after;
  int *refs;
  int *moves;    // [seqs, 2]
  int *missing;  // [seqs]
  PagesWork w;
  int pages, page_shift;
};
hipError_t launch_pages_resize(const ResizeArgs &a, int cus, hipStream_t stream);

struct CompactArgs {
  PageTable from, to;
  const int *lengths;
  const int *refs;
  int *refs_out;
  int *moves;  // [pages / 2, 2]
  int *used;
  PagesWork w;
  int pages, page_shift;
};
hipError_t launch_pages_compact(const CompactArgs &a, int cus, hipStream_t stream);

// Copies pages moves[i][0] to moves[i][1] of up to four arrays.
struct CopyArgs {
  char *base[4];
  int64_t bytes[4];  // of a page, multiples of 16
  const int *moves;  // [n, 2]
  int64_t n;
  int64_t pages;
};
hipError_t launch_pages_copy(const CopyArgs &a, int cus, hipStream_t stream);

}  // namespace q8
