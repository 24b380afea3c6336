/*
 * q8_gemv.h -- C ABI of the MI355X (gfx950) Q8_0 matvec and i8 dot_t library.
 *
 * Operations (Phobos documentation pages):
 *   q8_matvec  "Q8_0 matvec" (docs/examples/q8-matvec), section "The tensors":
 *              C[m,n] = sum_k A[m,k] * W[k,n] * S[k/32, n], with i8 weights,
 *              one f32 scale per block of 32 rows along K and per column.
 *              Section "Factoring out the scale": the scale is applied once
 *              per block and column to the block's unscaled partial.
 *              Section "Bounds": N and K need not be multiples of any tile;
 *              the ragged column tile and the K remainder block are masked.
 *   q8_dot_t   "dot and tensor cores" (docs/language/dot-and-tensor-cores),
 *              table of built-ins and section "Hardware paths":
 *              C[m,n] = sum_k A[m,k] * W[n,k], i8 operands, i32 result.
 *   q8_cache_* a paged cache of keys and values in Q8_0 and the attention over
 *              it (declared and described below).
 *   q8_mx4_*   the same in 4-bit floats.
 *   q8_pages_* the pages of these caches: shared by forks, given and taken
 *              back as sequences grow and leave, moved together.
 *   q8_rope    rotary positions of queries and keys.
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers (memory of the current HIP
 *     device) to dense row-major arrays; there are no leading-dimension
 *     arguments (but for the rows and the page tables that q8_cache_*, q8_mx4_*,
 *     q8_pages_* and q8_rope take, which may be apart).  The caller owns them;
 *     the library only reads the inputs and overwrites the output (a cache, and
 *     a pool and its table, change in place where their operations say so).  It
 *     reads C only through an epilogue with row factors (corr != NULL, below).
 *     C must not alias an input.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls are asynchronous on that stream: a status of Q8_OK means the work
 *     was enqueued; faults surface at the caller's next synchronisation.
 *   - Arguments are validated on the host before anything is enqueued.  No
 *     C++ exception crosses this boundary.
 *   - Sizes: every extent must be >= 0.  M == 0 or N == 0 is a no-op.  The
 *     library uses 32-bit element offsets, so K*N, M*K and M*N must each be
 *     below 2^31 (otherwise Q8_ERR_TOO_LARGE).
 *   - Thread safety: concurrent calls are safe on distinct streams.  Host
 *     threads that share one stream must serialise their calls.
 *   - Workspace (the attentions, q8_pages_resize and q8_pages_compact take
 *     theirs from the caller; the other operations on caches, pages and
 *     positions need none): the split-K workspace (partial sums and arrival
 *     counters) is owned by the library, one per (device, stream).  It is allocated by
 *     the first call that needs it on that stream and grown by a later call
 *     that needs more; buffers it grows out of stay allocated (a graph
 *     captured earlier may still use them) until q8_release() frees them
 *     all.  Allocation cannot be recorded into a graph, so a call made while
 *     its stream is being captured and that would have to allocate or grow
 *     the workspace returns Q8_ERR_INVALID and enqueues nothing: make one
 *     eager call of the same (or a larger) shape on that stream first.
 *     Captured calls replay correctly: their arrival counters return to zero
 *     inside every launch, and no call records a memset.
 *   - XCD placement: when a matvec plan cuts every column tile into whole
 *     K runs and the tiles and workgroups are multiples of 8, the library
 *     places all runs of a tile on one XCD (the dispatcher deals workgroups
 *     to the eight XCDs in turn) and keeps the tile's split-K partials in
 *     that XCD's L2.  The first such call on a device, unless its stream is
 *     being captured, first runs a small probe kernel on the stream and
 *     waits for it (once per device and process) to confirm that placement;
 *     without it the partials go through the device's coherence point as for
 *     other plans.  If the contributors of a tile are ever found on
 *     different XCDs, that tile's outputs are written as NaN, never as a
 *     wrong sum.  The environment variable Q8_XCD_LOCAL=0 turns this off;
 *     results are bitwise the same either way.
 */
#ifndef Q8_GEMV_H
#define Q8_GEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum q8_status {
  Q8_OK = 0,
  Q8_ERR_INVALID = 1,            /* negative extent, null pointer with a non-zero extent, bad plan */
  Q8_ERR_TOO_LARGE = 2,          /* an offset would not fit the library's 32-bit indexing */
  Q8_ERR_UNSUPPORTED_DEVICE = 3, /* the current device is not gfx950 */
  Q8_ERR_HIP = 4                 /* a HIP call failed; see q8_last_hip_error() */
} q8_status;

/* Q8_0 block length along K ("The tensors": row b of S scales rows 32b..32b+31). */
#define Q8_BLOCK 32

/*
 * q8_matvec -- C = A (x) dequant(W, S).
 *   A  f32 [M, K]            activations, row-major
 *   W  i8  [K, N]            quantized weights, one column per output
 *   S  f32 [ceil(K/32), N]   scales; row b scales rows 32b .. min(32b+32, K)
 *   C  f32 [M, N]            output, overwritten (K == 0 writes zeros)
 * Errors: Q8_ERR_INVALID, Q8_ERR_TOO_LARGE, Q8_ERR_UNSUPPORTED_DEVICE,
 * Q8_ERR_HIP.  Deterministic: the same inputs give bitwise-equal outputs.
 */
q8_status q8_matvec(const float *A, const int8_t *W, const float *S, float *C,
                    int64_t M, int64_t K, int64_t N, void *stream);

/*
 * q8_matvec_noalloc -- q8_matvec that allocates nothing, for callers that
 * cannot call hipMalloc (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments, plan choice, kernels
 * and results (bitwise) as q8_matvec.  Instead of the library's workspace it
 * uses a fixed scratch array that every device the library runs on holds for
 * the life of the process: 32 MiB of split-K partial sums and 64 KiB of
 * arrival counters.  The counters are cleared once per device, on that
 * device's first call (a fill kernel on `stream`), and every launch leaves
 * them at zero again.  A call whose plan needs more partial space returns
 * Q8_ERR_TOO_LARGE and enqueues nothing (for example the matrix-core product
 * of 33..64 rows at N much above 28672); q8_matvec has no such limit.
 * All calls on one device share the scratch array: calls that overlap in
 * time on one device (on different streams, or concurrently from several
 * threads) race and give wrong results; serialise them.
 * Errors: as q8_matvec, plus Q8_ERR_TOO_LARGE for plans beyond the scratch.
 */
q8_status q8_matvec_noalloc(const float *A, const int8_t *W, const float *S, float *C,
                            int64_t M, int64_t K, int64_t N, void *stream);

/*
 * Launch plan of q8_matvec.  Every field 0 means "choose automatically".
 *   kind    Q8_PLAN_STREAM or Q8_PLAN_MATRIX (below); 0 picks one from the
 *           shape: the matrix cores, when allowed, above 16 rows; at 9..16
 *           rows when their automatic plan fills at least a quarter of the
 *           device, at 5..8 rows three eighths; at 3-4 rows when it fills
 *           half and K * N reaches 2^25; at 2 rows when it fills half and
 *           K * N reaches 2^27.
 * For Q8_PLAN_STREAM, the per-row FMA stream:
 *   vec     columns (= bytes of W) each lane loads per row: 16, 8, 4, 2 or 1.
 *           N must be a multiple of vec, W 'vec'-byte aligned and S
 *           min(16, 4*vec)-byte aligned.
 *   m_tile  activation rows per pass: 1, 2, 4 or 8, with m_tile*vec <= 32.
 *   workgroups  workgroups per pass over W.  W is cut into column tiles of
 *           64*vec columns and groups of four 32-row blocks along K; the
 *           (tile, group) units are dealt to the workgroups in contiguous runs
 *           of equal length (within one), at most 16/m_tile units each.  A
 *           tile shared by several workgroups is combined in K order.
 *   waves   waves per workgroup; 4 is the only value supported.
 * For Q8_PLAN_MATRIX, the matrix-core product of 2..64 rows ("dot and tensor
 * cores", "Hardware paths"; A is split into three bf16 parts so that the
 * result keeps f32 accuracy; one pass over W serves all rows): it needs
 * N % 4 == 0, 4-byte aligned W, 16-byte aligned S and 4*M*K < 2^31 (W is
 * read in 16-, 8- or 4-byte pieces, the widest that N and W's address both
 * allow, so a ragged last column tile is masked, "Bounds"; A's byte offsets
 * are 32-bit on this path; an explicit matrix plan beyond that returns
 * Q8_ERR_TOO_LARGE, and automatic plans use the stream), and serves
 * q8_matvec, q8_matvec_with_plan and a plain single-sibling fused call.
 *   vec, m_tile  must be 0.
 *   workgroups   tiles of 512 columns times K splits (a multiple of the tile
 *           count; every split gets at least one 32-row block; at most 65535
 *           splits, and one tile's split partials, splits x rows x 2 KiB with
 *           rows rounded up to 16, 32 or 64, below 2 GiB), or 0.
 *   waves   8 or 0 (eight waves per workgroup, 64 columns each).
 */
#define Q8_PLAN_STREAM 1
#define Q8_PLAN_MATRIX 2
#define Q8_MATRIX_MIN_ROWS 2
#define Q8_MATRIX_MAX_ROWS 64
typedef struct q8_plan {
  int32_t vec;
  int32_t m_tile;
  int32_t workgroups;
  int32_t waves;
  int32_t kind;
} q8_plan;

/*
 * q8_matvec_choose_plan -- host-only: the plan q8_matvec would use for these
 * extents on a device with `num_cus` compute units, given the byte
 * alignment of W's and S's addresses (pass the pointers' low bits, or 256
 * for allocator-aligned buffers).  Fills *out.  Touches no device.
 * Errors: Q8_ERR_INVALID (bad extents, num_cus < 1, out == NULL).
 */
q8_status q8_matvec_choose_plan(int64_t M, int64_t K, int64_t N,
                                int64_t w_align, int64_t s_align,
                                int32_t num_cus, q8_plan *out);

/*
 * q8_matvec_with_plan -- q8_matvec with explicit launch parameters (zero
 * fields are chosen automatically).  Results are equal for every valid plan
 * up to the f32 rounding of the summation order; a fixed plan is
 * deterministic.  Errors: as q8_matvec; Q8_ERR_INVALID for an unsupported
 * plan.
 */
q8_status q8_matvec_with_plan(const float *A, const int8_t *W, const float *S, float *C,
                              int64_t M, int64_t K, int64_t N, const q8_plan *plan,
                              void *stream);

/*
 * Fused matvec: sibling projections and the elementwise epilogue.
 *
 * "dot and tensor cores", section "The fused epilogue": the elementwise
 * statement that consumes a product runs on each element while the product
 * is written, with no second pass over a stored result (the page's examples
 * multiply a product by a scale, s = s * scale, and multiply an existing
 * accumulator by a factor before adding a product, acc = acc * corr +
 * dot(p, v)).  Here, for every sibling g:
 *
 *   C_g[m,n] = alpha * P_g[m,n] + corr[m] * C_g[m,n]     (corr != NULL)
 *   C_g[m,n] = alpha * P_g[m,n]                          (corr == NULL)
 *
 * where P_g = A (x) dequant(W_g, S_g) is the Q8_0 matvec of q8_matvec.  Each
 * output is rounded as fmaf(corr[m], C_old, alpha * P) (alpha * P alone
 * without corr), so alpha == 1 with no corr reproduces q8_matvec's values.
 *
 * Siblings are up to Q8_MAX_SIBLINGS weight sets of the same shape that share
 * the activation matrix A (for example the gate and up projections of an
 * MLP, or q, k and v); they run in one launch, which streams every sibling's
 * W and S once and stages A once per workgroup.
 */
#define Q8_MAX_SIBLINGS 4

typedef struct q8_sibling {
  const int8_t *W;  /* i8  [K, N], device */
  const float *S;   /* f32 [ceil(K/32), N], device */
  float *C;         /* f32 [M, N], device; read only when corr != NULL */
} q8_sibling;

typedef struct q8_epilogue {
  float alpha;        /* scale of the product */
  const float *corr;  /* f32 [M] device row factors of the existing C, or NULL */
} q8_epilogue;

/*
 * q8_matvec_fused -- the siblings' matvecs with the epilogue, in one launch.
 *   A         f32 [M, K], shared by all siblings
 *   siblings  host array of n_siblings (1..Q8_MAX_SIBLINGS) descriptors; the
 *             C arrays must be distinct and must not alias any input
 *   epilogue  host pointer, or NULL for alpha = 1 and no corr
 *   plan      as for q8_matvec_with_plan, or NULL for automatic; the
 *             siblings' tiles form one list of n_siblings * ceil(N/(64*vec))
 *             tiles, and W and S of every sibling must meet vec's alignment
 * K == 0 gives a zero product (C = corr[m] * C, or zeros).  Deterministic.
 * Errors: as q8_matvec; Q8_ERR_INVALID for n_siblings outside 1..4, a NULL
 * siblings array or pointer, or an unsupported plan.
 */
q8_status q8_matvec_fused(const float *A, const q8_sibling *siblings, int32_t n_siblings,
                          int64_t M, int64_t K, int64_t N, const q8_epilogue *epilogue,
                          const q8_plan *plan, void *stream);

/*
 * q8_dot_t -- C = A @ W^T in exact integer arithmetic.
 *   A  i8  [M, K]   row-major
 *   W  i8  [N, K]   row-major, one output row per row (K contiguous)
 *   C  i32 [M, N]   overwritten; each element is the exact sum reduced modulo
 *                   2^32 (exact whenever |sum| < 2^31, e.g. K <= 131071)
 * Errors: Q8_ERR_INVALID, Q8_ERR_TOO_LARGE, Q8_ERR_UNSUPPORTED_DEVICE,
 * Q8_ERR_HIP.
 */
q8_status q8_dot_t(const int8_t *A, const int8_t *W, int32_t *C,
                   int64_t M, int64_t K, int64_t N, void *stream);

/*
 * Dense f32 products ("dot and tensor cores": the table of built-ins, "The k
 * loop", "Hardware paths" and "The fused epilogue"):
 *   q8_dot_f32    C = alpha * (A @ B)   (+ corr[m] * C),  B f32 [K, N]
 *   q8_dot_t_f32  C = alpha * (A @ B^T) (+ corr[m] * C),  B f32 [N, K]
 *   A  f32 [M, K] row-major, device
 *   B  as above, row-major, device
 *   C  f32 [M, N] row-major, device; overwritten, read only when corr != NULL;
 *      must not alias A or B
 *   epilogue  host pointer, or NULL for alpha = 1 and no corr (an attention
 *      score tile is dot_t with alpha = 1/sqrt(head dim))
 * f32 operands and f32 accumulation: each operand is split exactly into three
 * bf16 parts and the six largest part products are accumulated in f32 on the
 * bf16 matrix cores (the three dropped ones are below 2^-24 |a b| together),
 * so the products keep f32 accuracy; each output is rounded as
 * fmaf(corr[m], C_old, alpha * P).  Any M, K, N >= 0; every pointer 4-byte
 * aligned; when K % 4 == 0 and A and B are 16-byte aligned (and N % 4 == 0
 * for q8_dot_f32), the k-contiguous operands take 16-byte loads.  Operands
 * below about 2^-110 in magnitude may lose their low parts to denormal
 * handling.  K == 0 gives a zero product.  Deterministic: the summation order
 * depends only on K.
 * Errors: Q8_ERR_INVALID (negative extent, NULL or misaligned pointer),
 * Q8_ERR_TOO_LARGE ((M + 128) * (K + 32) or (N + 128) * (K + 32) at or above
 * 2^30, or M * N at or above 2^31), Q8_ERR_UNSUPPORTED_DEVICE, Q8_ERR_HIP.
 */
q8_status q8_dot_f32(const float *A, const float *B, float *C, int64_t M, int64_t K, int64_t N,
                     const q8_epilogue *epilogue, void *stream);
q8_status q8_dot_t_f32(const float *A, const float *B, float *C, int64_t M, int64_t K, int64_t N,
                       const q8_epilogue *epilogue, void *stream);

/*
 * The Q8_0 cache: keys and values of an attention layer in pages, in the
 * weights' own format (i8 codes, one f32 scale per 32 values; value = code *
 * scale), what goes in and out of it, and the attention that reads it.
 *
 * A page holds page_size tokens of every head.  Codes of a token's row of dim
 * channels lie in pair order: channel d = 32 b + 2 j + i (j < 16, i < 2) is
 * byte j * (dim / 16) + 2 b + i of the row; block b's scale is scale b.
 */
typedef struct q8_cache {
  int8_t *K;         /* i8  [pages, heads, page_size, dim], device, 16-byte aligned */
  float *KS;         /* f32 [pages, heads, page_size, dim / 32], device */
  int8_t *V;         /* as K */
  float *VS;         /* as KS */
  int64_t pages;     /* below 2^31; the arrays themselves may be of any size */
  int32_t heads;     /* 1 .. 65535 */
  int32_t page_size; /* a power of two, 16 .. 1024 */
  int32_t dim;       /* 64, 128 or 256 */
} q8_cache;

/*
 * The sequences of a call (device arrays, read when the work runs, so a
 * captured graph follows their contents).  Sequence b owns the pages
 * table[b, 0], table[b, 1], ... and holds lengths[b] tokens, the new ones
 * among them: its newest n = offsets[b+1] - offsets[b] tokens are rows
 * offsets[b] .. offsets[b+1]-1 of the call's row tensors.  Rows before
 * offsets[0] and from offsets[seqs] on belong to no sequence: what they hold
 * counts for nothing (a write may load it), and none of them is written.  Sequences must
 * not share pages that a call writes.
 *
 * The contents are checked where they are used: a sequence whose offsets do
 * not ascend within the rows has no rows; one with lengths[b] < n, or with more
 * tokens than its table row holds, and a position whose page is not one of
 * the cache's (0 .. pages-1), is skipped by a write or keep, and gives NaN in
 * the rows of a read or an attention that would need it (a cache of no pages
 * holds no tokens at all).  A row that the
 * offsets give to two sequences holds either one's result.
 */
typedef struct q8_cache_seqs {
  const int32_t *table;   /* [seqs, max_pages], rows table_stride apart; entries past a sequence's tokens are not read */
  const int32_t *lengths; /* [seqs] */
  const int32_t *offsets; /* [seqs + 1], ascending */
  int64_t seqs;
  int64_t max_pages;      /* max_pages * page_size below 2^30 */
  int64_t table_stride;
} q8_cache_seqs;

/* Element types of the rows outside the cache. */
typedef enum q8_type { Q8_F32 = 0, Q8_BF16 = 1, Q8_F16 = 2 } q8_type;

/*
 * q8_cache_write -- quantises the new tokens' keys and values into the cache.
 *   k, v  [rows, heads, dim] of `type`, rows k_stride / v_stride elements apart
 *         (at least heads * dim), aligned to their elements
 * Per 32 channels x: scale = f32(max|x| / 127), code = x / scale rounded to
 * the nearest, ties to even, both correctly rounded (a scale of zero gives
 * zeros; where the scale is denormal and so coarse that a quotient passes 127,
 * the code is 127).  A block that holds an infinity or a NaN is stored so that it reads
 * back as NaN.  Everything else in the cache is left as it was.
 * q8_cache_read -- the reverse: k, v = code * scale, an f32 product that is then
 * rounded to `type`, for the newest tokens of each sequence (offsets that count all of its tokens
 * read the whole sequence).
 * Errors of both: Q8_ERR_INVALID, Q8_ERR_TOO_LARGE, Q8_ERR_UNSUPPORTED_DEVICE,
 * Q8_ERR_HIP.
 */
q8_status q8_cache_write(const q8_cache *cache, const void *k, const void *v, q8_type type,
                         int64_t rows, int64_t k_stride, int64_t v_stride,
                         const q8_cache_seqs *seqs, void *stream);
q8_status q8_cache_read(const q8_cache *cache, void *k, void *v, q8_type type, int64_t rows,
                        int64_t k_stride, int64_t v_stride, const q8_cache_seqs *seqs,
                        void *stream);

/*
 * q8_cache_keep -- after a tree of drafted tokens has been verified, moves the
 * accepted ones to the front of the sequence's new tokens: for a = 0, 1, ...
 * the codes and scales of new token keep[b, a] go to the place of new token a.
 *   keep  i32 [seqs, width], device: indexes among sequence b's new tokens in
 *         strictly ascending order; the first entry that is negative, not
 *         below n or not above the one before it ends the list
 *   rows  of the row tensors that the offsets refer to
 * Places past the kept ones hold what they held or were moved from; the caller
 * shortens lengths[b].
 */
q8_status q8_cache_keep(const q8_cache *cache, int64_t rows, const q8_cache_seqs *seqs,
                        const int32_t *keep, int64_t width, void *stream);

/*
 * q8_cache_attention -- attention of the new tokens' queries over the cache
 * (their own keys and values included: write them first):
 *   out[t, h] = sum_j softmax_j(alpha * q[t, h] . K[j, h / g]) V[j, h / g]
 * with g = q_heads / heads, over the tokens j that row t sees: all tokens
 * before the new ones, and of the new ones
 *   tree == NULL  those up to the row's own (one new token per sequence is
 *                 plain decoding, many are a piece of a prompt)
 *   tree != NULL  those whose bit is set: bit j % 64 of word j / 64 of the
 *                 row's tree_words words (u64 [rows, tree_words], 8-byte
 *                 aligned) for new token j; tokens past the words are not seen
 * A row that sees nothing gives zeros.  What a token that no row sees holds
 * (NaN among it) changes nothing.
 *   q, out  [rows, q_heads, dim] of `type`, rows q_stride / out_stride elements
 *           apart; out must not overlap anything else
 *   workspace  device memory of at least the size that
 *           q8_cache_attention_workspace gives for the same cache, type, rows,
 *           q_heads, seqs and max_pages, 16-byte aligned (NULL where that size is 0); its
 *           contents need no preparation and are free again when the call's work is done.
 *           Calls that may overlap in time (and graphs whose replays may) need one each
 * Sums, maxima, scores, weights and scales are f32, and codes are exact.  What
 * the matrix cores take of the rest is rounded as follows.
 *   q        f32 rows: to 2^-23 of the row's largest channel; bf16 and f16 rows: not
 *            at all (channels below 2^-32 of the row's largest lose bits)
 *   weights  (each times its value scale) f32 rows: not at all; bf16 and f16
 *            rows: to 2^-16 of itself (products below 2^-110 may lose more).  This
 *            holds for any number of rows and whatever else a call brings
 * A query that is not finite, a key whose score is NaN or +infinity and a value
 * scale that is not finite give NaN in the rows that see them (a value scale in
 * its block of channels).
 * With scales up to 2^60 (values up to 2^67) no sum overflows.
 * Deterministic: the order of the sums depends on the extents, the lengths and
 * offsets, never on timing.
 * Errors: as q8_cache_write; Q8_ERR_INVALID also for q_heads that is no multiple
 * of heads and for a missing, misaligned or small workspace; Q8_ERR_TOO_LARGE also
 * for more than 2^24 query heads and where seqs * rows * heads * max_pages * page_size
 * is so large (about 2^57 and more) that the work cannot be numbered.
 */
q8_status q8_cache_attention_workspace(const q8_cache *cache, q8_type type, int64_t rows,
                                       int32_t q_heads, const q8_cache_seqs *seqs, int64_t *bytes);
q8_status q8_cache_attention(const q8_cache *cache, const void *q, void *out, q8_type type,
                             int64_t rows, int32_t q_heads, int64_t q_stride, int64_t out_stride,
                             const q8_cache_seqs *seqs, const uint64_t *tree, int64_t tree_words,
                             float alpha, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The cache in 4-bit floats: the same pages, sequences and operations as the
 * Q8_0 cache in a little under half of its bytes (a token's key and value of 128
 * channels: 136 instead of 288).
 *
 * A code is 4 bits: sign, then the index of 0, 0.5, 1, 1.5, 2, 3, 4 or 6.  32
 * channels of a row share a scale byte e, which stands for 2^(e - 127); value = code
 * * scale, exactly.  255 stands for NaN; bytes of 253 and 254 are not used, and
 * what they give is not defined.
 * Channel d = 32 b + 2 j + i of a token's row (j < 16, i < 2) is nibble i (low first) of
 *   K  byte j * (dim / 32) + b of the row's dim / 2;
 *   V  byte (4 j + token % 4) * (dim / 32) + b of the 2 * dim that tokens 4 n .. 4 n + 3 of
 *      a page share (token: the place within the page).
 * Block b's scale is byte b of the token's scales.
 */
typedef struct q8_mx4_cache {
  uint8_t *K;        /* u8 [pages, heads, page_size, dim / 2], device; all four 16-byte aligned */
  uint8_t *KS;       /* u8 [pages, heads, page_size, dim / 32] */
  uint8_t *V;        /* as K */
  uint8_t *VS;       /* as KS */
  int64_t pages;     /* these as in q8_cache */
  int32_t heads;
  int32_t page_size;
  int32_t dim;
} q8_mx4_cache;

/*
 * q8_mx4_write, q8_mx4_read, q8_mx4_keep, q8_mx4_attention -- what q8_cache_write,
 * q8_cache_read, q8_cache_keep and q8_cache_attention do, for this cache; the
 * arguments, what is checked where, and what happens to sequences that are
 * described wrongly are the same, but for
 *   write      per 32 channels x: s = the smallest power of two with max|x| <= 7 s, from 2^-125
 *              to 2^125; code = x / s to the nearest, ties to the even code, with its
 *              sign, at most 6.  A block that holds an infinity or a NaN reads back as NaN
 *   read       code * s, rounded once to `type`
 *   attention  alpha must be finite.  Keys, values and queries reach the matrix cores
 *              exactly (parts of a query below 2^-126, or of a value below 2^-126,
 *              may be lost).  Weights are rounded to 2^-16 of themselves for bf16 and f16
 *              rows, not at all for f32; those below 2^-126 of the row's largest count
 *              for nothing.  Everything else is f32
 * Errors: as theirs; Q8_ERR_INVALID also for arrays that are not 16-byte aligned and an alpha
 * that is not finite.
 */
q8_status q8_mx4_write(const q8_mx4_cache *cache, const void *k, const void *v, q8_type type,
                       int64_t rows, int64_t k_stride, int64_t v_stride, const q8_cache_seqs *seqs,
                       void *stream);
q8_status q8_mx4_read(const q8_mx4_cache *cache, void *k, void *v, q8_type type, int64_t rows,
                      int64_t k_stride, int64_t v_stride, const q8_cache_seqs *seqs, void *stream);
q8_status q8_mx4_keep(const q8_mx4_cache *cache, int64_t rows, const q8_cache_seqs *seqs,
                      const int32_t *keep, int64_t width, void *stream);
q8_status q8_mx4_attention_workspace(const q8_mx4_cache *cache, q8_type type, int64_t rows,
                                     int32_t q_heads, const q8_cache_seqs *seqs, int64_t *bytes);
q8_status q8_mx4_attention(const q8_mx4_cache *cache, const void *q, void *out, q8_type type,
                           int64_t rows, int32_t q_heads, int64_t q_stride, int64_t out_stride,
                           const q8_cache_seqs *seqs, const uint64_t *tree, int64_t tree_words,
                           float alpha, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The pages of a cache: who owns them, and how they are shared.
 *
 * A pool counts owners: refs[p] is the number of table rows that own page p; a
 * page with refs[p] <= 0 is free.  The caches of all layers share one pool and one
 * table.  Everything is on the device and read when the work runs, so a captured
 * decode step can grow its sequences.  Table rows hold -1 where they own no page.
 * Results depend on the order of pages and sequences, never on timing.
 */
typedef struct q8_pool {
  int32_t *refs;     /* i32 [pages], device */
  int64_t pages;     /* 0 .. 2^31 - 1 */
  int32_t page_size; /* tokens: a power of two, 16 .. 1024 */
} q8_pool;

typedef struct q8_page_table {
  int32_t *table;       /* i32 [seqs, max_pages], device, rows table_stride apart */
  int64_t seqs;
  int64_t max_pages;    /* max_pages * page_size below 2^30 */
  int64_t table_stride; /* at least max_pages */
} q8_page_table;

/*
 * q8_pages_fork -- children share their parents' pages: row i of `to` becomes
 * the pages of the lengths[parent[i]] tokens of row parent[i] of `from`, each of
 * which counts one owner more, and -1 behind them; lengths_out[i] = lengths[parent[i]].
 * A child whose parent is no row of `from`, or whose length is negative or past either
 * table's columns, gets no pages and length 0; an entry that is no page is copied as
 * -1.  What the rows of `to` owned before is not released (resize them to 0 first).
 *   lengths      i32 [from->seqs], device
 *   parent       i32 [to->seqs], device; any row any number of times
 *   lengths_out  i32 [to->seqs], device
 * `to` and lengths_out must not overlap anything else.
 */
q8_status q8_pages_fork(const q8_pool *pool, const q8_page_table *from, const int32_t *lengths,
                        const int32_t *parent, const q8_page_table *to, int32_t *lengths_out,
                        void *stream);

/*
 * q8_pages_resize -- sequences grow, shrink or leave: sequence b holds the pages of
 * before[b] tokens (entries 0 .. ceil(before / page_size) - 1 of its row) and is to
 * hold those of after[b].
 *   1. Pages past what after[b] needs lose an owner, and their entries become -1
 *      (after[b] = 0 frees the sequence).
 *   2. A sequence that grows and whose last page is partly filled and shared
 *      (refs > 1 after step 1) gets a page of its own in its place, and then its new ones.
 *      Pages are given in the order of the sequences, the lowest free ones first;
 *      what step 1 released counts as free, what step 2 replaces does not yet.
 *      A sequence that cannot have all that it lacks gets none, as does every later
 *      one that lacks any.
 *   moves    i32 [seqs, 2]: (replaced page, its replacement), or (-1, -1); copy them in
 *            every layer's cache (q8_cache_copy, q8_mx4_copy) before the new tokens are
 *            written
 *   missing  i32 [seqs]: 0, or the pages that the sequence lacks (nothing of it has
 *            changed: give it the same lengths again once pages are free, the others
 *            after[b] as their before[b]), or -1 where before[b] or after[b] is negative or
 *            past the table (it is left alone).  New tokens of a sequence with anything
 *            but 0 must not be written: its last page may still be others' too.  With a
 *            length of -1 in that step the cache's calls write none and give NaN
 *   workspace  q8_pages_workspace bytes of device memory, 16-byte aligned; needs no preparation, and
 *            one call at a time may use it
 * Entries that are no page are released as nothing and never replaced.
 */
q8_status q8_pages_resize(const q8_pool *pool, const q8_page_table *table, const int32_t *before,
                          const int32_t *after, int32_t *moves, int32_t *missing, void *workspace,
                          int64_t workspace_bytes, void *stream);

/*
 * q8_pages_compact -- the order in which the used pages of a pool lie at its
 * front: with U used pages, those from page U on move to the free ones below U, both
 * in ascending order; the others stay.
 *   lengths    i32 [from->seqs], device: tokens of each row, whose pages are renamed
 *   refs_out   i32 [pages]: the counts in the new order
 *   to         the table with the new names, as many rows and columns as `from`; -1 behind a
 *              row's pages, in rows whose length is negative or past the table, and for
 *              entries that are no used page
 *   moves      i32 [pages / 2, 2]: (from, to), and (-1, -1) behind the last move; copy them in
 *              every layer's cache before the new table is used
 *   used       i32 [1]: U
 *   workspace  as of q8_pages_resize
 * Nothing that is read is written: refs and `from` stay as they were.
 */
q8_status q8_pages_compact(const q8_pool *pool, const q8_page_table *from, const int32_t *lengths,
                           int32_t *refs_out, const q8_page_table *to, int32_t *moves, int32_t *used,
                           void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes that q8_pages_resize and q8_pages_compact need for this many pages and sequences; host only. */
q8_status q8_pages_workspace(int64_t pages, int64_t seqs, int64_t *bytes);

/*
 * q8_cache_copy, q8_mx4_copy -- page moves[i, 0] of the cache, all heads, codes and
 * scales of keys and values, is copied to page moves[i, 1], for i < n.  A pair that
 * is not two different pages of the cache is passed over.  No page may be written twice, or
 * written and read (moves of one resize or compact never are).
 *   moves  i32 [n, 2], device
 * Errors of all page operations: Q8_ERR_INVALID, Q8_ERR_TOO_LARGE, Q8_ERR_UNSUPPORTED_DEVICE,
 * Q8_ERR_HIP.
 */
q8_status q8_cache_copy(const q8_cache *cache, const int32_t *moves, int64_t n, void *stream);
q8_status q8_mx4_copy(const q8_mx4_cache *cache, const int32_t *moves, int64_t n, void *stream);

/*
 * Rotary positions: the first `rot` channels of every head are rot / 2 pairs, and pair
 * i of a row at position p turns by the angle p * f_i:
 *   (x, y) -> amplitude * (x cos - y sin, x sin + y cos)
 * Pair i is channels (2 i, 2 i + 1) if interleaved, (i, i + rot / 2) if not.  The other
 * channels stay as they are.  Frequencies are held as fractions of a turn in 64 bits,
 * so that the angle is exact at any position; sine, cosine and products are f32,
 * rounded once to the rows' type.
 */
typedef struct q8_rope_angles {
  const uint64_t *turns; /* [rot / 2], device, 8-byte aligned: as q8_rope_turns makes them */
  int32_t rot;           /* even, 2 .. dim */
  int32_t interleaved;
  float amplitude;       /* 1 unless the scaling wants another */
} q8_rope_angles;

#define Q8_MAX_ROPE_TENSORS 4
typedef struct q8_rope_rows {
  const void *x;      /* [rows, heads, dim], rows x_stride elements apart (at least heads * dim) */
  void *out;          /* the same, out_stride apart; x itself (with its stride), or no part of any x */
  int32_t heads;
  int64_t x_stride, out_stride;
} q8_rope_rows;

/*
 * q8_rope -- turns the rows of up to Q8_MAX_ROPE_TENSORS tensors (queries and keys, say) that
 * share their positions, in one launch.
 *   positions  i32 [rows], device, of any sign; or NULL:
 *   seqs       the rows' sequences (its lengths and offsets; the table is not used): new token i of
 *              sequence b, row offsets[b] + i, is at lengths[b] - n + i.  Rows of no sequence are
 *              not written.  NULL where positions are given
 *   inverse    nonzero: turns back (the sine's sign changes, the amplitude stays): the gradient
 *              of the forward turn, and with an amplitude of 1 its inverse
 *   dim        2 .. 4096
 * Errors: Q8_ERR_INVALID, Q8_ERR_TOO_LARGE, Q8_ERR_UNSUPPORTED_DEVICE, Q8_ERR_HIP.
 */
q8_status q8_rope(const q8_rope_angles *angles, const q8_rope_rows *tensors, int32_t n_tensors,
                  q8_type type, int64_t rows, int32_t dim, const int32_t *positions,
                  const q8_cache_seqs *seqs, int32_t inverse, void *stream);

/* Host only: turns[i] = frequencies[i] / (2 pi) modulo 1, in units of 2^-64 (finite radians per position). */
q8_status q8_rope_turns(const double *frequencies, int64_t n, uint64_t *turns);

/*
 * q8_rope_frequencies -- host only: frequencies[i] = base^(-2 i / rot), i < rot / 2, for a
 * context stretched by `factor`:
 *   Q8_ROPE_PLAIN   as they are (factor is not used)
 *   Q8_ROPE_LINEAR  all divided by factor
 *   Q8_ROPE_BASE    from base * factor^(rot / (rot - 2)) (rot of 4 or more), so that the slowest is
 *                   divided by factor and the fastest stays
 *   Q8_ROPE_TURNS   by the turns r that the pair makes in the `length` tokens of the
 *                   unstretched context: divided for r <= low, kept for r >= high, and between
 *                   w f + (1 - w) f / factor with w = (r - low) / (high - low)
 *   Q8_ROPE_INDEX   the same, with w linear in the pair's index: 1 at
 *                   max(floor(index(high)), 0), 0 at min(ceil(index(low)), rot - 1), where
 *                   index(r) = rot ln(length / (2 pi r)) / (2 ln base)
 */
typedef enum q8_rope_scaling {
  Q8_ROPE_PLAIN = 0, Q8_ROPE_LINEAR = 1, Q8_ROPE_BASE = 2, Q8_ROPE_TURNS = 3, Q8_ROPE_INDEX = 4
} q8_rope_scaling;
q8_status q8_rope_frequencies(int32_t rot, double base, q8_rope_scaling scaling, double factor,
                              double length, double low, double high, double *frequencies);

/* Static, human-readable name of a status code (never NULL). */
const char *q8_status_string(q8_status s);

/* The hipError_t behind the calling thread's most recent Q8_ERR_HIP (0 if none). */
int q8_last_hip_error(void);

/* Frees every library-owned workspace, including buffers a workspace grew out
 * of, after synchronising the device(s) that own one.  Call it when no call is
 * in flight and no captured graph that uses the workspaces will be replayed
 * again.  The scratch array of q8_matvec_noalloc is not freed. */
void q8_release(void);

#ifdef __cplusplus
}
#endif

#endif /* Q8_GEMV_H */
