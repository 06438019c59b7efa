/*
 * satk.h -- C ABI of libsatk.so: exact per-row top-K for a DSA sparse
 * attention indexer, on one GB300 (sm_103a).
 *
 * Pages cited by title and section:
 *  [P1] vLLM PR #65178 "DCP top-k merge reads the rank-major all-gather
 *       buffer in place": Overview (rank-major [W, R, K, 2] (score,
 *       global_id) buffer read in place), Details (topk in {512,1024,2048}).
 *  [P2] vLLM API page vllm.models.kimi_k3.nvidia.ops.dcp_topk_merge.kernels:
 *       module docstring (B' word, exactness, saturation, rescue),
 *       DCPTopkPackKernel, DCPTopkSelectKernel, DCPTopkRescueKernel,
 *       DCPTopkRescueWorkspace, dcp_topk_pack_indices, dcp_topk_select,
 *       _check_exact.
 *  [P3] vLLM PR #57206 "Use DeepSelect for eligible sparse-indexer prefill
 *       chunks": Purpose (causal per-row end bounds, preallocated output),
 *       Test Plan (strided output, untouched padding, -1 tails).
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller.  No entry
 *    point allocates, frees or synchronises; each enqueues its kernels on
 *    `stream` (NULL = the legacy default stream) and returns at once.
 *    Inputs must stay unmodified, and outputs untouched by others, until
 *    the stream reaches the call.
 *  - Sizes are element counts; strides (`ld_*`) are in elements.
 *  - Host-side argument checks run before any launch.  A rejected call
 *    launches nothing and returns a negative SATK_E* code; there is no
 *    fallback of any kind.  SATK_ECUDA reports a launch failure.
 *  - Scores rank descending with NaN dropped, +-inf ordinary and -0.0 just
 *    below +0.0; ties break toward the lower id.
 *  - `status` (where taken) is a nullable device int32; the kernels OR
 *    SATK_STATUS_* bits into it and never clear it.
 */
#ifndef SATK_H_
#define SATK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without the CUDA headers: the same opaque struct pointer. */
struct CUstream_st;
typedef struct CUstream_st *satk_stream_t;

enum satk_dtype { SATK_F32 = 0, SATK_BF16 = 1, SATK_F16 = 2 };
enum satk_format { SATK_PAIRS_F32 = 0, SATK_PACKED_BF16 = 1 };

enum satk_rc {
  SATK_OK = 0,
  SATK_EINVAL = -1,       /* a pointer, size, stride or alignment is invalid */
  SATK_EUNSUPPORTED = -2, /* valid, but outside the instantiated range       */
  SATK_ECUDA = -3         /* the launch itself failed                         */
};

/* device status bits */
#define SATK_STATUS_SLOTS_EXCEEDED 1 /* more saturated ranks than rescue slots:
                                        the row keeps its round-1 ids [P2
                                        DCPTopkSelectKernel] */
#define SATK_STATUS_DUPLICATE_KEYS 2 /* a repeated (score, id) candidate sat
                                        on the cut: fewer than K ids kept   */
#define SATK_STATUS_BAD_REQUEST 4    /* satk_dcp_emit_rows: a req_id outside
                                        the block table; that row emits
                                        nothing (also satk_latent_attend)   */
#define SATK_STATUS_NO_BLOCK 8       /* satk_step_tables: a token on this rank
                                        has no block (free list or table
                                        width used up); its slot is -1      */
#define SATK_STATUS_TOO_MANY_TOKENS 16 /* satk_step_tables: more new tokens
                                        than the token arrays hold          */
#define SATK_STATUS_BAD_ROW 32       /* a physical row outside the cache (or
                                        above 2**31 - 1 in a slot): skipped  */
#define SATK_STATUS_BAD_POSITION 64  /* satk_latent_store: a position outside
                                        the cos/sin table; token skipped    */
#define SATK_STATUS_STALLED 128      /* an attention kernel gave up a wait
                                        inside the GPU (about two seconds):
                                        results that it may have touched are
                                        NaN, with or without a status word   */

/* Largest K of satk_topk_rows and of the rescue push. */
#define SATK_TOPK_MAX_K 4096
/* Largest W * n of the merges, and of W * n + ((k-1)/n) * k in the rescue. */
#define SATK_MERGE_MAX_CANDIDATES 32768
/* Local ids of the packed format are below 2**17 [P2 module docstring]. */
#define SATK_LOCAL_INDEX_LIMIT (1 << 17)

/*
 * satk_topk_rows -- exact top-k of each row of a logits matrix [P3 Purpose].
 *
 * logits : [rows, ld_logits] of `dtype` (SATK_F32 float, SATK_BF16 raw
 *          bfloat16); row i's candidates are columns [0, end_i), end_i =
 *          clamp(row_ends[i], 0, cols), or cols when row_ends is NULL.
 *          Columns >= end_i are never read.
 * k      : 1..SATK_TOPK_MAX_K.
 * out    : int32 [rows, ld_out], ld_out >= k.  Row i receives the column
 *          ids of its k best scores: first those strictly above the k-th
 *          score, ascending, then those equal to it (the lowest columns of
 *          the tie), ascending; a row with fewer than k non-NaN candidates
 *          lists them all in ascending order, then -1.  Columns [k, ld_out)
 *          are never written.
 * Errors : SATK_EINVAL for NULL logits/out, rows < 0, cols < 0,
 *          ld_logits < cols, k outside 1..SATK_TOPK_MAX_K, ld_out < k,
 *          cols >= 2**31, or an unknown dtype.
 */
int satk_topk_rows(const void *logits, int dtype, int64_t rows, int64_t cols,
                   int64_t ld_logits, const int32_t *row_ends, int32_t k,
                   int32_t *out, int64_t ld_out, satk_stream_t stream);

/*
 * satk_topk_rows_sorted -- satk_topk_rows with the chosen ids in score
 * order: descending score, ties by ascending column (a score-sorted output
 * option; the pages' selectors never sort, they emit in an order fixed by
 * their thread layout [P2 DCPTopkSelectKernel]).  The chosen set, the -1
 * tail, the untouched columns
 * [k, ld_out), the arguments and the errors are those of satk_topk_rows.
 * Slower: every row takes one CTA and a shared-memory sort of the k ids.
 */
int satk_topk_rows_sorted(const void *logits, int dtype, int64_t rows,
                          int64_t cols, int64_t ld_logits,
                          const int32_t *row_ends, int32_t k, int32_t *out,
                          int64_t ld_out, satk_stream_t stream);

/*
 * satk_dcp_pack -- pack a local top-n into B' rows [P2 DCPTopkPackKernel,
 * dcp_topk_pack_indices].
 *
 * logits_bf16 : [rows, ld_logits] raw bfloat16 scores, S valid columns.
 * local_idx   : int32 [rows, ld_idx], slots [0, n) of each row; -1 pads.
 * n           : a positive multiple of 32.
 * row_ends    : nullable int32 [rows].
 * packed      : int32 [rows, n + n/32], contiguous.  Slot j holds
 *               (ord16(score) << 16) | (0xFFFF - (local & 0xFFFF)), or 0
 *               when local is outside [0, min(row_end, S, 2**17)) or its
 *               score is NaN; word n + j/32 holds bit (local >> 16) & 1 at
 *               bit j % 32.  ord16 flips a negative bf16 pattern and sets
 *               the sign bit of a non-negative one [P2 _ord16].
 * Errors      : SATK_EINVAL for NULL pointers, rows < 0, S < 0,
 *               ld_logits < S, n not a positive multiple of 32, ld_idx < n.
 */
int satk_dcp_pack(const uint16_t *logits_bf16, int64_t rows, int64_t S,
                  int64_t ld_logits, const int32_t *local_idx, int64_t ld_idx,
                  int32_t n, const int32_t *row_ends, int32_t *packed,
                  satk_stream_t stream);

/*
 * satk_dcp_topk_pack -- each bf16 row's local top-n written straight as a B'
 * row: the result of satk_dcp_pack applied to the ids satk_topk_rows(logits,
 * n) returns, in one pass over the logits and without the ids or the
 * gathered re-read of the scores [P2 DCPTopkPackKernel, dcp_topk_pack_indices;
 * P3 Purpose for the row top-K].
 *
 * logits_bf16 : [rows, ld_logits] raw bfloat16, S valid columns; row i's
 *               candidates are columns [0, min(row_ends[i], S)) (NULL row_ends:
 *               S).  Columns >= end are never read.
 * n           : a positive multiple of 32, at most SATK_TOPK_MAX_K.
 * packed      : int32 [rows, n + n/32], contiguous.  Slot j holds the B' word
 *               of the j-th id of the row's top-n layout (satk_topk_rows: the
 *               ids above the n-th score ascending, then its ties), or 0 past
 *               the last valid column or for a column >= 2**17; word n + j/32
 *               holds that column's bit 16 at bit j % 32.
 * Errors      : SATK_EINVAL for NULL pointers, rows < 0, S < 0, ld_logits < S,
 *               n not a positive multiple of 32 or above SATK_TOPK_MAX_K,
 *               S >= 2**31.
 */
int satk_dcp_topk_pack(const uint16_t *logits_bf16, int64_t rows, int64_t S,
                       int64_t ld_logits, const int32_t *row_ends, int32_t n,
                       int32_t *packed, satk_stream_t stream);

/*
 * satk_dcp_merge_select -- top-k over a rank-major candidate buffer read in
 * place [P1 Overview; P2 DCPTopkSelectKernel].
 *
 * cand   : SATK_PAIRS_F32: [W, T, n, 2] 4-byte elements (float score,
 *          int32 global id); an entry with id < 0 or a NaN score is empty.
 *          SATK_PACKED_BF16: int32 [W, T, n + n/32] B' rows; global id
 *          local * W + r for rank r, 0 words empty.
 *          Both contiguous; the pairs buffer 16-byte aligned.
 * W, n   : ranks and candidates per rank; W * n <=
 *          SATK_MERGE_MAX_CANDIDATES; packed needs W <= 16 and n % 32 == 0;
 *          pairs needs n % 32 == 0.
 * k      : 1..W*n is useful; any k >= 1 is accepted.  The chosen set is
 *          the k best under (score desc, global id asc); fewer than k
 *          non-empty candidates keep them all.
 * ids_out: int32 [T, ld_out], ld_out >= k: the chosen global ids in
 *          ascending flat candidate order (rank-major, then slot), then -1.
 * sat_word: packed only (nullable): int32 [T], (mask << 16) | tau16 with
 *          tau16 the ord16 of the k-th chosen candidate (0 when fewer than
 *          k were chosen) and bit r of mask set iff all n slots of rank r
 *          hold words with ord16 > tau16; a mask with more than (k-1)/n
 *          bits is cleared and SATK_STATUS_SLOTS_EXCEEDED raised
 *          [P2 DCPTopkSelectKernel docstring].
 * Errors : SATK_EINVAL for NULL cand/ids_out, W < 1, T < 0, n < 1, k < 1,
 *          ld_out < k, an unknown format, a shape rule above, a pairs
 *          buffer not 16-byte aligned, or a non-NULL sat_word with the
 *          pairs format; SATK_EUNSUPPORTED when W * n exceeds
 *          SATK_MERGE_MAX_CANDIDATES.
 */
int satk_dcp_merge_select(const void *cand, int format, int32_t W, int64_t T,
                          int32_t n, int32_t k, int32_t *ids_out,
                          int64_t ld_out, int32_t *sat_word, int32_t *status,
                          satk_stream_t stream);

/*
 * satk_dcp_rescue_select -- second round of the packed merge for the rows
 * whose sat_word mask is non-zero [P2 module docstring, DCPTopkRescueKernel,
 * push_local_topk].
 *
 * packed      : int32 [W, T, n + n/32], the round-1 input.
 * logits_bf16 : [W, T, ld_logits] raw bfloat16 (rank-major rows of S
 *               valid columns); row_ends nullable int32 [W, T].
 * sat_word    : int32 [T] as written by satk_dcp_merge_select.
 * recv        : int32 scratch of satk_rescue_recv_words(T, n, k) words,
 *               [T, (k-1)/n, k + k/32].  For a row with mask != 0, slot s
 *               receives the s-th saturated rank's local top-min(k, valid)
 *               in B' layout (the same column order as satk_topk_rows), 0
 *               after; other slots and rows are not written.
 * ids_out     : int32 [T, ld_out]; rows with mask != 0 are overwritten with
 *               the top-k of the other ranks' round-1 candidates at or above
 *               tau16 plus the pushed lists (slot s owned by the s-th set
 *               bit of mask), in ascending flat order (round-1 region
 *               rank-major, then slot-major); other rows are untouched.
 * A row whose mask has more than (k-1)/n bits, or a bit at or above W, is
 * left unchanged and raises SATK_STATUS_SLOTS_EXCEEDED.
 * Errors      : SATK_EINVAL for NULL packed/logits/sat_word/recv/ids_out,
 *               W outside 1..16, T < 0, n or k not positive multiples of 32,
 *               n >= k, k > SATK_TOPK_MAX_K, ld_out < k, S < 0,
 *               ld_logits < S; SATK_EUNSUPPORTED when
 *               W * n + ((k-1)/n) * k exceeds SATK_MERGE_MAX_CANDIDATES.
 */
int satk_dcp_rescue_select(const int32_t *packed, int32_t W, int64_t T,
                           int32_t n, int32_t k, const uint16_t *logits_bf16,
                           int64_t S, int64_t ld_logits,
                           const int32_t *row_ends, const int32_t *sat_word,
                           int32_t *recv, int32_t *ids_out, int64_t ld_out,
                           int32_t *status, satk_stream_t stream);

/* Words of the rescue scratch: T * ((k-1)/n) * (k + k/32)
 * [P2 DCPTopkRescueWorkspace].  0 for invalid arguments. */
size_t satk_rescue_recv_words(int64_t T, int32_t n, int32_t k);

/* Scratch words available to satk_dcp_rescue_select_noalloc (8 MiB). */
#define SATK_RESCUE_NOALLOC_MAX_WORDS (2 * 1024 * 1024)

/*
 * satk_dcp_rescue_select_noalloc -- satk_dcp_rescue_select without the
 * `recv` argument, for callers that cannot allocate device memory (code
 * that only receives pointers to its inputs and outputs, or runs where
 * cudaMalloc may not be called).  The pages have no counterpart: it is a
 * convenience of this library.
 *
 * The pushed lists go to a fixed array inside the library's own device
 * memory, SATK_RESCUE_NOALLOC_MAX_WORDS int32 words on every GPU that loads
 * the library, kept until the process exits.  Nothing is allocated and no
 * allocating routine is called.  All other arguments, results, status bits
 * and errors are those of satk_dcp_rescue_select; in addition a call whose
 * satk_rescue_recv_words(T, n, k) exceeds SATK_RESCUE_NOALLOC_MAX_WORDS is
 * rejected with SATK_EUNSUPPORTED before anything is launched.
 *
 * - The first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current) and keeps it for the
 *   rest of the process; make that first call before any stream capture.
 *   A failed look-up returns SATK_ECUDA.  Resetting the device after that
 *   (cudaDeviceReset, or anything else that destroys its primary context)
 *   is not supported: the array moves when the library's module is loaded
 *   again, and the kept address would be stale.
 * - Every call on a device uses the same array and leaves its contents
 *   behind.  Nothing in it needs to start at zero: each slot a call reads
 *   is written by that same call first.  Calls that can run at the same
 *   time on the GPU (different streams without ordering) race on it.
 */
int satk_dcp_rescue_select_noalloc(const int32_t *packed, int32_t W, int64_t T,
                                   int32_t n, int32_t k,
                                   const uint16_t *logits_bf16, int64_t S,
                                   int64_t ld_logits, const int32_t *row_ends,
                                   const int32_t *sat_word, int32_t *ids_out,
                                   int64_t ld_out, int32_t *status,
                                   satk_stream_t stream);

/*
 * satk_dcp_emit_rows -- this rank's physical KV rows of the selected tokens
 * [P2 DCPTopkSelectKernel docstring (emit_rows), dcp_topk_merge_rows].
 *
 * ids         : int32 [T, ld_ids], columns [0, k): the selected global ids
 *               of each row (as written by satk_dcp_merge_select or
 *               satk_dcp_rescue_select; -1 entries are skipped).
 * W, dcp_rank : ranks, and this rank (0 <= dcp_rank < W).  A global id g
 *               belongs to rank g % W; its local index is l = g / W.
 * req_id      : int32 [T], the request of each row: its row of block_table.
 * block_table : int32 [table_rows, ld_block_table], physical block ids of
 *               each request; max_blocks (<= ld_block_table) is the table's
 *               width: a token in block b = l / block_size >= max_blocks is
 *               dropped.
 * stride_rows : physical rows per block id.  The row of token l is
 *               block_table[req_id[t], b] * stride_rows + l % block_size,
 *               stored as the low 32 bits (the page computes it in 32-bit
 *               integers).
 * rows_out    : int32 [T, ld_rows_out], ld_rows_out >= k: the rows of this
 *               rank's tokens in the order of their ids, then -1 up to k.
 *               Columns [k, ld_rows_out) are never written.
 * valid_out   : int32 [T], the number of rows emitted.
 * A req_id outside [0, table_rows) emits nothing for its row and raises
 * SATK_STATUS_BAD_REQUEST.
 * Errors      : SATK_EINVAL for NULL ids/req_id/block_table/rows_out/
 *               valid_out, T < 0, k < 1, ld_ids < k, W < 1, dcp_rank outside
 *               [0, W), table_rows < 0, max_blocks < 0,
 *               ld_block_table < max_blocks, block_size < 1,
 *               ld_rows_out < k, T >= 2**31.
 */
int satk_dcp_emit_rows(const int32_t *ids, int64_t T, int32_t k, int64_t ld_ids,
                       int32_t W, int32_t dcp_rank, const int32_t *req_id,
                       const int32_t *block_table, int64_t table_rows,
                       int64_t ld_block_table, int32_t max_blocks,
                       int32_t block_size, int64_t stride_rows,
                       int32_t *rows_out, int64_t ld_rows_out,
                       int32_t *valid_out, int32_t *status,
                       satk_stream_t stream);

/* Largest request count of satk_step_tables. */
#define SATK_TABLES_MAX_REQUESTS 8192
/* Largest latent width and rotated tail of the latent operators, the widest
 * query/key and value of one head of the expanded form, and the most ranks of
 * a merge. */
#define SATK_LATENT_MAX 512
#define SATK_LATENT_TAIL_MAX 64
#define SATK_EXPANDED_MAX_QK 256
#define SATK_EXPANDED_MAX_V 128
#define SATK_LATENT_MAX_RANKS 64

/*
 * The latent cache.  A cached token is one row of `dl` latent values followed
 * by `dr` rotated values, all 16-bit (`dtype` SATK_BF16 or SATK_F16); a key is
 * the whole row, a value its first dl columns.  Rows are addressed as
 * satk_dcp_emit_rows does it: token l of a request (its local index on this
 * rank) lives in row block_table[req][l / block_size] * stride_rows +
 * l % block_size.  The attention calls below share these rules:
 *  - softmax over the keys a token sees of scale * (query . key); sums and
 *    statistics in 32 bits, the weights rounded to `dtype` before the product
 *    with the values, the output rounded once;
 *  - a token that sees no key gets an output of zeros and an lse of -inf;
 *  - lse (nullable, float [T, H] contiguous) is the natural logarithm of the
 *    sum of exp(score), what satk_latent_merge takes;
 *  - what cache rows hold that a token does not see, infinities and NaN
 *    included, does not reach its output (rows near them may be read).  A
 *    non-finite key row that it does see may make its whole output row NaN,
 *    and so may a non-finite value row of the expanded form, whose lse goes
 *    by the keys alone.
 */

/*
 * satk_step_tables -- the metadata of one step from request lengths: extends
 * the block table and writes, per new token, what satk_topk_rows,
 * satk_dcp_emit_rows, satk_latent_store and satk_latent_attend take.
 *
 * context_lens, new_lens : int32 [R], tokens of each request before the step
 *               and new in it (global counts; negative counts as 0).  Global
 *               token p belongs to rank p % W as its local token p / W.
 * free_blocks : int32 [n_free], physical blocks, taken from the front in
 *               request order.
 * block_table : int32 [R, ld_block_table], extended in place: columns
 *               [ceil(local(context) / block_size), ceil(local(context + new)
 *               / block_size)) receive free blocks, others are not written.
 *               local(p) = tokens below p that dcp_rank holds.
 * T           : capacity of the per-token arrays.  New tokens come in request
 *               order, each request's in position order; entries past the
 *               last one get req_id 0, position 0, row_end 0, slot -1.
 * drafted     : 0: row_ends[t] = local(position + 1) (causal, the token
 *               itself included); 1: local(context) for every token of the
 *               request (tokens of a drafted tree, whose own visibility is a
 *               mask).
 * token_starts: int32 [R + 1], first token of each request and the total,
 *               each at most T.  lens: int32 [R], local tokens after the step.
 * req_id, positions, row_ends, slots : int32 [T].  slots: the physical row of
 *               a token this rank holds, else -1.
 * blocks_used : int32 [1], blocks taken from free_blocks.
 * Errors : SATK_EINVAL for a NULL pointer (free_blocks may be NULL when n_free
 *          is 0; lens/token arrays may not), R or T or n_free negative or
 *          >= 2**31, W < 1, dcp_rank outside [0, W), block_size < 1,
 *          stride_rows < 0, max_blocks < 0, ld_block_table < max_blocks,
 *          drafted not 0 or 1; SATK_EUNSUPPORTED for R >
 *          SATK_TABLES_MAX_REQUESTS.
 */
int satk_step_tables(const int32_t *context_lens, const int32_t *new_lens,
                     int32_t R, int32_t W, int32_t dcp_rank,
                     int32_t block_size, int64_t stride_rows,
                     const int32_t *free_blocks, int64_t n_free,
                     int32_t *block_table, int64_t ld_block_table,
                     int32_t max_blocks, int32_t drafted, int64_t T,
                     int32_t *token_starts, int32_t *lens, int32_t *req_id,
                     int32_t *positions, int32_t *row_ends, int32_t *slots,
                     int32_t *blocks_used, int32_t *status,
                     satk_stream_t stream);

/*
 * satk_latent_store -- writes new tokens into the latent cache: row slots[t]
 * receives [latent * rsqrt(mean(latent^2) + eps) * weight | rotated tail].
 *
 * latent  : [T, ld_latent] of `dtype`, dl columns; weight: nullable float [dl]
 *           (NULL: the latent is stored as it is, no norm).
 * tail    : [T, ld_tail] of `dtype`, dr columns (NULL when dr is 0);
 *           cos_sin: nullable float [n_positions, dr], dr/2 cosines then dr/2
 *           sines; positions: int32 [T] (NULL cos_sin: stored as it is).
 *           Pair i is columns (i, i + dr/2), or (2i, 2i + 1) when
 *           `interleaved`; (a, b) becomes (a cos - b sin, a sin + b cos).
 * slots   : int32 [T]; a negative slot skips the token, the others are
 *           distinct (as satk_step_tables gives them): tokens that share a
 *           slot are written at once, and the row may end up with parts of
 *           each.
 * cache   : [cache_rows, ld_cache] of `dtype`, ld_cache >= dl + dr; only
 *           columns [0, dl + dr) of the slots' rows are written.
 * Errors  : SATK_EINVAL for NULL latent/slots/cache, NULL tail with dr > 0,
 *           NULL positions with cos_sin, T or cache_rows or n_positions < 0,
 *           T >= 2**31, dl < 1, dr < 0, dr odd, ld_latent < dl, ld_tail < dr,
 *           ld_cache < dl + dr, a dtype other than SATK_BF16 / SATK_F16;
 *           SATK_EUNSUPPORTED for dl > SATK_LATENT_MAX or dr >
 *           SATK_LATENT_TAIL_MAX.
 */
int satk_latent_store(const void *latent, int64_t ld_latent, const void *tail,
                      int64_t ld_tail, int dtype, int64_t T, int32_t dl,
                      int32_t dr, const float *weight, float eps,
                      const float *cos_sin, int64_t n_positions,
                      const int32_t *positions, int32_t interleaved,
                      const int32_t *slots, void *cache, int64_t cache_rows,
                      int64_t ld_cache, int32_t *status, satk_stream_t stream);

/* Bytes of the workspace of satk_latent_attend and satk_latent_attend_rows
 * (the same for every call of these H and dl on the current device); 0 for
 * invalid arguments.  It need not be initialised, belongs to one call at a
 * time and holds nothing between calls. */
size_t satk_latent_workspace_bytes(int32_t H, int32_t dl);

/*
 * satk_latent_attend -- attention of query tokens over their requests' whole
 * caches (the absorbed form: every head reads the same latent rows).
 *
 * q        : [T, H, dl + dr] of `dtype`, token and head strides ld_q_t and
 *            ld_q_h, unit stride inside; already projected into the latent
 *            space.  Consecutive tokens with one req_id share their key reads,
 *            in groups of up to T / table_rows tokens (rounded up) and 64
 *            score columns: a table of the requests that have tokens, rather
 *            than of all slots, makes the largest groups.
 * cache    : [cache_rows, ld_cache] of `dtype`.
 * req_id   : int32 [T]; block_table [table_rows, ld_block_table], max_blocks,
 *            block_size, stride_rows: as in satk_dcp_emit_rows.
 * row_ends : int32 [T]; token t sees its request's local tokens
 *            [0, row_ends[t]) (clamped to the table's max_blocks * block_size).
 * tree     : nullable, int32 [T, tree_words]: it also sees local token
 *            row_ends[t] + b for each set bit b (bit b % 32 of word b / 32) --
 *            the drafted tokens on its path, itself among them.  With tokens
 *            spread over W ranks the bits count this rank's drafted tokens.
 * out      : [T, H, dl] of `dtype`, strides ld_out_t and ld_out_h.
 * A req_id outside the table, and a row outside [0, cache_rows), raise
 * SATK_STATUS_BAD_REQUEST / SATK_STATUS_BAD_ROW; what they name is not seen.
 * Errors   : SATK_EINVAL for NULL q/cache/req_id/block_table/row_ends/out/
 *            workspace, T < 0, T >= 2**31, H < 1, dl < 1, dr < 0, a stride
 *            below its extent (ld_q_t, ld_q_h, ld_cache, ld_block_table,
 *            ld_out_t, ld_out_h; token strides are not used at T = 1, head
 *            strides at H = 1), cache_rows < 0, table_rows < 0,
 *            max_blocks < 0, block_size < 1, tree_words < 1 with a tree, a
 *            scale that is not finite, workspace not 16-byte aligned or
 *            smaller than satk_latent_workspace_bytes, a dtype other than
 *            SATK_BF16 / SATK_F16; SATK_EUNSUPPORTED for H > 1024,
 *            dl > SATK_LATENT_MAX, dr > SATK_LATENT_TAIL_MAX or
 *            tree_words > 32.
 */
int satk_latent_attend(const void *q, int dtype, int64_t T, int32_t H,
                       int32_t dl, int32_t dr, int64_t ld_q_t, int64_t ld_q_h,
                       const void *cache, int64_t cache_rows, int64_t ld_cache,
                       const int32_t *req_id, const int32_t *block_table,
                       int64_t table_rows, int64_t ld_block_table,
                       int32_t max_blocks, int32_t block_size,
                       int64_t stride_rows, const int32_t *row_ends,
                       const int32_t *tree, int32_t tree_words, float scale,
                       void *out, int64_t ld_out_t, int64_t ld_out_h,
                       float *lse, void *workspace, size_t workspace_bytes,
                       int32_t *status, satk_stream_t stream);

/*
 * satk_latent_attend_rows -- the same attention over each token's selected
 * cache rows, as satk_dcp_emit_rows writes them.
 *
 * rows   : int32 [T, ld_rows], columns [0, k): physical rows; a negative entry
 *          is skipped, a row named twice counts twice.
 * counts : nullable int32 [T] (the valid_out of satk_dcp_emit_rows): only the
 *          first clamp(counts[t], 0, k) entries are read.
 * All other arguments, results and errors as in satk_latent_attend; also
 * SATK_EINVAL for NULL rows, k < 1 or ld_rows < k.
 */
int satk_latent_attend_rows(const void *q, int dtype, int64_t T, int32_t H,
                            int32_t dl, int32_t dr, int64_t ld_q_t,
                            int64_t ld_q_h, const void *cache,
                            int64_t cache_rows, int64_t ld_cache,
                            const int32_t *rows, int64_t ld_rows, int32_t k,
                            const int32_t *counts, float scale, void *out,
                            int64_t ld_out_t, int64_t ld_out_h, float *lse,
                            void *workspace, size_t workspace_bytes,
                            int32_t *status, satk_stream_t stream);

/*
 * satk_latent_attend_expanded -- prompt attention with the latent expanded to
 * keys and values per head (the rotated tail of a key stays shared by the
 * heads), over ragged requests.
 *
 * q    : [T, H, dn + dr] of `dtype`, strides ld_q_t, ld_q_h.
 * k    : [S, H, dn], strides ld_k_s, ld_k_h; tail: [S, ld_tail], dr columns
 *        (NULL when dr is 0); v: [S, H, dv], strides ld_v_s, ld_v_h.
 * token_starts, key_starts : int32 [R + 1], ascending: request r owns tokens
 *        [token_starts[r], token_starts[r+1]) and keys [key_starts[r],
 *        key_starts[r+1]).  Tokens outside every request get empty rows.
 * row_ends : int32 [T]; token t sees its request's first row_ends[t] keys
 *        (clamped to the request's keys).
 * out  : [T, H, dv] of `dtype`, strides ld_out_t, ld_out_h.
 * Errors : SATK_EINVAL for NULL q/k/v/token_starts/key_starts/row_ends/out,
 *        NULL tail with dr > 0, T or S or R < 0 or >= 2**31, H < 1, dn < 1,
 *        dr < 0, dv < 1, a stride below its extent, a scale that is not
 *        finite, a dtype other than SATK_BF16 / SATK_F16; SATK_EUNSUPPORTED
 *        for H > 1024, dn + dr > SATK_EXPANDED_MAX_QK, dv >
 *        SATK_EXPANDED_MAX_V.
 */
int satk_latent_attend_expanded(const void *q, int dtype, int64_t T, int32_t H,
                                int32_t dn, int32_t dr, int64_t ld_q_t,
                                int64_t ld_q_h, const void *k, int64_t S,
                                int64_t ld_k_s, int64_t ld_k_h,
                                const void *tail, int64_t ld_tail,
                                const void *v, int32_t dv, int64_t ld_v_s,
                                int64_t ld_v_h, const int32_t *token_starts,
                                const int32_t *key_starts, int32_t R,
                                const int32_t *row_ends, float scale,
                                void *out, int64_t ld_out_t, int64_t ld_out_h,
                                float *lse, satk_stream_t stream);

/*
 * satk_latent_merge -- joins W partial attention results over disjoint keys
 * (the ranks of a decode, or a prompt chunk and its context):
 * lse_out = log sum_w exp(lse_w), out = sum_w exp(lse_w - lse_out) parts_w.
 *
 * parts : [W, T, H, dv] of `dtype`, strides ld_w, ld_t, ld_h, unit inside.
 * lse   : float [W, T, H] contiguous.  What a part with lse -inf
 *         holds does not count, whatever it is.
 * out   : [T, H, dv] of `dtype`, strides ld_out_t, ld_out_h; lse_out: nullable
 *         float [T, H].  All parts empty: zeros and -inf.
 * Errors: SATK_EINVAL for NULL parts/lse/out, W < 1, T < 0, T * H >= 2**31,
 *         H < 1, dv < 1, a stride below its extent, a dtype other than
 *         SATK_BF16 / SATK_F16; SATK_EUNSUPPORTED for W >
 *         SATK_LATENT_MAX_RANKS.
 */
int satk_latent_merge(const void *parts, int dtype, int32_t W, int64_t T,
                      int32_t H, int32_t dv, int64_t ld_w, int64_t ld_t,
                      int64_t ld_h, const float *lse, void *out,
                      int64_t ld_out_t, int64_t ld_out_h, float *lse_out,
                      satk_stream_t stream);

/*
 * satk_debug_flags -- the bounds-check bits of the debug build.  A library
 * built with -DSATK_DEBUG (libsatk_debug.so) checks, inside its selection
 * kernels (the latent-cache ones test what they are given in every build),
 * every shared-memory list index, output position, histogram bin and
 * scratch index that the code relies on an invariant for; a failed check
 * skips the access and ORs a bit into a device word (1 list index, 2 output
 * position, 4 histogram bin, 8 scratch or plane-word index) instead of
 * trapping.  This call waits for the device, returns the word and, when
 * `clear` is non-zero, zeroes it; 0xffffffff if the device could not be
 * read.  With `clear` = 2 it leaves 256 there instead of 0: until the next
 * clearing, each CTA of satk_latent_attend and satk_latent_attend_rows treats
 * the last of its results as if a wait inside the GPU had been given up
 * (SATK_STATUS_STALLED).  The normal build checks nothing and returns 0.  Not part of the
 * pages' interface: a test aid of this library.
 */
uint32_t satk_debug_flags(int clear);

/* A static, human-readable string for an SATK_* return code. */
const char *satk_status_string(int rc);

/* Short names, the same functions. */
int topk_rows(const void *logits, int dtype, int64_t rows, int64_t cols,
              int64_t ld_logits, const int32_t *row_ends, int32_t k,
              int32_t *out, int64_t ld_out, satk_stream_t stream);
int topk_rows_sorted(const void *logits, int dtype, int64_t rows,
                     int64_t cols, int64_t ld_logits, const int32_t *row_ends,
                     int32_t k, int32_t *out, int64_t ld_out,
                     satk_stream_t stream);
int dcp_pack(const uint16_t *logits_bf16, int64_t rows, int64_t S,
             int64_t ld_logits, const int32_t *local_idx, int64_t ld_idx,
             int32_t n, const int32_t *row_ends, int32_t *packed,
             satk_stream_t stream);
int dcp_topk_pack(const uint16_t *logits_bf16, int64_t rows, int64_t S,
                  int64_t ld_logits, const int32_t *row_ends, int32_t n,
                  int32_t *packed, satk_stream_t stream);
int dcp_merge_select(const void *cand, int format, int32_t W, int64_t T,
                     int32_t n, int32_t k, int32_t *ids_out, int64_t ld_out,
                     int32_t *sat_word, int32_t *status, satk_stream_t stream);
int dcp_rescue_select(const int32_t *packed, int32_t W, int64_t T, int32_t n,
                      int32_t k, const uint16_t *logits_bf16, int64_t S,
                      int64_t ld_logits, const int32_t *row_ends,
                      const int32_t *sat_word, int32_t *recv,
                      int32_t *ids_out, int64_t ld_out, int32_t *status,
                      satk_stream_t stream);
int dcp_emit_rows(const int32_t *ids, int64_t T, int32_t k, int64_t ld_ids,
                  int32_t W, int32_t dcp_rank, const int32_t *req_id,
                  const int32_t *block_table, int64_t table_rows,
                  int64_t ld_block_table, int32_t max_blocks,
                  int32_t block_size, int64_t stride_rows, int32_t *rows_out,
                  int64_t ld_rows_out, int32_t *valid_out, int32_t *status,
                  satk_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SATK_H_ */
