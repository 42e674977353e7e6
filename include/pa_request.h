/*
 * pa_request.h -- the calls a serving loop makes for whole requests over the
 * paged cache of pa.h, in the same library (libpa.so) and with the same
 * conventions as pa_serving.h: device pointers owned by the caller,
 * asynchronous on `stream`, argument errors returned before anything is
 * launched, index errors that only the device can see skipped and reported by
 * pa_get_status, nothing allocated, nothing kept from one call for the next.
 * All of them may be captured into a CUDA graph.  The tensors of a call must be
 * on the device that is current.
 *
 *   pa_prefill, pa_prefill_fp8
 *       the attention of prompts and their chunks: any number of query tokens
 *       per sequence, over 16-bit and E4M3 pools;
 *   pa_alloc_pages, pa_free_pages, pa_fork_pages, pa_compact_pages
 *       the pool's pages by reference counts: taken, given back, shared by
 *       forks, moved together;
 *   pa_process_logits
 *       penalties, biases and grammar masks on logits, and the probabilities
 *       that pa_verify_drafts draws from.
 */
#ifndef PA_REQUEST_H
#define PA_REQUEST_H

#include "pa_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Another bit of the device status word (PA_ERR_BOUNDS). */
#define PA_STATUS_BAD_ROW 128u   /* a row outside the tables, or forked onto itself */

/*
 * Attention of prompts.  Sequence b has the n_b = query_starts[b + 1] -
 * query_starts[b] query tokens q[query_starts[b]] .. , its last ones: query i
 * sits at position L - n_b + i (L = context_lens[b], whose keys and values are in
 * the cache already, the queries' own among them) and attends causally, as
 * pa_decode's queries_per_seq do, but any number of them, another one for each
 * sequence (0: none; 1: a decode step):
 *   out[t][hq][:] = sum_j softmax_j(scale * q[t][hq] . K_j) * V_j
 * over positions j up to its own, within the last window_size of them when that is
 * not 0.  Scores, sums and statistics are fp32; the weights enter the products with V
 * in 16 bits, bf16 for bf16 pools (each off by 2^-8 of itself at most), else fp16
 * (2^-11; weights, over E4M3 pools times V's scales, below 2^-20 of the largest lose
 * bits, and below 2^-31 they count as 0);
 * the result is rounded to dtype.  Weights are divided by their sum last: values of
 * bf16 pools above 2^88 in magnitude may overflow.  A query before position 0 gets
 * zeros, as does one that sees no page with a valid id, and so do the queries of a
 * sequence whose context_len is out of bounds (PA_STATUS_BAD_LEN).  Pages of a
 * sequence before the windows of all its queries are not looked at: their table
 * entries may be anything.  Tokens that belong to no sequence (before
 * query_starts[0], from query_starts[num_seqs] on) are left as they were.  Starts
 * that decrease or leave [0, num_tokens] set PA_STATUS_BAD_LEN and their sequence's
 * queries are left as they were.
 *   q: num_q_heads x head_dim dense elements a token, q_stride elements from one
 *   token to the next (a multiple of 8: a view of one projection's output);
 *   out: [num_tokens][num_q_heads][head_dim]; query_starts: int32
 *   [num_seqs + 1]; num_q_heads / num_kv_heads 1..32; head_dim 64 or 128;
 *   block_size 16; num_tokens * num_q_heads at most 2^30; max_context_len at most
 *   2^30; num_seqs at most 65535; num_blocks * num_kv_heads of a 16-bit pool below
 *   2^31; scale finite; out must not overlap q.
 *   workspace: pa_prefill_workspace_size bytes, 256-byte aligned, of any
 *   contents (its size goes by the current device's SMs and head_dim: one serves all
 *   calls); calls that share one must not overlap on the device.
 * Every wait of the kernel is bounded by 2 s: one that runs out sets
 * PA_STATUS_TIMEOUT, and the outputs are not to be used.
 * Results do not depend on the order of execution.
 */
size_t pa_prefill_workspace_size(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                                 int head_dim);
int pa_prefill(void *out, const void *q, int64_t q_stride, const void *k_cache,
               const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
               const int32_t *context_lens, int max_context_len, const int32_t *query_starts,
               int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
               int block_size, int num_blocks, float scale, int window_size, int dtype,
               void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same over E4M3 pools: K_j = e4m3(code) * k_scale[block][kv head], V_j
 * likewise (scales finite and not negative, as the appends and quantisers
 * make them).  bf16 queries enter the products in fp16, each row scaled by a power of
 * two: exactly, down to 2^-28 of the row's largest element.
 */
int pa_prefill_fp8(void *out, const void *q, int64_t q_stride, const uint8_t *k_cache,
                   const uint8_t *v_cache, const float *k_scale, const float *v_scale,
                   const int32_t *block_tables, int max_blocks_per_seq,
                   const int32_t *context_lens, int max_context_len, const int32_t *query_starts,
                   int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                   int block_size, int num_blocks, float scale, int window_size, int dtype,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * The pool's pages.  ref_counts int32 [num_blocks] says how many rows hold each
 * page; one with 0 (or less) is free.  block_tables int32 [num_rows][max_blocks_per_seq]
 * holds each row's pages, num_pages int32 [num_rows] how many there are.  These
 * three are the whole state, on the device; the calls keep it, in the order of
 * the stream, without a host round trip.  Items (rows, pairs) are served in
 * their order and the lowest free page is always taken first, so results do not
 * depend on the order of execution.  An item's row outside [0, num_rows) sets
 * PA_STATUS_BAD_ROW and the item is passed over; a num_pages outside [0,
 * max_blocks_per_seq] sets PA_STATUS_BAD_LEN, likewise.  num_blocks at most 2^30;
 * num_items at most 32768 where granted is written, else 2^24; ref_counts
 * 16-byte aligned.  These calls write tables, lengths and pages: a decode that
 * follows one of them with nothing else between on the stream must not be one with
 * PA_DECODE_EARLY_PROLOGUE or PA_DECODE_EARLY_COPIES.
 *
 * pa_alloc_pages: rows[i] gets pages until it holds ceil(new_lens[i] / 16)
 * (one that holds as many keeps what it has), from the lowest free ones on, with
 * a count of 1.  granted[i] is 1, or 0 once the pool does not hold enough for an
 * item: it and those behind it get nothing.  An item passed over (its new_len
 * negative or beyond its table: PA_STATUS_BAD_LEN) gets 0 and takes nothing.
 * Rows must be distinct.
 */
int pa_alloc_pages(int32_t *block_tables, int max_blocks_per_seq, int32_t *num_pages,
                   int num_rows, const int32_t *rows, const int32_t *new_lens, int num_items,
                   int32_t *ref_counts, int num_blocks, int block_size, int32_t *granted,
                   void *stream);

/*
 * pa_free_pages: the pages of each row lose one owner, its table entries become
 * -1 and its num_pages 0 (a row listed twice is freed once).  An entry outside
 * [0, num_blocks), or of a page that is free, sets PA_STATUS_BAD_BLOCK and
 * changes no count.
 */
int pa_free_pages(int32_t *block_tables, int max_blocks_per_seq, int32_t *num_pages, int num_rows,
                  const int32_t *rows, int num_items, int32_t *ref_counts, int num_blocks,
                  void *stream);

/*
 * pa_fork_pages: row dst_rows[i] becomes a fork of row src_rows[i] (beam search,
 * parallel sampling): it shares src's full pages (their counts grow by one),
 * gets a page of its own with a copy of src's last page when that is part full
 * (all 16 rows of it, and in an E4M3 pool its scales), and src's context_len.
 * Pages that src holds beyond its context_len are not shared.  What dst held
 * before is overwritten, not freed: free it first.  granted as in
 * pa_alloc_pages (a fork whose last page is full needs none); a dst that is not
 * granted stays as it was.  context_lens int32 [num_rows]; one that is negative
 * or above what src holds passes the pair over (PA_STATUS_BAD_LEN), as does a
 * src that is its own dst (PA_STATUS_BAD_ROW).  An entry of src outside the pool
 * sets PA_STATUS_BAD_BLOCK, counts and copies nothing: that of a full page is taken
 * over as it is; where it is the part-full last one, dst gets a page of its own whose
 * contents stay as they were.
 * Destinations must be distinct and not the source of another pair; a source may
 * be forked many times.
 *   pool_type: PA_F16 / PA_BF16 (scales NULL) or PA_E4M3.
 */
int pa_fork_pages(void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                  int32_t *block_tables, int max_blocks_per_seq, int32_t *num_pages,
                  int32_t *context_lens, int num_rows, const int32_t *src_rows,
                  const int32_t *dst_rows, int num_items, int32_t *ref_counts, int num_blocks,
                  int num_kv_heads, int head_dim, int block_size, int pool_type,
                  int32_t *granted, void *stream);

/*
 * pa_compact_pages: the live pages (count > 0) are moved together at the front
 * of the pool: with n of them, those at n and above move, in order, to the free
 * pages below n, in order; the rest stay.  Their contents (and scales) are
 * copied; the pages they left keep theirs.
 *   num_live[0] = n;
 *   moved_to[p] = where page p is now (p when it stayed, -1 when it was free);
 *   ref_counts_out = the counts afterwards; tables_out = the tables with the new
 *   ids (entries behind num_pages as they were).  An entry that is outside the
 *   pool or free sets PA_STATUS_BAD_BLOCK; it is kept, or becomes -1.
 * ref_counts_out may be ref_counts and tables_out block_tables (in place); no
 * other overlap.  workspace: pa_compact_workspace_size bytes, 256-byte aligned,
 * of any contents.
 */
size_t pa_compact_workspace_size(int num_blocks);
int pa_compact_pages(void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                     const int32_t *block_tables, int max_blocks_per_seq,
                     const int32_t *num_pages, int num_rows, const int32_t *ref_counts,
                     int num_blocks, int num_kv_heads, int head_dim, int block_size,
                     int pool_type, int32_t *tables_out, int32_t *ref_counts_out,
                     int32_t *moved_to, int32_t *num_live, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * The adjustment of logits.  For row i (0 <= i < rows_per_seq) of sequence b and
 * token t, in fp32, in this order, each step where its pointer is not NULL:
 *   x = logits[b][i][t];
 *   t occurs in the history, or among the first i of draft_tokens[b]:
 *     x = x > 0 ? x / repetition[b] : x * repetition[b];
 *   it occurs c > 0 times among the output, which is the history from
 *     prompt_lens[b] on and those drafts: x -= frequency[b] * c + presence[b];
 *   x += the sum of the bias_values[b][j] with bias_tokens[b][j] == t, in order;
 *   bit t % 32 of allowed[b][i][t / 32] clear: x = -inf.
 * as_probs 0: x, rounded to dtype, into out [..][vocab_size] of dtype (which may
 * be the logits themselves).  as_probs 1: softmax(x / temperature[b]) in fp32, as
 * pa_verify_drafts takes it; where temperature[b] is not above 0, 1 at the
 * largest x (of equal ones the lowest token) and 0 elsewhere.  There, a NaN
 * counts as -inf, a row of -inf gives zeros, and tokens at +inf share the row.
 *   history int32 [num_seqs][history_stride], its first history_lens[b] entries
 *   (prompt first, then output); prompt_lens NULL: all of it is output; a length
 *   outside [0, history_stride] sets PA_STATUS_BAD_LEN and that history counts as
 *   empty (a prompt_len beyond its history as all of it).  Negative tokens in
 *   history, drafts and biases are padding; those from vocab_size on set
 *   PA_STATUS_BAD_TOKEN and count as padding.
 *   draft_tokens int32 [num_seqs][rows_per_seq - 1]; bias_tokens int32 and
 *   bias_values fp32 [num_seqs][num_bias], num_bias at most 1024; allowed
 *   uint32, allowed_stride words from row to row (at least ceil(vocab_size /
 *   32)); repetition (above 0), frequency, presence, temperature fp32
 *   [num_seqs].  All of them device pointers, 4-byte aligned; NULL for none
 *   (temperature NULL: 1).  The struct itself is host memory, read during the
 *   call.  logits_stride and out_stride: elements from row to row, at least
 *   vocab_size; rows follow one another evenly, rows_per_seq (1..1025) for each
 *   sequence.  dtype PA_F32, PA_F16 or PA_BF16; logits and out 16-byte aligned;
 *   vocab_size at most 2^19; num_seqs * rows_per_seq at most 2^24.
 */
typedef struct pa_logits_spec {
    const int32_t *history;
    const int32_t *history_lens;
    const int32_t *prompt_lens;
    const int32_t *draft_tokens;
    const float *repetition;
    const float *presence;
    const float *frequency;
    const float *temperature;
    const int32_t *bias_tokens;
    const float *bias_values;
    const uint32_t *allowed;
    int64_t history_stride;
    int64_t allowed_stride;
    int num_bias;
} pa_logits_spec;

int pa_process_logits(void *out, int64_t out_stride, const void *logits, int64_t logits_stride,
                      const pa_logits_spec *spec, int num_seqs, int rows_per_seq, int vocab_size,
                      int dtype, int as_probs, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_REQUEST_H */
