/*
 * pa_serving.h -- the calls a serving loop makes around the decode step of
 * pa.h, in the same library (libpa.so) and with the same conventions: device
 * pointers owned by the caller, asynchronous on `stream`, argument errors
 * returned before anything is launched, index errors that only the device can
 * see skipped and reported by pa_get_status, nothing allocated, nothing kept
 * from one call for the next.  All of them may be captured into a CUDA graph.
 *
 *   pa_rope, pa_rope_append, pa_rope_append_fp8
 *       rotary positions of one to four axes (text; time, height and width of
 *       images and video) for q and k, and the append of the rotated k and of
 *       v into the paged pools in the same launch;
 *   pa_attention_weights, pa_attention_weights_fp8
 *       the attention weight each cached token receives, accumulated over
 *       query tokens and steps;
 *   pa_evict, pa_evict_fp8
 *       the cut of a cache to a budget by that weight: the heaviest tokens of
 *       each (sequence, kv head), moved into spare blocks;
 *   pa_verify_drafts
 *       speculative decoding's verification of drafted tokens against the
 *       target's probabilities, from given random numbers.
 *
 * The tensors of a call must be on the device that is current.
 */
#ifndef PA_SERVING_H
#define PA_SERVING_H

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of pa_verify_drafts' probabilities, besides PA_F16 and PA_BF16. */
enum { PA_F32 = 3 };

/* Another bit of the device status word (PA_ERR_BOUNDS). */
#define PA_STATUS_BAD_TOKEN 64u   /* a drafted token outside [0, vocab_size) */

/*
 * The rotation.  Pair i (0 <= i < rotary_dim / 2) of a head's first rotary_dim
 * elements turns by the angle positions[freq_axis[i]][token] * inv_freq[i]:
 *   (x, y) -> (x cos - y sin, y cos + x sin),
 * cos and sin multiplied by `amplitude` (1 unless a long-context scaling asks
 * for more); elements behind rotary_dim pass through.  The pair is
 * (i, i + rotary_dim / 2) when adjacent is 0, and (2i, 2i + 1) when it is 1.
 * Angles are reduced in 64-bit fractions of a turn: inv_freq's to 2^-63 of a turn
 * (for |inv_freq| up to 2^40), its product with the position exactly, so far
 * positions lose nothing; the rotation is made in fp32 and rounded once.
 *   inv_freq: HOST, radians per position, finite; freq_axis: HOST, the axis of
 *   each pair, in [0, num_axes), or NULL when num_axes is 1.  Both are read
 *   during the call.  num_axes 1..4; rotary_dim a multiple of 16 in
 *   [16, head_dim].
 */
typedef struct pa_rope_spec {
    const double *inv_freq;
    const int32_t *freq_axis;
    int num_axes;
    int rotary_dim;
    int adjacent;
    float amplitude;
} pa_rope_spec;

/*
 * Rotates q into q_out [num_tokens][num_q_heads][head_dim] and k into k_out
 * [num_tokens][num_kv_heads][head_dim].  q and k hold num_*_heads x head_dim
 * dense elements a token, q_stride / k_stride elements from one token to the
 * next (so they may be views of one projection's output).  In place when q_out
 * == q (k_out == k) and the input is dense; any other overlap is undefined.
 * num_q_heads or num_kv_heads 0 leaves that side out (its pointers unused).
 *   positions: int32 [num_axes][num_tokens], any value (negative ones turn the
 *   other way); head_dim a multiple of 8, at most 256; strides multiples of 8;
 *   num_q_heads + 2 num_kv_heads at most 65535; dtype PA_F16 or PA_BF16.
 */
int pa_rope(void *q_out, const void *q, int64_t q_stride, void *k_out, const void *k,
            int64_t k_stride, const int32_t *positions, const pa_rope_spec *spec, int num_tokens,
            int num_q_heads, int num_kv_heads, int head_dim, int dtype, void *stream);

/*
 * pa_rope followed by pa_cache_append in one launch: q rotated into q_out, k
 * rotated into k_cache and v copied into v_cache at slot_mapping (as
 * pa_cache_append; a negative slot appends nothing, its q is rotated all the
 * same).  Two tokens with the same slot race.
 */
int pa_rope_append(void *q_out, const void *q, int64_t q_stride, const void *k_new,
                   int64_t k_stride, const void *v_new, int64_t v_stride, void *k_cache,
                   void *v_cache, const int64_t *slot_mapping, const int32_t *positions,
                   const pa_rope_spec *spec, int num_tokens, int num_q_heads, int num_kv_heads,
                   int head_dim, int block_size, int num_blocks, int dtype, void *stream);

/*
 * pa_rope followed by pa_cache_append_fp8 in one launch: k is rotated, rounded
 * to dtype and encoded with its page's scale, v encoded, as that call does,
 * bit for bit.  head_dim 64 or 128.  Tokens of the same page race: give them
 * in separate calls.
 */
int pa_rope_append_fp8(void *q_out, const void *q, int64_t q_stride, const void *k_new,
                       int64_t k_stride, const void *v_new, int64_t v_stride, uint8_t *k_cache,
                       uint8_t *v_cache, float *k_scale, float *v_scale,
                       const int64_t *slot_mapping, const int32_t *positions,
                       const pa_rope_spec *spec, int num_tokens, int num_q_heads,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks, int dtype,
                       void *stream);

/*
 * Accumulated attention weights.  For every sequence b, kv head h and token t
 * in [0, context_lens[b]):
 *   weights[b][h][t] = old(t) + sum over the n_q query tokens i and the q heads
 *                      g of h's group of softmax_t(scale * q[b][i][g] . K_t)
 * with old(t) = decay * weights[b][h][t], or 0 for the last fresh_tokens tokens
 * (those appended since the last call, whose entry still holds what a former
 * token left there).  decay 0 reads no old weight.  Query i sits at position
 * L - n_q + i and attends positions up to its own, as in pa_decode without a
 * window (there is no window here: the weights are those of the whole context,
 * and all of its blocks have to be in the table); one before position 0 adds
 * nothing, nor does one whose logits are all -inf.  Entries behind the context stay
 * as they are.
 *   weights: fp32 [num_seqs][num_kv_heads][weights_stride], weights_stride >=
 *   max_context_len; a row belongs to its sequence, so sequences that share
 *   blocks keep weights of their own.
 *   q: [num_seqs][n_q][num_q_heads][head_dim]; queries_per_seq n_q 1..1024: up
 *   to 32 query rows (n_q x group) take one pass over K, more take several.
 *   workspace: pa_attention_weights_workspace_size bytes, 256-byte aligned,
 *   zero-filled by the caller once before its first use; it then serves call
 *   after call, whatever their sizes.  After a status with PA_STATUS_TIMEOUT or
 *   PA_STATUS_WS_DIRTY (it held what no call leaves; results may be wrong)
 *   zero-fill it again.  Calls that share one must not overlap on the device.
 *   Its size goes by the bounds: 512 bytes for every 16 tokens of max_context_len
 *   of each (sequence, kv head) with up to 8 query rows a pass, twice that with up
 *   to 16, four times with more (of at most 512 sequences).
 * One launch per pass and 512 sequences.  With max_context_len above 4096 it is
 * a cooperative one, whose warps wait, bounded by 2 s, for one another's softmax
 * statistics; only these can set PA_STATUS_TIMEOUT or PA_STATUS_WS_DIRTY.  Its
 * grid is sized for all SMs of the device: in a context limited to some of them
 * it may be refused (PA_ERR_CUDA).  The launch is chosen by max_context_len, not by
 * the lengths, so a tight bound makes short contexts faster.
 * max_context_len at most 2^30.
 * Results do not depend on the order of execution.
 */
size_t pa_attention_weights_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                           int max_context_len, int queries_per_seq);
int pa_attention_weights(float *weights, int64_t weights_stride, const void *q,
                         const void *k_cache, const int32_t *block_tables, int max_blocks_per_seq,
                         const int32_t *context_lens, int max_context_len, int num_seqs,
                         int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, float scale, float decay, int fresh_tokens,
                         int queries_per_seq, int dtype, void *workspace, size_t workspace_bytes,
                         void *stream);

/* The same over an E4M3 pool: K_t = e4m3(code) * k_scale[block][kv head]. */
int pa_attention_weights_fp8(float *weights, int64_t weights_stride, const void *q,
                             const uint8_t *k_cache, const float *k_scale,
                             const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, int max_context_len, int num_seqs,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int num_blocks, float scale, float decay, int fresh_tokens,
                             int queries_per_seq, int dtype, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * Eviction.  Each sequence with more than `keep` tokens is cut to `keep`, for
 * every kv head on its own: its first first_tokens tokens, its last
 * recent_tokens tokens, and of those between them the keep - first_tokens -
 * recent_tokens with the largest weights (of equal weights the lowest index; a
 * NaN counts as the lowest weight).  The kept tokens' K and V rows are moved,
 * in order, into the first ceil(keep / 16) blocks of the sequence's row of
 * spare_tables; the source blocks stay as they are (they may be shared with
 * other sequences) and are the caller's to free.  Rows behind the keep-th of
 * the last block stay as they are.  A spare block must not be a block that
 * this call reads or another one's spare block.  Shorter sequences move
 * nothing.  For every sequence, evicted or not:
 *   new_lens[b]          its length afterwards, min(context_lens[b], keep);
 *   kept[b][h][j]        the token now at position j, for j < new_lens[b]
 *                        (entries behind are left as they were);
 *   weights_out[b][h][j] that token's weight (likewise; NULL: not wanted);
 *   tables_out[b]        its block table afterwards: the row of spare_tables,
 *                        or, when nothing was moved, the first
 *                        spare_blocks_per_seq entries of its row of
 *                        block_tables (-1 behind them; NULL: not wanted).
 * weights [num_seqs][num_kv_heads][weights_stride] as pa_attention_weights
 * leaves them; weights_out [num_seqs][num_kv_heads][weights_out_stride] must
 * not overlap weights, and weights_out_stride >= keep; kept int32
 * [num_seqs][num_kv_heads][keep]; spare_tables and tables_out int32
 * [num_seqs][spare_blocks_per_seq], spare_blocks_per_seq >= ceil(keep / 16),
 * and not overlapping block_tables; new_lens must not be context_lens.
 * Keys keep the rotation of the position they were written at.
 * max_context_len at most 2^30.  The next pa_decode or pa_decode_step over the
 * moved blocks must not be one with PA_DECODE_EARLY_COPIES, nor with
 * PA_DECODE_EARLY_PROLOGUE when it reads tables_out or new_lens.
 */
int pa_evict(void *k_cache, void *v_cache, const float *weights, int64_t weights_stride,
             float *weights_out, int64_t weights_out_stride, const int32_t *block_tables,
             int max_blocks_per_seq, const int32_t *context_lens, int max_context_len,
             const int32_t *spare_tables, int spare_blocks_per_seq, int32_t *tables_out,
             int32_t *new_lens, int32_t *kept, int num_seqs, int num_kv_heads, int head_dim,
             int block_size, int num_blocks, int keep, int first_tokens, int recent_tokens,
             int dtype, void *stream);

/*
 * The same over E4M3 pools.  A page that is written gets the scale of the rows
 * it now holds: with x = fl32(e4m3(code) * source page's scale), scale = amax
 * |x| / 448 (1 when amax is 0) and code = E4M3(fl32(x / scale)), as
 * pa_quantize_fp8 does.
 */
int pa_evict_fp8(uint8_t *k_cache, uint8_t *v_cache, float *k_scale, float *v_scale,
                 const float *weights, int64_t weights_stride, float *weights_out,
                 int64_t weights_out_stride, const int32_t *block_tables, int max_blocks_per_seq,
                 const int32_t *context_lens, int max_context_len, const int32_t *spare_tables,
                 int spare_blocks_per_seq, int32_t *tables_out, int32_t *new_lens, int32_t *kept,
                 int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                 int keep, int first_tokens, int recent_tokens, void *stream);

/*
 * Verification of drafted tokens.  For sequence b with n_b = num_drafts[b]
 * drafts x_i, target distributions p_i (i <= n_b) and draft distributions q_i:
 *   drafts are accepted in order while uniforms[b][i] * q_i(x_i) < p_i(x_i)
 *   (the product not rounded); with r the number accepted, one more token is
 *   drawn with u = uniforms[b][max_drafts]: from max(p_r - q_r, 0) when r < n_b
 *   (from p_r if that is zero everywhere), from p_r when r = n_b; the lowest
 *   token whose cumulative sum exceeds u times the total.
 *   num_accepted[b] = r; out_tokens[b] = x_0 .. x_{r-1}, the drawn token, then
 *   -1 up to max_drafts + 1 entries.
 * The tokens drawn follow the distribution p whatever the drafts were.
 *   target_probs [num_seqs][max_drafts + 1] rows of vocab_size values,
 *   target_stride elements from row to row; draft_probs [num_seqs][max_drafts]
 *   rows likewise, or NULL for drafts without probabilities (q_i is then 1 at
 *   x_i and 0 elsewhere); both of dtype PA_F32, PA_F16 or PA_BF16.  Rows need
 *   not add up to exactly 1 (to at most 4); negative values and NaN count as 0,
 *   values above 2 as 2.  draft_tokens int32 [num_seqs][max_drafts]; num_drafts
 *   int32 [num_seqs], or NULL when all have max_drafts; uniforms fp32
 *   [num_seqs][max_drafts + 1] in [0, 1).  max_drafts 0..1024 (0: a plain draw);
 *   vocab_size and num_seqs at most 2^24.
 * Sums are 64-bit fixed-point numbers (2^-60), so a result does not depend on
 * the order of summation.  A row of zeros draws -1.  A draft outside
 * [0, vocab_size) is rejected and sets PA_STATUS_BAD_TOKEN; a num_drafts
 * outside [0, max_drafts] sets PA_STATUS_BAD_LEN and its sequence gets 0 and
 * -1s.
 */
int pa_verify_drafts(int32_t *out_tokens, int32_t *num_accepted, const void *target_probs,
                     int64_t target_stride, const void *draft_probs, int64_t draft_stride,
                     const int32_t *draft_tokens, const int32_t *num_drafts,
                     const float *uniforms, int num_seqs, int max_drafts, int vocab_size,
                     int dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_SERVING_H */
