/*
 * pa_serving_test.h -- the failure-path test of the wait in pa_serving.h, as the
 * two of pa.h are for its own: it makes the wait run out on purpose, with a
 * short limit, so that a test can check the status, that nothing wrong is
 * written and that the context and the workspace stay usable.  It neither
 * faults, traps nor spins without bound.
 */
#ifndef PA_SERVING_TEST_H
#define PA_SERVING_TEST_H

#include "pa_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pa_attention_weights (one query token, decay 0, no fresh tokens, block size
 * 16) in its cooperative launch (max_context_len above 4096, else
 * PA_ERR_UNSUPPORTED; at most 512 sequences), in which warp `silent_warp` of
 * the launch (>= 0; one behind the last that has pages changes nothing) does
 * not announce the softmax statistics of its pages: the warps that wait for
 * them give up after limit_ns (1 .. 2e9), set PA_STATUS_TIMEOUT and write no
 * weights of the (sequence, kv head) they wait for, nor of those that they
 * would have come to after it; a CTA does so for all of its pages when the
 * (sequence, kv head) at its first or its last page is one of more than 16
 * parts.  All other weights are written as ever.
 */
int pa_test_weights_timeout(float *weights, int64_t weights_stride, const void *q,
                            const void *k_cache, const int32_t *block_tables,
                            int max_blocks_per_seq, const int32_t *context_lens,
                            int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads,
                            int head_dim, int num_blocks, float scale, int dtype, int silent_warp,
                            uint64_t limit_ns, void *workspace, size_t workspace_bytes,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_SERVING_TEST_H */
