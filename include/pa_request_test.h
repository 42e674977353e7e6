/*
 * pa_request_test.h -- the failure-path test of the waits in pa_request.h, as those
 * of pa_serving_test.h and pa.h are for theirs: it makes them run out on purpose,
 * with a short limit, so that a test can check the status and that the context and
 * the workspace stay usable.  It neither faults, traps nor spins without bound.
 */
#ifndef PA_REQUEST_TEST_H
#define PA_REQUEST_TEST_H

#include "pa_request.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pa_prefill (block size 16, no window) where the keys of tile drop_tile (0 ..) of each
 * CTA's stream of tiles are never copied: a CTA with that many waits for them, gives up
 * after limit_ns (1 .. 2e9), sets PA_STATUS_TIMEOUT and returns once its copies and
 * products in flight have ended (the one that never comes is waited for, for 2 s at
 * most).  Outputs may be missing.
 */
int pa_test_prefill_timeout(void *out, const void *q, int64_t q_stride, const void *k_cache,
                            const void *v_cache, const int32_t *block_tables,
                            int max_blocks_per_seq, const int32_t *context_lens,
                            int max_context_len, const int32_t *query_starts, int num_tokens,
                            int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                            int num_blocks, float scale, int dtype, int drop_tile,
                            uint64_t limit_ns, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_REQUEST_TEST_H */
