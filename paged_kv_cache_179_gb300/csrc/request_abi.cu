// request_abi.cu -- the extern "C" entry points declared in include/pa_request.h.
// As in abi.cu, arguments are checked on the host before anything is launched.
#include <climits>
#include <cmath>

#include "pa_launch.h"
#include "pa_request.h"
#include "pa_request_test.h"
#include "request_launch.h"

using namespace pa;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }
constexpr int kMaxContext = 1 << 30;   // positions and what lies a tile behind them fit 32 bits
constexpr int kMaxBlocks = 1 << 30;
bool is_act(int dtype) { return dtype == PA_F16 || dtype == PA_BF16; }

int prefill(PrefillArgs a, int block_size, int dtype, size_t workspace_bytes, bool fp8,
            void* stream) {
  if (a.B < 0 || a.T < 0 || a.Hq <= 0 || a.Hkv <= 0 || a.Hq % a.Hkv != 0) return PA_ERR_INVALID_ARG;
  if (a.num_blocks <= 0 || a.mbs <= 0 || a.max_context_len < 0 || a.window < 0)
    return PA_ERR_INVALID_ARG;
  if (a.max_context_len > static_cast<int64_t>(a.mbs) * block_size) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(a.scale) || !is_act(dtype)) return PA_ERR_INVALID_ARG;
  if (a.D != 64 && a.D != 128) return PA_ERR_UNSUPPORTED;
  if (block_size != 16) return PA_ERR_UNSUPPORTED;
  a.group = a.Hq / a.Hkv;
  if (a.group > 32) return PA_ERR_UNSUPPORTED;
  if (a.B > 65535 || a.Hkv > 65535 || a.max_context_len > kMaxContext) return PA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a.T) * a.Hq > (1 << 30)) return PA_ERR_UNSUPPORTED;
  // a 16-bit pool's (block, kv head) tiles are coordinates of its tensor map
  if (!fp8 && static_cast<int64_t>(a.num_blocks) * a.Hkv > INT_MAX) return PA_ERR_UNSUPPORTED;
  if (a.window >= a.max_context_len) a.window = 0;   // the whole context
  if (!a.out || !a.q || !a.k_cache || !a.v_cache || !a.block_tables || !a.context_lens || !a.starts)
    return PA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(a.out), a.q, a.k_cache, a.v_cache})
    if (!aligned(p, 16)) return PA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(a.block_tables),
                        static_cast<const void*>(a.context_lens),
                        static_cast<const void*>(a.starts), static_cast<const void*>(a.k_scale),
                        static_cast<const void*>(a.v_scale)})
    if (!aligned(p, 4)) return PA_ERR_INVALID_ARG;
  if (a.q_stride % 8 != 0 || a.q_stride < static_cast<int64_t>(a.Hq) * a.D)
    return PA_ERR_INVALID_ARG;
  // q is read while out is written: rows of other kv heads would be lost
  if (a.out == a.q) return PA_ERR_INVALID_ARG;
  if (fp8 && (!a.k_scale || !a.v_scale)) return PA_ERR_INVALID_ARG;
  if (a.workspace == nullptr || !aligned(a.workspace, 256)) return PA_ERR_WORKSPACE;
  if (int rc = device_status_word(&a.status)) return rc;
  if (workspace_bytes < prefill_workspace_bytes(a.B, a.T, a.Hq, a.Hkv, a.D)) return PA_ERR_WORKSPACE;
  return cuda_status(launch_prefill(a, fp8, dtype == PA_BF16, static_cast<cudaStream_t>(stream)));
}

// The tables and counts that the page calls share.
int check_pages(const void* tables, int mbs, const void* num_pages, int num_rows,
                const void* ref_counts, int num_blocks) {
  if (mbs <= 0 || num_rows <= 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
  if (num_blocks > kMaxBlocks) return PA_ERR_UNSUPPORTED;
  if (!tables || !num_pages || !ref_counts) return PA_ERR_INVALID_ARG;
  if (!aligned(tables, 4) || !aligned(num_pages, 4) || !aligned(ref_counts, 16))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// The pools whose pages move.
int check_pools(void* k, void* v, float* ks, float* vs, int Hkv, int D, int block_size,
                int pool_type, PagePools* p) {
  if (Hkv <= 0) return PA_ERR_INVALID_ARG;
  if (!is_act(pool_type) && pool_type != PA_E4M3) return PA_ERR_INVALID_ARG;
  const bool fp8 = pool_type == PA_E4M3;
  if (fp8 != (ks != nullptr) || fp8 != (vs != nullptr)) return PA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return PA_ERR_UNSUPPORTED;
  if (block_size != 16 || Hkv > 65535) return PA_ERR_UNSUPPORTED;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(ks, 4) || !aligned(vs, 4))
    return PA_ERR_INVALID_ARG;
  *p = PagePools{k, v, ks, vs, static_cast<int64_t>(Hkv) * 16 * D * (fp8 ? 1 : 2), Hkv};
  return PA_OK;
}

}  // namespace

extern "C" {

size_t pa_prefill_workspace_size(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                                 int head_dim) {
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || num_q_heads <= 0 ||
      num_q_heads % num_kv_heads != 0 || num_q_heads / num_kv_heads > 32 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return prefill_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim);
}

int pa_prefill(void* out, const void* q, int64_t q_stride, const void* k_cache,
               const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
               const int32_t* context_lens, int max_context_len, const int32_t* query_starts,
               int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
               int block_size, int num_blocks, float scale, int window_size, int dtype,
               void* workspace, size_t workspace_bytes, void* stream) {
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  PrefillArgs a{};
  a.out = out;
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.starts = query_starts;
  a.workspace = workspace;
  a.mbs = max_blocks_per_seq;
  a.T = num_tokens;
  a.B = num_seqs;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.num_blocks = num_blocks;
  a.max_context_len = max_context_len;
  a.window = window_size;
  a.scale = scale;
  a.wait_limit_ns = kWaitLimitNs;
  a.drop_tile = -1;
  return prefill(a, block_size, dtype, workspace_bytes, false, stream);
}

int pa_prefill_fp8(void* out, const void* q, int64_t q_stride, const uint8_t* k_cache,
                   const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                   const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* context_lens, int max_context_len, const int32_t* query_starts,
                   int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                   int block_size, int num_blocks, float scale, int window_size, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  PrefillArgs a{};
  a.out = out;
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.starts = query_starts;
  a.workspace = workspace;
  a.mbs = max_blocks_per_seq;
  a.T = num_tokens;
  a.B = num_seqs;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.num_blocks = num_blocks;
  a.max_context_len = max_context_len;
  a.window = window_size;
  a.scale = scale;
  a.wait_limit_ns = kWaitLimitNs;
  a.drop_tile = -1;
  return prefill(a, block_size, dtype, workspace_bytes, true, stream);
}

int pa_test_prefill_timeout(void* out, const void* q, int64_t q_stride, const void* k_cache,
                            const void* v_cache, const int32_t* block_tables,
                            int max_blocks_per_seq, const int32_t* context_lens,
                            int max_context_len, const int32_t* query_starts, int num_tokens,
                            int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                            int num_blocks, float scale, int dtype, int drop_tile,
                            uint64_t limit_ns, void* workspace, size_t workspace_bytes, void* stream) {
  if (limit_ns == 0 || limit_ns > kWaitLimitNs) return PA_ERR_INVALID_ARG;
  if (num_seqs <= 0 || num_tokens <= 0 || drop_tile < 0) return PA_ERR_INVALID_ARG;
  PrefillArgs a{};
  a.out = out;
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.starts = query_starts;
  a.workspace = workspace;
  a.mbs = max_blocks_per_seq;
  a.T = num_tokens;
  a.B = num_seqs;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.num_blocks = num_blocks;
  a.max_context_len = max_context_len;
  a.scale = scale;
  a.wait_limit_ns = limit_ns;
  a.drop_tile = drop_tile;
  return prefill(a, 16, dtype, workspace_bytes, false, stream);
}

int pa_alloc_pages(int32_t* block_tables, int max_blocks_per_seq, int32_t* num_pages,
                   int num_rows, const int32_t* rows, const int32_t* new_lens, int num_items,
                   int32_t* ref_counts, int num_blocks, int block_size, int32_t* granted,
                   void* stream) {
  if (num_items == 0) return PA_OK;
  if (num_items < 0) return PA_ERR_INVALID_ARG;
  if (int rc = check_pages(block_tables, max_blocks_per_seq, num_pages, num_rows, ref_counts,
                           num_blocks))
    return rc;
  if (block_size != 16 || num_items > kPagesMaxItems) return PA_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(rows), static_cast<const void*>(new_lens),
                        static_cast<const void*>(granted)})
    if (p == nullptr || !aligned(p, 4)) return PA_ERR_INVALID_ARG;
  TakeArgs a{};
  a.block_tables = block_tables;
  a.num_pages = num_pages;
  a.rows = rows;
  a.lens = new_lens;
  a.ref_counts = ref_counts;
  a.granted = granted;
  a.mbs = max_blocks_per_seq;
  a.num_rows = num_rows;
  a.items = num_items;
  a.num_blocks = num_blocks;
  if (int rc = device_status_word(&a.status)) return rc;
  return cuda_status(launch_alloc_pages(a, static_cast<cudaStream_t>(stream)));
}

int pa_free_pages(int32_t* block_tables, int max_blocks_per_seq, int32_t* num_pages, int num_rows,
                  const int32_t* rows, int num_items, int32_t* ref_counts, int num_blocks,
                  void* stream) {
  if (num_items == 0) return PA_OK;
  if (num_items < 0) return PA_ERR_INVALID_ARG;
  if (int rc = check_pages(block_tables, max_blocks_per_seq, num_pages, num_rows, ref_counts,
                           num_blocks))
    return rc;
  if (num_items > (1 << 24)) return PA_ERR_UNSUPPORTED;
  if (rows == nullptr || !aligned(rows, 4)) return PA_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  if (int rc = device_status_word(&status)) return rc;
  return cuda_status(launch_free_pages(block_tables, max_blocks_per_seq, num_pages, num_rows, rows,
                                       num_items, ref_counts, num_blocks, status,
                                       static_cast<cudaStream_t>(stream)));
}

int pa_fork_pages(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                  int32_t* block_tables, int max_blocks_per_seq, int32_t* num_pages,
                  int32_t* context_lens, int num_rows, const int32_t* src_rows,
                  const int32_t* dst_rows, int num_items, int32_t* ref_counts, int num_blocks,
                  int num_kv_heads, int head_dim, int block_size, int pool_type,
                  int32_t* granted, void* stream) {
  if (num_items == 0) return PA_OK;
  if (num_items < 0) return PA_ERR_INVALID_ARG;
  if (int rc = check_pages(block_tables, max_blocks_per_seq, num_pages, num_rows, ref_counts,
                           num_blocks))
    return rc;
  PagePools p{};
  if (int rc = check_pools(k_cache, v_cache, k_scale, v_scale, num_kv_heads, head_dim, block_size,
                           pool_type, &p))
    return rc;
  if (num_items > kPagesMaxItems) return PA_ERR_UNSUPPORTED;
  for (const void* x : {static_cast<const void*>(context_lens), static_cast<const void*>(src_rows),
                        static_cast<const void*>(dst_rows), static_cast<const void*>(granted)})
    if (x == nullptr || !aligned(x, 4)) return PA_ERR_INVALID_ARG;
  TakeArgs a{};
  a.block_tables = block_tables;
  a.num_pages = num_pages;
  a.rows = dst_rows;
  a.src_rows = src_rows;
  a.lens = context_lens;
  a.ref_counts = ref_counts;
  a.granted = granted;
  a.mbs = max_blocks_per_seq;
  a.num_rows = num_rows;
  a.items = num_items;
  a.num_blocks = num_blocks;
  if (int rc = device_status_word(&a.status)) return rc;
  return cuda_status(launch_fork_pages(a, context_lens, p, static_cast<cudaStream_t>(stream)));
}

size_t pa_compact_workspace_size(int num_blocks) {
  return num_blocks > 0 && num_blocks <= kMaxBlocks ? compact_workspace_bytes(num_blocks) : 0;
}

int pa_compact_pages(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                     const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* num_pages, int num_rows, const int32_t* ref_counts,
                     int num_blocks, int num_kv_heads, int head_dim, int block_size,
                     int pool_type, int32_t* tables_out, int32_t* ref_counts_out,
                     int32_t* moved_to, int32_t* num_live, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (int rc = check_pages(block_tables, max_blocks_per_seq, num_pages, num_rows, ref_counts,
                           num_blocks))
    return rc;
  PagePools p{};
  if (int rc = check_pools(k_cache, v_cache, k_scale, v_scale, num_kv_heads, head_dim, block_size,
                           pool_type, &p))
    return rc;
  for (const void* x : {static_cast<const void*>(tables_out),
                        static_cast<const void*>(ref_counts_out),
                        static_cast<const void*>(moved_to), static_cast<const void*>(num_live)})
    if (x == nullptr || !aligned(x, 4)) return PA_ERR_INVALID_ARG;
  if (moved_to == ref_counts || moved_to == ref_counts_out) return PA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256) ||
      workspace_bytes < compact_workspace_bytes(num_blocks))
    return PA_ERR_WORKSPACE;
  CompactArgs a{};
  a.block_tables = block_tables;
  a.num_pages = num_pages;
  a.ref_counts = ref_counts;
  a.tables_out = tables_out;
  a.ref_counts_out = ref_counts_out;
  a.moved_to = moved_to;
  a.num_live = num_live;
  a.workspace = workspace;
  a.mbs = max_blocks_per_seq;
  a.num_rows = num_rows;
  a.num_blocks = num_blocks;
  if (int rc = device_status_word(&a.status)) return rc;
  return cuda_status(launch_compact_pages(a, p, static_cast<cudaStream_t>(stream)));
}

int pa_process_logits(void* out, int64_t out_stride, const void* logits, int64_t logits_stride,
                      const pa_logits_spec* spec, int num_seqs, int rows_per_seq, int vocab_size,
                      int dtype, int as_probs, void* stream) {
  if (num_seqs == 0) return PA_OK;
  if (spec == nullptr || num_seqs < 0 || rows_per_seq < 1 || rows_per_seq > 1025 || vocab_size <= 0)
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_F32 && !is_act(dtype)) return PA_ERR_INVALID_ARG;
  if (as_probs != 0 && as_probs != 1) return PA_ERR_INVALID_ARG;
  if (vocab_size > kLogitsMaxVocab || static_cast<int64_t>(num_seqs) * rows_per_seq > (1 << 24))
    return PA_ERR_UNSUPPORTED;
  if (!out || !logits || !aligned(out, 16) || !aligned(logits, 16)) return PA_ERR_INVALID_ARG;
  if (out_stride < vocab_size || logits_stride < vocab_size) return PA_ERR_INVALID_ARG;
  // in place: the same rows, of the same type
  if (out == logits && (out_stride != logits_stride || (as_probs && dtype != PA_F32)))
    return PA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(spec->history),
                        static_cast<const void*>(spec->history_lens),
                        static_cast<const void*>(spec->prompt_lens),
                        static_cast<const void*>(spec->draft_tokens),
                        static_cast<const void*>(spec->repetition),
                        static_cast<const void*>(spec->presence),
                        static_cast<const void*>(spec->frequency),
                        static_cast<const void*>(spec->temperature),
                        static_cast<const void*>(spec->bias_tokens),
                        static_cast<const void*>(spec->bias_values),
                        static_cast<const void*>(spec->allowed)})
    if (!aligned(p, 4)) return PA_ERR_INVALID_ARG;
  if (spec->history != nullptr && (spec->history_lens == nullptr || spec->history_stride < 0))
    return PA_ERR_INVALID_ARG;
  if (spec->history == nullptr && spec->prompt_lens != nullptr) return PA_ERR_INVALID_ARG;
  if ((spec->bias_tokens != nullptr) != (spec->bias_values != nullptr)) return PA_ERR_INVALID_ARG;
  if (spec->num_bias < 0 || (spec->bias_tokens == nullptr && spec->num_bias > 0))
    return PA_ERR_INVALID_ARG;
  if (spec->num_bias > kLogitsMaxBias) return PA_ERR_UNSUPPORTED;
  if (spec->history != nullptr && spec->history_stride > kMaxContext) return PA_ERR_UNSUPPORTED;
  if (spec->allowed != nullptr && spec->allowed_stride < (vocab_size + 31) / 32)
    return PA_ERR_INVALID_ARG;
  LogitsArgs a{};
  a.out = out;
  a.logits = logits;
  a.out_stride = out_stride;
  a.in_stride = logits_stride;
  a.spec = *spec;
  if (rows_per_seq == 1) a.spec.draft_tokens = nullptr;
  a.B = num_seqs;
  a.rows = rows_per_seq;
  a.V = vocab_size;
  if (int rc = device_status_word(&a.status)) return rc;
  return cuda_status(launch_logits(a, dtype, as_probs != 0, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
