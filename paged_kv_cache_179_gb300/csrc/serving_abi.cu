// serving_abi.cu -- the extern "C" entry points declared in include/pa_serving.h.
// As in abi.cu, arguments are checked on the host before anything is launched.
#include <climits>
#include <cmath>

#include "pa_launch.h"
#include "pa_serving.h"
#include "pa_serving_test.h"
#include "serving_launch.h"

using namespace pa;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }
constexpr int kMaxContext = 1 << 30;   // the kernels step beyond a token's index in 32 bits
bool is_act(int dtype) { return dtype == PA_F16 || dtype == PA_BF16; }

// f radians as a fraction of a turn, modulo 1, in units of 2^-64.  1 / 2 pi as the sum
// of two doubles and the first product's rounding (the fma gives it exactly) make
// f / 2 pi to 2^-104 of itself, which is below 2^-64 for every f up to 2^40; one
// division would leave 2^-53 of it, times the position: 7e-7 rad for 1 radian at
// position 2^31.
uint64_t turn_fraction(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / 2 pi
  const double t = f * kHi, rest = std::fma(f, kHi, -t) + f * kLo;
  auto fixed = [](double x) {
    x -= std::trunc(x);   // exact, as the product with a power of two is
    const uint64_t m = static_cast<uint64_t>(std::fabs(x) * 0x1p64);
    return x < 0 ? 0 - m : m;
  };
  return fixed(t) + fixed(rest);
}

// Checks the rotation's arguments and fills the launch's table.
int rope_table(const pa_rope_spec* spec, int head_dim, RopeTable* t) {
  if (spec == nullptr || spec->inv_freq == nullptr) return PA_ERR_INVALID_ARG;
  if (spec->num_axes < 1 || spec->num_axes > kMaxRopeAxes) return PA_ERR_INVALID_ARG;
  if (spec->freq_axis == nullptr && spec->num_axes != 1) return PA_ERR_INVALID_ARG;
  if (spec->adjacent != 0 && spec->adjacent != 1) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(spec->amplitude)) return PA_ERR_INVALID_ARG;
  if (spec->rotary_dim < 16 || spec->rotary_dim > head_dim) return PA_ERR_INVALID_ARG;
  if (spec->rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;   // 8 pairs a 16-byte chunk pair
  for (int i = 0; i < spec->rotary_dim / 2; ++i) {
    const double f = spec->inv_freq[i];
    if (!std::isfinite(f)) return PA_ERR_INVALID_ARG;
    const int axis = spec->freq_axis != nullptr ? spec->freq_axis[i] : 0;
    if (axis < 0 || axis >= spec->num_axes) return PA_ERR_INVALID_ARG;
    t->turns[i] = turn_fraction(f);                   // whole turns do not matter
    t->axis[i] = static_cast<uint8_t>(axis);
  }
  return PA_OK;
}

int check_rope(int T, int Hq, int Hkv, int D, int dtype, const int32_t* positions) {
  if (T < 0 || Hq < 0 || Hkv < 0 || D <= 0) return PA_ERR_INVALID_ARG;
  if (!is_act(dtype)) return PA_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 2 * kMaxRopePairs) return PA_ERR_UNSUPPORTED;
  if (positions == nullptr || !aligned(positions, 4)) return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(Hkv) > 65535) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// One side's tensors: 16-byte aligned, a stride that keeps rows aligned and apart.
bool rope_side(const void* out, const void* in, int64_t stride, int heads, int D) {
  if (heads == 0) return true;
  return out != nullptr && in != nullptr && aligned(out, 16) && aligned(in, 16) &&
         stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * D;
}

int rope_append(RopeArgs& a, bool fp8, const pa_rope_spec* spec, int dtype, void* stream) {
  RopeTable t{};
  if (int rc = check_rope(a.T, a.Hq, a.Hkv, a.D, dtype, a.positions)) return rc;
  if (int rc = rope_table(spec, a.D, &t)) return rc;
  if (a.Hkv == 0 || a.slots == nullptr || !aligned(a.slots, 8)) return PA_ERR_INVALID_ARG;
  if (a.block_size <= 0 || a.num_blocks <= 0) return PA_ERR_INVALID_ARG;
  if (fp8 && a.D != 64 && a.D != 128) return PA_ERR_UNSUPPORTED;
  if (fp8 && a.block_size != 16) return PA_ERR_UNSUPPORTED;
  // CTAs of one launch
  if (static_cast<int64_t>(a.T) * (1 + a.Hkv) > INT_MAX) return PA_ERR_UNSUPPORTED;
  if (!rope_side(a.q_out, a.q, a.q_stride, a.Hq, a.D) ||
      !rope_side(a.k_cache, a.k, a.k_stride, a.Hkv, a.D) ||
      !rope_side(a.v_cache, a.v, a.v_stride, a.Hkv, a.D))
    return PA_ERR_INVALID_ARG;
  if (a.q_out == a.q && a.Hq > 0 && a.q_stride != static_cast<int64_t>(a.Hq) * a.D)
    return PA_ERR_INVALID_ARG;
  if (fp8 && (a.k_scale == nullptr || a.v_scale == nullptr || !aligned(a.k_scale, 4) ||
              !aligned(a.v_scale, 4)))
    return PA_ERR_INVALID_ARG;
  if (int rc = device_status_word(&a.status)) return rc;
  a.pairs = spec->rotary_dim / 2;
  a.adjacent = spec->adjacent;
  a.amplitude = spec->amplitude;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == PA_BF16;
  return cuda_status(fp8 ? launch_rope_append_fp8(a, t, bf16, s) : launch_rope(a, t, bf16, s));
}

int attention_weights(WeightsArgs a, int block_size, float scale, int dtype, size_t workspace_bytes,
                      bool fp8, void* stream) {
  if (a.B < 0 || a.Hq <= 0 || a.Hkv <= 0 || a.Hq % a.Hkv != 0) return PA_ERR_INVALID_ARG;
  if (a.num_blocks <= 0 || a.mbs <= 0 || a.max_context_len < 0) return PA_ERR_INVALID_ARG;
  if (a.max_context_len > static_cast<int64_t>(a.mbs) * block_size) return PA_ERR_INVALID_ARG;
  if (a.stride < a.max_context_len) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(a.decay) || a.decay < 0.f) return PA_ERR_INVALID_ARG;
  if (a.fresh < 0 || a.q_tokens < 1 || a.q_tokens > 1024) return PA_ERR_INVALID_ARG;
  if (!is_act(dtype)) return PA_ERR_INVALID_ARG;
  if (a.D != 64 && a.D != 128) return PA_ERR_UNSUPPORTED;
  if (block_size != 16) return PA_ERR_UNSUPPORTED;
  a.group = a.Hq / a.Hkv;
  if (a.group > kWeightsMaxRows) return PA_ERR_UNSUPPORTED;
  if (a.B > 65535 || a.Hkv > 65535) return PA_ERR_UNSUPPORTED;
  if (a.max_context_len > kMaxContext) return PA_ERR_UNSUPPORTED;
  // the pages of one launch's sequences are counted in 32 bits
  if ((a.max_context_len / 16 + INT64_C(1)) * (a.B < kWeightsMaxBatch ? a.B : kWeightsMaxBatch) > INT_MAX)
    return PA_ERR_UNSUPPORTED;
  if (!a.weights || !a.q || !a.k_cache || !a.block_tables || !a.context_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned(a.weights, 4) || !aligned(a.q, 16) || !aligned(a.k_cache, 16) ||
      !aligned(a.block_tables, 4) || !aligned(a.context_lens, 4))
    return PA_ERR_INVALID_ARG;
  if (fp8 && (a.k_scale == nullptr || !aligned(a.k_scale, 4))) return PA_ERR_INVALID_ARG;
  if (a.workspace == nullptr || !aligned(a.workspace, 256)) return PA_ERR_WORKSPACE;
  if (int rc = device_status_word(&a.status)) return rc;
  if (workspace_bytes < pa_attention_weights_workspace_size(a.B, a.Hq, a.Hkv, a.max_context_len,
                                                            a.q_tokens))
    return PA_ERR_WORKSPACE;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wide = aligned(a.k_cache, 32);
  return cuda_status(launch_weights(a, fp8, dtype == PA_BF16, static_cast<cudaStream_t>(stream)));
}

int evict(EvictArgs a, int block_size, bool fp8, void* stream) {
  if (a.B < 0 || a.Hkv <= 0 || a.num_blocks <= 0 || a.mbs <= 0 || a.max_context_len < 0)
    return PA_ERR_INVALID_ARG;
  if (a.max_context_len > static_cast<int64_t>(a.mbs) * block_size) return PA_ERR_INVALID_ARG;
  if (a.keep <= 0 || a.first < 0 || a.recent < 0 ||
      static_cast<int64_t>(a.first) + a.recent > a.keep)
    return PA_ERR_INVALID_ARG;
  if (a.stride < a.max_context_len) return PA_ERR_INVALID_ARG;
  if (a.weights_out != nullptr && (a.out_stride < a.keep || a.weights_out == a.weights))
    return PA_ERR_INVALID_ARG;
  if (a.D != 64 && a.D != 128) return PA_ERR_UNSUPPORTED;
  if (block_size != 16) return PA_ERR_UNSUPPORTED;
  if (a.B > 65535 || a.Hkv > 65535 || a.max_context_len > kMaxContext) return PA_ERR_UNSUPPORTED;
  if (a.spare_blocks < (a.keep + static_cast<int64_t>(15)) / 16) return PA_ERR_INVALID_ARG;
  if (!a.k_cache || !a.v_cache || !a.weights || !a.block_tables || !a.context_lens || !a.spare ||
      !a.new_lens || !a.kept)
    return PA_ERR_INVALID_ARG;
  if (a.new_lens == a.context_lens || a.spare == a.block_tables ||
      a.tables_out == a.block_tables || a.tables_out == a.spare)
    return PA_ERR_INVALID_ARG;
  if (!aligned(a.k_cache, 16) || !aligned(a.v_cache, 16)) return PA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(a.weights), static_cast<const void*>(a.weights_out),
                        static_cast<const void*>(a.block_tables),
                        static_cast<const void*>(a.context_lens), static_cast<const void*>(a.spare),
                        static_cast<const void*>(a.tables_out),
                        static_cast<const void*>(a.new_lens), static_cast<const void*>(a.kept),
                        static_cast<const void*>(a.k_scale), static_cast<const void*>(a.v_scale)})
    if (!aligned(p, 4)) return PA_ERR_INVALID_ARG;
  if (fp8 && (!a.k_scale || !a.v_scale)) return PA_ERR_INVALID_ARG;
  if (int rc = device_status_word(&a.status)) return rc;
  return cuda_status(launch_evict(a, fp8, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int pa_rope(void* q_out, const void* q, int64_t q_stride, void* k_out, const void* k,
            int64_t k_stride, const int32_t* positions, const pa_rope_spec* spec, int num_tokens,
            int num_q_heads, int num_kv_heads, int head_dim, int dtype, void* stream) {
  if (num_tokens == 0) return PA_OK;
  RopeTable t{};
  if (int rc = check_rope(num_tokens, num_q_heads, num_kv_heads, head_dim, dtype, positions))
    return rc;
  if (int rc = rope_table(spec, head_dim, &t)) return rc;
  if (!rope_side(q_out, q, q_stride, num_q_heads, head_dim) ||
      !rope_side(k_out, k, k_stride, num_kv_heads, head_dim))
    return PA_ERR_INVALID_ARG;
  if ((num_q_heads > 0 && q_out == q && q_stride != static_cast<int64_t>(num_q_heads) * head_dim) ||
      (num_kv_heads > 0 && k_out == k && k_stride != static_cast<int64_t>(num_kv_heads) * head_dim))
    return PA_ERR_INVALID_ARG;
  if (num_q_heads == 0 && num_kv_heads == 0) return PA_OK;
  RopeArgs a{};
  a.q_out = q_out;
  a.q = q;
  a.q_stride = q_stride;
  a.k_out = k_out;
  a.k = k;
  a.k_stride = k_stride;
  a.positions = positions;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.pairs = spec->rotary_dim / 2;
  a.adjacent = spec->adjacent;
  a.amplitude = spec->amplitude;
  return cuda_status(launch_rope(a, t, dtype == PA_BF16, static_cast<cudaStream_t>(stream)));
}

int pa_rope_append(void* q_out, const void* q, int64_t q_stride, const void* k_new,
                   int64_t k_stride, const void* v_new, int64_t v_stride, void* k_cache,
                   void* v_cache, const int64_t* slot_mapping, const int32_t* positions,
                   const pa_rope_spec* spec, int num_tokens, int num_q_heads, int num_kv_heads,
                   int head_dim, int block_size, int num_blocks, int dtype, void* stream) {
  if (num_tokens == 0) return PA_OK;
  RopeArgs a{};
  a.q_out = q_out;
  a.q = q;
  a.q_stride = q_stride;
  a.k = k_new;
  a.k_stride = k_stride;
  a.v = v_new;
  a.v_stride = v_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.slots = slot_mapping;
  a.positions = positions;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  return rope_append(a, false, spec, dtype, stream);
}

int pa_rope_append_fp8(void* q_out, const void* q, int64_t q_stride, const void* k_new,
                       int64_t k_stride, const void* v_new, int64_t v_stride, uint8_t* k_cache,
                       uint8_t* v_cache, float* k_scale, float* v_scale,
                       const int64_t* slot_mapping, const int32_t* positions,
                       const pa_rope_spec* spec, int num_tokens, int num_q_heads,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks, int dtype,
                       void* stream) {
  if (num_tokens == 0) return PA_OK;
  RopeArgs a{};
  a.q_out = q_out;
  a.q = q;
  a.q_stride = q_stride;
  a.k = k_new;
  a.k_stride = k_stride;
  a.v = v_new;
  a.v_stride = v_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slots = slot_mapping;
  a.positions = positions;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  return rope_append(a, true, spec, dtype, stream);
}

size_t pa_attention_weights_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                           int max_context_len, int queries_per_seq) {
  if (num_seqs < 0 || num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      max_context_len < 0 || queries_per_seq < 1)
    return 0;
  const int64_t rows = static_cast<int64_t>(queries_per_seq) * (num_q_heads / num_kv_heads);
  return weights_workspace_bytes(num_seqs, num_kv_heads, max_context_len,
                                 static_cast<int>(rows < kWeightsMaxRows ? rows : kWeightsMaxRows));
}

int pa_attention_weights(float* weights, int64_t weights_stride, const void* q,
                         const void* k_cache, const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* context_lens, int max_context_len, int num_seqs,
                         int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, float scale, float decay, int fresh_tokens,
                         int queries_per_seq, int dtype, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (num_seqs == 0) return PA_OK;
  WeightsArgs a{};
  a.weights = weights;
  a.stride = weights_stride;
  a.q = q;
  a.k_cache = k_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.workspace = workspace;
  a.mbs = max_blocks_per_seq;
  a.B = num_seqs;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.num_blocks = num_blocks;
  a.max_context_len = max_context_len;
  a.q_tokens = queries_per_seq;
  a.decay = decay;
  a.fresh = fresh_tokens;
  a.wait_limit_ns = kWaitLimitNs;
  a.silent_warp = -1;
  return attention_weights(a, block_size, scale, dtype, workspace_bytes, false, stream);
}

int pa_attention_weights_fp8(float* weights, int64_t weights_stride, const void* q,
                             const uint8_t* k_cache, const float* k_scale,
                             const int32_t* block_tables, int max_blocks_per_seq,
                             const int32_t* context_lens, int max_context_len, int num_seqs,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                             int num_blocks, float scale, float decay, int fresh_tokens,
                             int queries_per_seq, int dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (num_seqs == 0) return PA_OK;
  WeightsArgs a{};
  a.weights = weights;
  a.stride = weights_stride;
  a.q = q;
  a.k_cache = k_cache;
  a.k_scale = k_scale;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.workspace = workspace;
  a.mbs = max_blocks_per_seq;
  a.B = num_seqs;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.num_blocks = num_blocks;
  a.max_context_len = max_context_len;
  a.q_tokens = queries_per_seq;
  a.decay = decay;
  a.fresh = fresh_tokens;
  a.wait_limit_ns = kWaitLimitNs;
  a.silent_warp = -1;
  return attention_weights(a, block_size, scale, dtype, workspace_bytes, true, stream);
}

int pa_test_weights_timeout(float* weights, int64_t weights_stride, const void* q,
                            const void* k_cache, const int32_t* block_tables,
                            int max_blocks_per_seq, const int32_t* context_lens,
                            int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads,
                            int head_dim, int num_blocks, float scale, int dtype, int silent_warp,
                            uint64_t limit_ns, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (limit_ns == 0 || limit_ns > kWaitLimitNs) return PA_ERR_INVALID_ARG;
  if (num_seqs <= 0 || num_seqs > kWeightsMaxBatch || silent_warp < 0) return PA_ERR_INVALID_ARG;
  if (max_context_len <= kWeightsClusterPages * 16) return PA_ERR_UNSUPPORTED;   // no warp waits
  WeightsArgs a{};
  a.weights = weights;
  a.stride = weights_stride;
  a.q = q;
  a.k_cache = k_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.workspace = workspace;
  a.mbs = max_blocks_per_seq;
  a.B = num_seqs;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.num_blocks = num_blocks;
  a.max_context_len = max_context_len;
  a.q_tokens = 1;
  a.wait_limit_ns = limit_ns;
  a.silent_warp = silent_warp;
  return attention_weights(a, 16, scale, dtype, workspace_bytes, false, stream);
}

int pa_evict(void* k_cache, void* v_cache, const float* weights, int64_t weights_stride,
             float* weights_out, int64_t weights_out_stride, const int32_t* block_tables,
             int max_blocks_per_seq, const int32_t* context_lens, int max_context_len,
             const int32_t* spare_tables, int spare_blocks_per_seq, int32_t* tables_out,
             int32_t* new_lens, int32_t* kept, int num_seqs, int num_kv_heads, int head_dim,
             int block_size, int num_blocks, int keep, int first_tokens, int recent_tokens,
             int dtype, void* stream) {
  if (num_seqs == 0) return PA_OK;
  if (!is_act(dtype)) return PA_ERR_INVALID_ARG;
  EvictArgs a{k_cache, v_cache, nullptr, nullptr, weights, weights_out, weights_stride,
              weights_out_stride, block_tables, context_lens, spare_tables, tables_out, new_lens,
              kept, nullptr, max_blocks_per_seq, spare_blocks_per_seq, num_seqs, num_kv_heads,
              head_dim, num_blocks, max_context_len, keep, first_tokens, recent_tokens};
  return evict(a, block_size, false, stream);
}

int pa_evict_fp8(uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale,
                 const float* weights, int64_t weights_stride, float* weights_out,
                 int64_t weights_out_stride, const int32_t* block_tables, int max_blocks_per_seq,
                 const int32_t* context_lens, int max_context_len, const int32_t* spare_tables,
                 int spare_blocks_per_seq, int32_t* tables_out, int32_t* new_lens, int32_t* kept,
                 int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                 int keep, int first_tokens, int recent_tokens, void* stream) {
  if (num_seqs == 0) return PA_OK;
  EvictArgs a{k_cache, v_cache, k_scale, v_scale, weights, weights_out, weights_stride,
              weights_out_stride, block_tables, context_lens, spare_tables, tables_out, new_lens,
              kept, nullptr, max_blocks_per_seq, spare_blocks_per_seq, num_seqs, num_kv_heads,
              head_dim, num_blocks, max_context_len, keep, first_tokens, recent_tokens};
  return evict(a, block_size, true, stream);
}

int pa_verify_drafts(int32_t* out_tokens, int32_t* num_accepted, const void* target_probs,
                     int64_t target_stride, const void* draft_probs, int64_t draft_stride,
                     const int32_t* draft_tokens, const int32_t* num_drafts,
                     const float* uniforms, int num_seqs, int max_drafts, int vocab_size,
                     int dtype, void* stream) {
  if (num_seqs == 0) return PA_OK;
  if (num_seqs < 0 || max_drafts < 0 || max_drafts > 1024 || vocab_size <= 0)
    return PA_ERR_INVALID_ARG;
  if (dtype != PA_F32 && !is_act(dtype)) return PA_ERR_INVALID_ARG;
  if (vocab_size > (1 << 24) || num_seqs > (1 << 24)) return PA_ERR_UNSUPPORTED;
  if (!out_tokens || !num_accepted || !target_probs || !uniforms) return PA_ERR_INVALID_ARG;
  if (max_drafts > 0 && !draft_tokens) return PA_ERR_INVALID_ARG;
  if (target_stride < vocab_size || (draft_probs && draft_stride < vocab_size))
    return PA_ERR_INVALID_ARG;
  if (!aligned(target_probs, 16) || !aligned(draft_probs, 16)) return PA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(out_tokens),
                        static_cast<const void*>(num_accepted),
                        static_cast<const void*>(draft_tokens),
                        static_cast<const void*>(num_drafts), static_cast<const void*>(uniforms)})
    if (!aligned(p, 4)) return PA_ERR_INVALID_ARG;
  VerifyArgs a{};
  a.out_tokens = out_tokens;
  a.num_accepted = num_accepted;
  a.p = target_probs;
  a.q = max_drafts > 0 ? draft_probs : nullptr;
  a.p_stride = target_stride;
  a.q_stride = draft_stride;
  a.draft_tokens = draft_tokens;
  a.num_drafts = num_drafts;
  a.uniforms = uniforms;
  a.B = num_seqs;
  a.n = max_drafts;
  a.V = vocab_size;
  if (int rc = device_status_word(&a.status)) return rc;
  return cuda_status(launch_verify(a, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
