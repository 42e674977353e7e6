// serving_launch.h -- kernel launchers of the calls in include/pa_serving.h.
// serving_abi.cu validates arguments and then calls these.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace pa {

constexpr unsigned kStatusBadToken = 64u;   // a drafted token outside the vocabulary

// ------------------------------------------------------------------ rotation
constexpr int kMaxRopePairs = 128;   // head_dim up to 256
constexpr int kMaxRopeAxes = 4;

// The rotation's frequencies, by value with the launch: turns per position as
// 64-bit fractions (2^-64), so that position * turns modulo 2^64 is the
// angle's exact fraction of a turn, and each pair's axis.
struct RopeTable {
  uint64_t turns[kMaxRopePairs];
  uint8_t axis[kMaxRopePairs];
};

struct RopeArgs {
  void* q_out;                 // [T][Hq][D]
  const void* q;
  void* k_out;                 // [T][Hkv][D], or null: k goes to the pool
  const void* k;
  const void* v;               // null: no append
  int64_t q_stride, k_stride, v_stride;   // elements a token
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  const int64_t* slots;
  const int32_t* positions;    // [axes][T]
  unsigned* status;
  int T, Hq, Hkv, D;
  int block_size;
  int64_t num_blocks;
  int pairs;                   // rotary_dim / 2
  int adjacent;
  float amplitude;
};

cudaError_t launch_rope(const RopeArgs& a, const RopeTable& t, bool bf16, cudaStream_t s);
cudaError_t launch_rope_append_fp8(const RopeArgs& a, const RopeTable& t, bool bf16,
                                   cudaStream_t s);

// ------------------------------------------------------------------- weights
struct WeightsArgs {
  float* weights;              // [B][Hkv][stride]
  int64_t stride;
  const void* q;               // [B][q_tokens][Hq][D]
  const void* k_cache;
  const float* k_scale;        // E4M3 pools
  const int32_t* block_tables;
  const int32_t* context_lens;
  void* workspace;
  unsigned* status;
  int mbs, B, Hq, Hkv, group, D, num_blocks, max_context_len;
  int q_tokens;                // query tokens per sequence in q
  int q_first, n_q;            // those this pass serves
  float scale_log2, decay;
  int fresh;                   // tokens whose old weight is 0
  bool wide;                   // k_cache is 32-byte aligned
  uint64_t wait_limit_ns;      // time limit of a warp's wait for others
  int silent_warp;             // of the launch, whose statistics are not announced (-1: none)
};
constexpr int kWeightsMaxBatch = 512;    // sequences per launch
constexpr int kWeightsClusterPages = 256;   // a longer bound takes the cooperative launch
constexpr int kWeightsMaxRows = 32;      // query rows per pass
size_t weights_workspace_bytes(int B, int Hkv, int max_context_len, int rows);
cudaError_t launch_weights(const WeightsArgs& a, bool fp8, bool bf16, cudaStream_t s);

// ------------------------------------------------------------------ eviction
struct EvictArgs {
  void* k_cache;
  void* v_cache;
  float* k_scale;              // E4M3 pools
  float* v_scale;
  const float* weights;
  float* weights_out;          // or null
  int64_t stride, out_stride;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* spare;        // [B][spare_blocks]
  int32_t* tables_out;         // or null
  int32_t* new_lens;
  int32_t* kept;               // [B][Hkv][keep]
  unsigned* status;
  int mbs, spare_blocks, B, Hkv, D, num_blocks, max_context_len;
  int keep, first, recent;
};
cudaError_t launch_evict(const EvictArgs& a, bool fp8, cudaStream_t s);

// -------------------------------------------------------------- verification
struct VerifyArgs {
  int32_t* out_tokens;         // [B][n + 1]
  int32_t* num_accepted;       // [B]
  const void* p;               // rows [B][n + 1]
  const void* q;               // rows [B][n], or null
  int64_t p_stride, q_stride;
  const int32_t* draft_tokens;
  const int32_t* num_drafts;   // or null
  const float* uniforms;       // [B][n + 1]
  unsigned* status;
  int B, n, V;
};
cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s);

}  // namespace pa
