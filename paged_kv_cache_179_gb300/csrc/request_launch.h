// request_launch.h -- kernel launchers of the calls in include/pa_request.h.
// request_abi.cu validates arguments and then calls these.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "pa_request.h"

namespace pa {

constexpr unsigned kStatusBadRow = 128u;   // a row outside the tables, or forked onto itself

// ------------------------------------------------------------------- prefill
struct PrefillArgs {
  void* out;                   // [T][Hq][D]
  const void* q;
  int64_t q_stride;            // elements a token
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;        // E4M3 pools
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* starts;       // [B + 1]
  void* workspace;
  unsigned* status;
  int mbs, T, B, Hq, Hkv, group, D, num_blocks, max_context_len, window;
  float scale;
  uint64_t wait_limit_ns;      // time limit of every wait
  int drop_tile;               // a test's: this tile of each CTA's is not copied (-1: none)
};
size_t prefill_workspace_bytes(int B, int T, int Hq, int Hkv, int D);
// Calls of these kernels follow one another: each is launched while the one before it on the
// stream still ends, and waits for that end before it touches memory (griddep_wait).
inline cudaLaunchAttribute after_previous() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                         const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {after_previous()};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_prefill(const PrefillArgs& a, bool fp8, bool bf16, cudaStream_t s);

// --------------------------------------------------------------------- pages
constexpr int kPagesMaxItems = 32768;   // items of a call that takes pages

struct TakeArgs {
  int32_t* block_tables;
  int32_t* num_pages;
  const int32_t* rows;         // the rows that get pages (a fork's destinations)
  const int32_t* src_rows;     // a fork's sources, or null
  const int32_t* lens;         // new_lens by item, or a fork's context_lens by row
  int32_t* ref_counts;
  int32_t* granted;
  unsigned* status;
  int mbs, num_rows, items, num_blocks;
};
cudaError_t launch_alloc_pages(const TakeArgs& a, cudaStream_t s);
cudaError_t launch_free_pages(int32_t* tables, int mbs, int32_t* num_pages, int num_rows,
                              const int32_t* rows, int items, int32_t* ref_counts, int num_blocks,
                              unsigned* status, cudaStream_t s);

// The pools whose pages move: bytes of one page of K (and of V), kv heads.
struct PagePools {
  void* k_cache;
  void* v_cache;
  float* k_scale;              // E4M3 pools, else null
  float* v_scale;
  int64_t page_bytes;
  int Hkv;
};
cudaError_t launch_fork_pages(const TakeArgs& a, int32_t* context_lens, const PagePools& p,
                              cudaStream_t s);

struct CompactArgs {
  const int32_t* block_tables;
  const int32_t* num_pages;
  const int32_t* ref_counts;
  int32_t* tables_out;
  int32_t* ref_counts_out;
  int32_t* moved_to;
  int32_t* num_live;
  void* workspace;
  unsigned* status;
  int mbs, num_rows, num_blocks;
};
size_t compact_workspace_bytes(int num_blocks);
cudaError_t launch_compact_pages(const CompactArgs& a, const PagePools& p, cudaStream_t s);

// -------------------------------------------------------------------- logits
constexpr int kLogitsMaxBias = 1024;
constexpr int kLogitsMaxVocab = 1 << 19;

struct LogitsArgs {
  void* out;
  const void* logits;
  int64_t out_stride, in_stride;
  pa_logits_spec spec;
  unsigned* status;
  int B, rows, V;              // rows per sequence
};
cudaError_t launch_logits(const LogitsArgs& a, int dtype, bool probs, cudaStream_t s);

}  // namespace pa
