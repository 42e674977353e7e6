// evict.cu -- a cache cut to a budget by accumulated attention weight.
//
// For each (sequence, kv head) of a sequence longer than `keep`: the first f
// tokens, the last r, and of those between them the k = keep - f - r heaviest
// (of equal weights the lowest index).  Two launches:
//   select: the k-th largest weight by radix selection on order-preserving
//           32-bit keys, then the kept positions in order, with their weights;
//   move:   the kept tokens' K and V rows gathered into the spare blocks.
// Bytes: the weights once (4 a token), the kept rows of K and V read once and
// written once.
#include <climits>

#include "pa_e4m3.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;

// Larger weight, larger key; NaN the lowest; -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Length of sequence b, 0 (and a status bit) when it is out of its bounds.
__device__ __forceinline__ int checked_len(const EvictArgs& a, int b, bool report) {
  const int L = __ldg(a.context_lens + b);
  if (L < 0 || L > a.max_context_len || L > static_cast<int64_t>(a.mbs) * 16) {
    if (report) atomicOr(a.status, kStatusBadLen);
    return 0;
  }
  return L;
}

// Exclusive sum of v over the CTA's threads and its total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[kSelectWarps - 1];
  const int base = warp > 0 ? warp_sums[warp - 1] : 0;
  __syncthreads();
  return base + s - v;
}

// One CTA per (kv head, sequence).
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kSelectWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int tid = threadIdx.x;
  const int h = blockIdx.x, b = blockIdx.y;
  const int L = checked_len(a, b, h == 0 && tid == 0);
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  const bool cut = L > a.keep;
  if (h == 0) {
    if (tid == 0) a.new_lens[b] = cut ? a.keep : L;
    if (a.tables_out != nullptr)
      for (int i = tid; i < a.spare_blocks; i += kSelectThreads)
        a.tables_out[static_cast<int64_t>(b) * a.spare_blocks + i] =
            cut ? a.spare[static_cast<int64_t>(b) * a.spare_blocks + i]
                : i < a.mbs ? a.block_tables[static_cast<int64_t>(b) * a.mbs + i] : -1;
  }
  const float* w = a.weights + unit * a.stride;
  float* w_out = a.weights_out != nullptr ? a.weights_out + unit * a.out_stride : nullptr;
  int32_t* kept = a.kept + unit * a.keep;
  if (!cut) {
    for (int t = tid; t < L; t += kSelectThreads) {
      kept[t] = t;
      if (w_out != nullptr) w_out[t] = w[t];
    }
    return;
  }
  const int lo = a.first, hi = L - a.recent;   // the candidates
  const int k = a.keep - a.first - a.recent;   // how many of them stay; k < hi - lo
  // the k-th largest key, 8 bits at a time from the top: `prefix` its bits so
  // far, `left` how many of the keys with that prefix stay
  uint32_t prefix = 0;
  int left = k;
  if (k > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int t = lo + tid; t < hi; t += kSelectThreads) {
        const uint32_t key = weight_key(w[t]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid < 32) {
        // digits from the largest down, eight a lane
        int c[8], s = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) s += c[j] = hist[255 - (tid * 8 + j)];
        int above = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, above, o);
          if (tid >= o) above += u;
        }
        above -= s;
        if (above < left && above + s >= left) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (above < left && above + c[j] >= left) {
              s_prefix = prefix | (static_cast<uint32_t>(255 - (tid * 8 + j)) << shift);
              s_left = left - above;
            }
            above += c[j];
          }
        }
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
      __syncthreads();
    }
  }
  // the kept positions in order: larger keys, and the first `left` equal ones
  int at = 0, ties = 0;
  for (int base = 0; base < L; base += kSelectThreads) {
    const int t = base + tid;
    const bool guarded = t < L && (t < lo || t >= hi);
    const uint32_t key = t >= lo && t < hi && k > 0 ? weight_key(w[t]) : 0u;
    const bool inner = t >= lo && t < hi && k > 0;
    const int tie = inner && key == prefix;
    int n_ties;
    const int tie_at = ties + block_scan(tie, warp_sums, n_ties);
    ties += n_ties;
    const int keep = guarded || (inner && (key > prefix || (tie && tie_at < left)));
    int n;
    const int pos = at + block_scan(keep, warp_sums, n);
    at += n;
    if (keep) {
      kept[pos] = t;
      if (w_out != nullptr) w_out[pos] = w[t];
    }
  }
}

// One CTA per (destination page, kv head, sequence): 16 rows of K and of V.
constexpr int kMoveThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  const int page = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int L = checked_len(a, b, false);
  if (L <= a.keep) return;
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  const int dst = __ldg(a.spare + static_cast<int64_t>(b) * a.spare_blocks + page);
  if (dst < 0 || dst >= a.num_blocks) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadBlock);
    return;
  }
  constexpr int C = D / 8;   // 16-byte chunks a row
  const int rows = min(16, a.keep - page * 16);
  for (int i = threadIdx.x; i < rows * C; i += kMoveThreads) {
    const int row = i / C, c = i % C;
    const int t = __ldg(a.kept + unit * a.keep + page * 16 + row);
    const int src = __ldg(a.block_tables + static_cast<int64_t>(b) * a.mbs + t / 16);
    if (src < 0 || src >= a.num_blocks) {
      if (c == 0) atomicOr(a.status, kStatusBadBlock);
      continue;
    }
    const int64_t from = ((static_cast<int64_t>(src) * a.Hkv + h) * 16 + t % 16) * C + c;
    const int64_t to = ((static_cast<int64_t>(dst) * a.Hkv + h) * 16 + row) * C + c;
    static_cast<uint4*>(a.k_cache)[to] = static_cast<const uint4*>(a.k_cache)[from];
    static_cast<uint4*>(a.v_cache)[to] = static_cast<const uint4*>(a.v_cache)[from];
  }
}

// E4M3: one warp per (destination page, kv head, sequence, K|V).  A page's
// scale is that of the rows it now holds, so all of them are read before any is
// written.
template <int D>
__global__ void __launch_bounds__(64) evict_move_e4m3_kernel(const EvictArgs a) {
  const int page = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, kv = threadIdx.x >> 5;
  const int L = checked_len(a, b, false);
  if (L <= a.keep) return;
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  const int dst = __ldg(a.spare + static_cast<int64_t>(b) * a.spare_blocks + page);
  if (dst < 0 || dst >= a.num_blocks) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadBlock);
    return;
  }
  uint8_t* pool = static_cast<uint8_t*>(kv ? a.v_cache : a.k_cache);
  float* scales = kv ? a.v_scale : a.k_scale;
  const int rows = min(16, a.keep - page * 16);
  // lane j holds row j's source
  int64_t src_row = -1;
  float src_scale = 0.f;
  if (lane < rows) {
    const int t = __ldg(a.kept + unit * a.keep + page * 16 + lane);
    const int src = __ldg(a.block_tables + static_cast<int64_t>(b) * a.mbs + t / 16);
    if (src < 0 || src >= a.num_blocks) {
      atomicOr(a.status, kStatusBadBlock);
    } else {
      const int64_t tile = static_cast<int64_t>(src) * a.Hkv + h;
      src_row = tile * 16 + t % 16;
      src_scale = scales[tile];
    }
  }
  constexpr int P = RowF16<D>::PER_LANE;
  uint32_t codes[16];
  float s[16];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int64_t r = __shfl_sync(0xffffffffu, src_row, j);
    s[j] = __shfl_sync(0xffffffffu, src_scale, j);
    codes[j] = r >= 0 ? load_row_codes<D>(pool + r * D, lane) : 0u;
  }
  auto value2 = [&](uint32_t two, float scale) {
    const uint32_t f = e4m3x2_to_f16x2(two);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
    return make_float2(__fmul_rn(v.x, scale), __fmul_rn(v.y, scale));
  };
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 v = value2(codes[j] & 0xffffu, s[j]);
    amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
    if constexpr (P == 4) {
      const float2 u = value2(codes[j] >> 16, s[j]);
      amax = fmaxf(amax, fmaxf(fabsf(u.x), fabsf(u.y)));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = e4m3_page_scale(amax);
  const int64_t tile = static_cast<int64_t>(dst) * a.Hkv + h;
  if (lane == 0) scales[tile] = scale;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (__shfl_sync(0xffffffffu, src_row, j) < 0) continue;   // behind the last row, or skipped
    RowF16<D> x;
    const float2 v = value2(codes[j] & 0xffffu, s[j]);
    x.x[0] = v.x;
    x.x[1] = v.y;
    if constexpr (P == 4) {
      const float2 u = value2(codes[j] >> 16, s[j]);
      x.x[2] = u.x;
      x.x[3] = u.y;
    }
    store_row_codes<D>(pool + (tile * 16 + j) * D, lane, e4m3_row_codes<D>(x, scale));
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, bool fp8, cudaStream_t s) {
  evict_select_kernel<<<dim3(a.Hkv, a.B), kSelectThreads, 0, s>>>(a);
  if (cudaError_t e = cudaGetLastError()) return e;
  const dim3 grid((a.keep + 15) / 16, a.Hkv, a.B);
  if (fp8) {
    auto* kernel = a.D == 128 ? evict_move_e4m3_kernel<128> : evict_move_e4m3_kernel<64>;
    kernel<<<grid, 64, 0, s>>>(a);
  } else {
    auto* kernel = a.D == 128 ? evict_move_kernel<128> : evict_move_kernel<64>;
    kernel<<<grid, kMoveThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace pa
