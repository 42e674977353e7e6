// evict.cu -- a cache cut to a budget by accumulated attention weight.
//
// For each (sequence, kv head) of a sequence longer than `keep`: the first f
// tokens, the last r, and of those between them the k = keep - f - r heaviest
// (of equal weights the lowest index).  Two launches, the second a programmatic
// dependent of the first:
//   select: the k-th largest weight by radix selection on order-preserving
//           32-bit keys, then the kept positions in order, with their weights;
//   move:   the kept tokens' K and V rows gathered into the spare blocks.
// Bytes: the weights once (4 a token), the kept rows of K and V read once and
// written once.
#include <mutex>

#include "pa_e4m3.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

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

// ------------------------------------------------------------------- select
// One CTA per (kv head, sequence).  A warp owns a contiguous part of the
// candidates, so that positions come out in order with one scan over the warps'
// counts and ballots inside each.  The keys of the first kKeys candidates stay in
// shared memory (those behind them are read again, from L2).
//
// Radix selection in digits of 11, 11 and 10 bits.  The first digit's histogram
// sees every key, and the weights' few exponents would make the lanes of a warp
// add to the same few bins: kCopies copies, one for every kCopies-th lane.  What
// falls into the chosen bin is then gathered into a list, on which the other
// digits work (on all keys again, if the list does not hold them).
template <int THREADS>
struct Select {
  static constexpr int kWarps = THREADS / 32;
  static constexpr int kKeys = THREADS * 32;
  static constexpr int kCopies = THREADS == 1024 ? 8 : 4;
  static constexpr int kBins = 2048;
  static constexpr int kList = (kCopies - 1) * kBins;   // in the other copies' place
  static constexpr int kSmem = (kKeys + kCopies * kBins) * 4;
};

// Exclusive sum of v over the CTA's threads.
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) before += w < warp ? warp_sums[w] : 0;
  __syncthreads();
  return before + s - v;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  using S = Select<THREADS>;
  extern __shared__ uint32_t smem[];
  uint32_t* keys = smem;
  int* hist = reinterpret_cast<int*>(smem + S::kKeys);
  uint32_t* list = smem + S::kKeys + S::kBins;
  __shared__ int warp_sums[S::kWarps];
  __shared__ int warp_gt[S::kWarps], warp_eq[S::kWarps];
  __shared__ int s_bin, s_left, s_count, s_listed;
  griddep_launch_dependents();   // the move may do its prologue
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  const int L = checked_len(a, b, h == 0 && tid == 0);
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  const bool cut = L > a.keep;
  if (h == 0) {
    if (tid == 0) a.new_lens[b] = cut ? a.keep : L;
    if (a.tables_out != nullptr)
      for (int i = tid; i < a.spare_blocks; i += THREADS)
        a.tables_out[static_cast<int64_t>(b) * a.spare_blocks + i] =
            cut ? a.spare[static_cast<int64_t>(b) * a.spare_blocks + i]
                : i < a.mbs ? a.block_tables[static_cast<int64_t>(b) * a.mbs + i] : -1;
  }
  const float* w = a.weights + unit * a.stride;
  float* w_out = a.weights_out != nullptr ? a.weights_out + unit * a.out_stride : nullptr;
  int32_t* kept = a.kept + unit * a.keep;
  // the protected ends, or, uncut, everything
  const int head = cut ? a.first : L, tail = cut ? a.recent : 0;
  for (int i = tid; i < head + tail; i += THREADS) {
    const int t = i < head ? i : L - tail + (i - head);
    const int pos = i < head ? i : a.keep - tail + (i - head);
    kept[pos] = t;
    if (w_out != nullptr) w_out[pos] = w[t];
  }
  const int k = a.keep - a.first - a.recent;   // how many of the m candidates stay; k < m
  if (!cut || k == 0) return;
  const int m = L - a.first - a.recent;
  const float* cand = w + a.first;
  const int part = ((m + S::kWarps - 1) / S::kWarps + 31) / 32 * 32;
  const int lo = min(warp * part, m), hi = min(lo + part, m);
  for (int i = tid; i < S::kCopies * S::kBins; i += THREADS) hist[i] = 0;
  if (tid == 0) s_listed = 0;
  __syncthreads();
  // ---- the first digit, and the keys into shared memory
  for (int i0 = lo; i0 < hi; i0 += 8 * 32) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i0 + j * 32 + lane < hi ? __ldg(cand + i0 + j * 32 + lane) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * 32 + lane;
      if (i < hi) {
        const uint32_t key = weight_key(v[j]);
        if (i < S::kKeys) keys[i] = key;
        atomicAdd(&hist[(key >> 21) * S::kCopies + (lane & (S::kCopies - 1))], 1);
      }
    }
  }
  __syncthreads();
  auto key_at = [&](int i) { return i < S::kKeys ? keys[i] : weight_key(__ldg(cand + i)); };
  // Finds the bin, from the largest down, in which the left-th key lies.
  int left = k;
  auto find_bin = [&](int bins, int copies) {
    const int each = bins / THREADS > 0 ? bins / THREADS : 1;
    int c[S::kBins / THREADS > 0 ? S::kBins / THREADS : 1];
    int sum = 0;
#pragma unroll
    for (int j = 0; j < S::kBins / THREADS; ++j) {
      c[j] = 0;
      const int bin = bins - 1 - (tid * each + j);
      if (j < each && bin >= 0)
        for (int x = 0; x < copies; ++x) c[j] += hist[bin * copies + x];
      sum += c[j];
    }
    int above = block_scan<S::kWarps>(sum, warp_sums);
    if (above < left && above + sum >= left) {
#pragma unroll
      for (int j = 0; j < S::kBins / THREADS; ++j) {
        if (above < left && above + c[j] >= left) {
          s_bin = bins - 1 - (tid * each + j);
          s_left = left - above;
          s_count = c[j];
        }
        above += c[j];
      }
    }
    __syncthreads();
    left = s_left;
  };
  find_bin(S::kBins, S::kCopies);
  uint32_t prefix = static_cast<uint32_t>(s_bin) << 21;
  const int count = s_count;
  const bool listed = count <= S::kList;
  __syncthreads();
  // ---- the other digits, on the keys of that bin
  if (listed) {
    for (int i = lo + lane; i - lane < hi; i += 32) {
      const uint32_t key = i < hi ? key_at(i) : 0u;
      const bool in = i < hi && (key >> 21) == (prefix >> 21);
      const unsigned mask = __ballot_sync(0xffffffffu, in);
      if (mask == 0) continue;
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_listed, __popc(mask));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1));
      if (in) list[at] = key;
    }
  }
#pragma unroll
  for (int digit = 0; digit < 2; ++digit) {
    const int shift = digit == 0 ? 10 : 0, bins = digit == 0 ? 2048 : 1024;
    for (int i = tid; i < S::kBins; i += THREADS) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = digit == 0 ? 0xffe00000u : 0xfffffc00u;
    if (listed) {
      for (int i = tid; i < count; i += THREADS)
        if ((list[i] & mask) == prefix) atomicAdd(&hist[(list[i] >> shift) & (bins - 1)], 1);
    } else {
      for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t key = key_at(i);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
      }
    }
    __syncthreads();
    find_bin(bins, 1);
    prefix |= static_cast<uint32_t>(s_bin) << shift;
    __syncthreads();
  }
  // ---- every warp's larger keys and ties, then the positions in order
  int gt = 0, eq = 0;
  for (int i = lo + lane; i < hi; i += 32) {
    const uint32_t key = key_at(i);
    gt += key > prefix;
    eq += key == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) warp_gt[warp] = gt, warp_eq[warp] = eq;
  __syncthreads();
  int gt_before = lane < warp && lane < S::kWarps ? warp_gt[lane] : 0;
  int ties = lane < warp && lane < S::kWarps ? warp_eq[lane] : 0;
  gt_before = __reduce_add_sync(0xffffffffu, gt_before);
  ties = __reduce_add_sync(0xffffffffu, ties);
  int pos = a.first + gt_before + min(ties, left);
  const unsigned below = (1u << lane) - 1;
  for (int i = lo + lane; i - lane < hi; i += 32) {
    const uint32_t key = i < hi ? key_at(i) : 0u;
    const unsigned tied = __ballot_sync(0xffffffffu, i < hi && key == prefix);
    const bool stay = i < hi && (key > prefix ||
                                 (key == prefix && ties + __popc(tied & below) < left));
    const unsigned staying = __ballot_sync(0xffffffffu, stay);
    if (stay) {
      const int at = pos + __popc(staying & below);
      kept[at] = a.first + i;
      if (w_out != nullptr) w_out[at] = __ldg(cand + i);
    }
    pos += __popc(staying);
    ties += __popc(tied);
  }
}

// --------------------------------------------------------------------- move
// One CTA per (two or four destination pages, kv head, sequence).  A thread
// moves one 16-byte chunk of K and of V of two pages; all four loads are made
// before the stores.
constexpr int kMoveThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int C = D / 8;                          // 16-byte chunks a row
  constexpr int kPages = kMoveThreads / (16 * C);   // that the CTA's threads cover at once
  const int h = blockIdx.y, b = blockIdx.z;
  const int L = checked_len(a, b, false);
  const int row = threadIdx.x / C % 16, c = threadIdx.x % C;
  int dst[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int page = (blockIdx.x * 2 + j) * kPages + threadIdx.x / (16 * C);
    dst[j] = -1;
    if (L > a.keep && page * 16 + row < a.keep) {
      dst[j] = __ldg(a.spare + static_cast<int64_t>(b) * a.spare_blocks + page);
      if (dst[j] < 0 || dst[j] >= a.num_blocks) {
        atomicOr(a.status, kStatusBadBlock);
        dst[j] = -1;
      }
    }
  }
  griddep_wait();   // the kept positions are written
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  int t[2], src[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int page = (blockIdx.x * 2 + j) * kPages + threadIdx.x / (16 * C);
    t[j] = dst[j] >= 0 ? a.kept[unit * a.keep + page * 16 + row] : 0;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    src[j] = dst[j] >= 0 ? __ldg(a.block_tables + static_cast<int64_t>(b) * a.mbs + t[j] / 16) : 0;
    if (src[j] < 0 || src[j] >= a.num_blocks) {
      atomicOr(a.status, kStatusBadBlock);
      dst[j] = -1;
    }
  }
  uint4 kv[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (dst[j] < 0) continue;
    const int64_t from = ((static_cast<int64_t>(src[j]) * a.Hkv + h) * 16 + t[j] % 16) * C + c;
    kv[j][0] = __ldcs(static_cast<const uint4*>(a.k_cache) + from);
    kv[j][1] = __ldcs(static_cast<const uint4*>(a.v_cache) + from);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (dst[j] < 0) continue;
    const int64_t to = ((static_cast<int64_t>(dst[j]) * a.Hkv + h) * 16 + row) * C + c;
    static_cast<uint4*>(a.k_cache)[to] = kv[j][0];
    static_cast<uint4*>(a.v_cache)[to] = kv[j][1];
  }
}

// E4M3 codes of x / scale, the quotient rounded to fp32 as the division rounds it,
// without dividing: x * (1 / scale) is within two steps of it, and where that is
// not near a border between two codes (the 20 bits of the significand that a code
// drops stand at their half), the code is the same.  Near one, and below the
// smallest normal code, it does divide.
struct Encoder {
  float scale, inv;
  bool divide;   // the reciprocal itself would leave fp32's normal range
  static __device__ __forceinline__ Encoder of(float s) {
    return Encoder{s, __fdiv_rn(1.f, s), !(s > 0x1p-100f && s < 0x1p100f)};
  }
  __device__ __forceinline__ uint32_t operator()(float x, float y) const {
    const float p = __fmul_rn(x, inv), q = __fmul_rn(y, inv);
    if (divide || doubtful(p) || doubtful(q))
      return f32x2_to_e4m3x2(__fdiv_rn(x, scale), __fdiv_rn(y, scale));
    return f32x2_to_e4m3x2(p, q);
  }
  static __device__ __forceinline__ bool doubtful(float q) {
    const uint32_t b = __float_as_uint(q);
    const bool border = (b + 4u - 0x80000u) * 4096u <= 8u * 4096u;
    const bool small = (b & 0x7fffffffu) - 1u < 0x3c800000u - 1u;   // 0 < |q| < 2^-6
    return border || small;
  }
};

// E4M3: one warp per (destination page, kv head, sequence, K|V).  A page's scale
// is that of the rows it now holds, so all of them are read before any is written.
constexpr int kMoveE4m3Warps = 4;

template <int D>
__global__ void __launch_bounds__(kMoveE4m3Warps * 32)
evict_move_e4m3_kernel(const __grid_constant__ EvictArgs a) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, kv = threadIdx.x >> 5 & 1;
  const int page = blockIdx.x * (kMoveE4m3Warps / 2) + (threadIdx.x >> 6);
  const int L = checked_len(a, b, false);
  const int rows = min(16, a.keep - page * 16);
  const bool live = L > a.keep && rows > 0;
  const int dst = live ? __ldg(a.spare + static_cast<int64_t>(b) * a.spare_blocks + page) : 0;
  griddep_wait();   // the kept positions are written
  if (!live) return;
  if (dst < 0 || dst >= a.num_blocks) {
    if (lane == 0) atomicOr(a.status, kStatusBadBlock);
    return;
  }
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  uint8_t* pool = static_cast<uint8_t*>(kv ? a.v_cache : a.k_cache);
  float* scales = kv ? a.v_scale : a.k_scale;
  // lane j holds row j's source
  int64_t src_row = -1;
  float src_scale = 0.f;
  if (lane < rows) {
    const int t = a.kept[unit * a.keep + page * 16 + lane];
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
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int64_t r = __shfl_sync(0xffffffffu, src_row, j);
    codes[j] = r >= 0 ? load_row_codes<D>(pool + r * D, lane) : 0u;
  }
  auto value2 = [&](uint32_t two, float scale) {
    const uint32_t f = e4m3x2_to_f16x2(two);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
    return make_float2(__fmul_rn(v.x, scale), __fmul_rn(v.y, scale));
  };
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float s = __shfl_sync(0xffffffffu, src_scale, j);
    const float2 v = value2(codes[j] & 0xffffu, s);
    amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
    if constexpr (P == 4) {
      const float2 u = value2(codes[j] >> 16, s);
      amax = fmaxf(amax, fmaxf(fabsf(u.x), fabsf(u.y)));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const Encoder encode = Encoder::of(e4m3_page_scale(amax));
  const int64_t tile = static_cast<int64_t>(dst) * a.Hkv + h;
  if (lane == 0) scales[tile] = encode.scale;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float s = __shfl_sync(0xffffffffu, src_scale, j);
    if (__shfl_sync(0xffffffffu, src_row, j) < 0) continue;   // behind the last row, or skipped
    const float2 v = value2(codes[j] & 0xffffu, s);
    uint32_t c = encode(v.x, v.y);
    if constexpr (P == 4) {
      const float2 u = value2(codes[j] >> 16, s);
      c |= encode(u.x, u.y) << 16;
    }
    store_row_codes<D>(pool + (tile * 16 + j) * D, lane, c);
  }
}

template <int THREADS>
cudaError_t launch_select(const EvictArgs& a, cudaStream_t s) {
  using S = Select<THREADS>;
  {
    // more than 48 KB of shared memory has to be asked for, once per device
    static std::mutex mu;
    static bool raised[kMaxDevices] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!raised[dev]) {
      if (cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<THREADS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem))
        return e;
      raised[dev] = true;
    }
  }
  evict_select_kernel<THREADS><<<dim3(a.Hkv, a.B), THREADS, S::kSmem, s>>>(a);
  return cudaGetLastError();
}

template <typename Kernel>
cudaError_t launch_move(Kernel* kernel, const EvictArgs& a, int pages, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(((a.keep + 15) / 16 + pages - 1) / pages, a.Hkv, a.B);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, bool fp8, cudaStream_t s) {
  // 8 warps select among up to 8192 candidates (three CTAs an SM), 32 among more
  if (cudaError_t e = a.max_context_len <= Select<256>::kKeys ? launch_select<256>(a, s)
                                                              : launch_select<1024>(a, s))
    return e;
  if (fp8)
    return launch_move(a.D == 128 ? evict_move_e4m3_kernel<128> : evict_move_e4m3_kernel<64>, a,
                       kMoveE4m3Warps / 2, kMoveE4m3Warps * 32, s);
  return a.D == 128 ? launch_move(evict_move_kernel<128>, a, 2, kMoveThreads, s)
                    : launch_move(evict_move_kernel<64>, a, 4, kMoveThreads, s);
}

}  // namespace pa
