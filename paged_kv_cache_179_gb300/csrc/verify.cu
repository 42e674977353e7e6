// verify.cu -- verification of drafted tokens against the target's probabilities.
//
// Draft x_i is accepted while u_i q_i(x_i) < p_i(x_i); at the first rejection r
// the next token is drawn from max(p_r - q_r, 0), else from p_n, as the lowest
// token whose cumulative sum exceeds u times the total.
//
// The sums are made in 64-bit fixed point (2^-61): integer addition is
// associative, so any split of the vocabulary gives the same token, a border
// between two tokens is as sharp as in 64-bit floating point, and the GPU's
// slow fp64 units are not used.  p - q is the difference of the two fixed-point
// values, so it is not rounded either.
//
// Bytes: one row of p and one of q per sequence; which ones is known only after
// the drafts' own probabilities have been read.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// A probability: negative values and NaN are 0, values above 2 are 2.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, 0.f), 2.f); }
__device__ __forceinline__ uint64_t fixed61(float x) {
  return static_cast<uint64_t>(__float2ll_rn(clean(x) * 0x1p61f));
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The weight that token j is drawn with.
template <typename T>
struct Row {
  const T* p;
  const T* q;       // null: nothing is taken off p, except at `spike`
  int spike;        // token whose weight is max(p - 1, 0) (a draft without probabilities), or -1
  __device__ __forceinline__ uint64_t at(int j) const {
    const uint64_t fp = fixed61(to_f32(p[j]));
    uint64_t fq = q != nullptr ? fixed61(to_f32(q[j])) : 0;
    if (j == spike) fq = uint64_t(1) << 61;
    return fp > fq ? fp - fq : 0;
  }
};

// floor(u * total) for u in [0, 1): the token drawn is the first whose
// cumulative sum is larger.
__device__ __forceinline__ uint64_t threshold(float u, uint64_t total) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return total;
  const uint64_t f = static_cast<uint64_t>(__float2ull_rz(u * 0x1p63f)) << 1;   // exact to 2^-63
  return __umul64hi(f, total);
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads)
verify_kernel(const VerifyArgs a) {
  __shared__ uint64_t sums[kVerifyWarps];
  __shared__ int first_reject;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x;
  int32_t* out = a.out_tokens + static_cast<int64_t>(b) * (a.n + 1);
  const float* u = a.uniforms + static_cast<int64_t>(b) * (a.n + 1);
  const int nb = a.num_drafts != nullptr ? __ldg(a.num_drafts + b) : a.n;
  if (nb < 0 || nb > a.n) {
    for (int i = tid; i <= a.n; i += kVerifyThreads) out[i] = -1;
    if (tid == 0) {
      a.num_accepted[b] = 0;
      atomicOr(a.status, kStatusBadLen);
    }
    return;
  }
  if (tid == 0) first_reject = nb;
  __syncthreads();
  const T* p = static_cast<const T*>(a.p) + static_cast<int64_t>(b) * (a.n + 1) * a.p_stride;
  const T* q = a.q == nullptr ? nullptr
             : static_cast<const T*>(a.q) + static_cast<int64_t>(b) * a.n * a.q_stride;
  for (int i = tid; i < nb; i += kVerifyThreads) {
    const int x = __ldg(a.draft_tokens + static_cast<int64_t>(b) * a.n + i);
    bool ok = x >= 0 && x < a.V;
    if (!ok) {
      atomicOr(a.status, kStatusBadToken);
    } else {
      const float px = clean(to_f32(p[i * a.p_stride + x]));
      const float qx = q != nullptr ? clean(to_f32(q[i * a.q_stride + x])) : 1.f;
      ok = static_cast<double>(u[i]) * static_cast<double>(qx) < static_cast<double>(px);
    }
    if (!ok) atomicMin(&first_reject, i);
  }
  __syncthreads();
  const int r = first_reject;
  Row<T> row;
  row.p = p + r * a.p_stride;
  row.q = r < nb && q != nullptr ? q + r * a.q_stride : nullptr;
  row.spike = r < nb && q == nullptr ? __ldg(a.draft_tokens + static_cast<int64_t>(b) * a.n + r) : -1;
  // each warp sums a contiguous part of the vocabulary
  const int part = (a.V + kVerifyWarps - 1) / kVerifyWarps;
  const int j0 = min(warp * part, a.V), j1 = min(j0 + part, a.V);
  uint64_t total;
  while (true) {
    uint64_t sum = 0;
    for (int j = j0 + lane; j < j1; j += 32) sum += row.at(j);
    sum = warp_sum(sum);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kVerifyWarps; ++w) total += sums[w];
    if (total != 0 || (row.q == nullptr && row.spike < 0)) break;
    row.q = nullptr;    // nothing left of p - q: drawn from p
    row.spike = -1;
    __syncthreads();
  }
  for (int i = tid; i <= a.n; i += kVerifyThreads)
    if (i != r) out[i] = i < r ? __ldg(a.draft_tokens + static_cast<int64_t>(b) * a.n + i) : -1;
  if (tid == 0) a.num_accepted[b] = r;
  const uint64_t thr = threshold(u[a.n], total);
  // the warp whose part holds the border looks for it; a u of 1 or more draws
  // the last token that has any weight
  const uint64_t want = thr < total ? thr : total - 1;
  if (total == 0) {
    if (tid == 0) out[r] = -1;
    return;
  }
  uint64_t before = 0;
  int w = 0;
  while (w < kVerifyWarps - 1 && before + sums[w] <= want) before += sums[w++];
  if (warp != w) return;
  for (int j = j0; j < j1; j += 32) {
    const uint64_t v = j + lane < j1 ? row.at(j + lane) : 0;
    const uint64_t cdf = before + warp_scan(v, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, cdf > want);
    if (hit != 0) {
      if (lane == 0) out[r] = j + __ffs(hit) - 1;
      return;
    }
    before = __shfl_sync(0xffffffffu, cdf, 31);
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
  auto* kernel = dtype == 0 ? verify_kernel<__half>
               : dtype == 1 ? verify_kernel<__nv_bfloat16> : verify_kernel<float>;
  kernel<<<static_cast<unsigned>(a.B), kVerifyThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace pa
