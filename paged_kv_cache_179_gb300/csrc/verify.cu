// verify.cu -- verification of drafted tokens against the target's probabilities.
//
// Draft x_i is accepted while u_i q_i(x_i) < p_i(x_i); at the first rejection r
// the next token is drawn from max(p_r - q_r, 0), else from p_n, as the lowest
// token whose cumulative sum exceeds u times the total.
//
// The sums are made in 64-bit fixed point (2^-60): integer addition is
// associative, so any split of the vocabulary gives the same token, a border
// between two tokens is as sharp as in 64-bit floating point, and the GPU's
// slow fp64 units are not used.  p - q is the difference of the two fixed-point
// values, so it is not rounded either.
//
// Bytes: one row of p and one of q per sequence; which ones is known only after
// the drafts' own probabilities have been read.  Measured on a GB300: 33 us for
// 128 sequences of 128000 fp32 tokens with draft probabilities (131 MB, 58 % of
// the measured copy bandwidth), 8.2 us for one sequence of 32000: that much is
// the chain launch, drafts, their probabilities, row, cluster barrier, border.
// CTAs of 256 threads at 32 registers, eight an SM (six: 39 us; 512 threads 40 us),
// 16 bytes a lane (4 bytes, four in flight: 35 us; 32 bytes at 40 registers: 35 us);
// one CTA a sequence 195 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_cluster.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;

// Stores v at the address that `p` (this CTA's shared memory) has in CTA `rank`.
__device__ __forceinline__ void st_cluster(void* p, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cluster(p, rank)), "l"(v) : "memory");
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Fixed point, in units of 2^-60.  The weight of a token is fix(x) - fix(y) with
// x = p, y = min(p, q), so it is never negative and nothing has to be selected.
//
// fix() works in three limbs of 20 bits on the floating-point pipe: adding C1 =
// 12 (one step of whose binade is 2^-20) rounds x to that step, and the bits of
// the sum are the limb plus those of C1; the rest x - (t - C1) is exact and goes
// to C2 (steps of 2^-40), then C3 (2^-60).  The limbs of x and y are accumulated
// as integers, s += bits(t_x) - bits(t_y), in which C's own bits cancel.  The
// integer pipe, which runs at half the rate, was what bounded the shifts that a
// conversion by exponent needs (nine operations a value).
constexpr float kC1 = 12.f, kC2 = 1.5f * 0x1p-17f, kC3 = 1.5f * 0x1p-37f;

// A probability: negative values and NaN are 0, values above 2 are 2.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, 0.f), 2.f); }

struct Limbs {
  int a = 0, b = 0, c = 0;   // steps of 2^-20, 2^-40, 2^-60
  // += fix(x) - fix(y), for x and y in [0, 2]
  __device__ __forceinline__ void add(float x, float y) {
    const float x1 = __fadd_rn(x, kC1), y1 = __fadd_rn(y, kC1);
    a += __float_as_int(x1) - __float_as_int(y1);
    x = __fsub_rn(x, __fsub_rn(x1, kC1));
    y = __fsub_rn(y, __fsub_rn(y1, kC1));
    const float x2 = __fadd_rn(x, kC2), y2 = __fadd_rn(y, kC2);
    b += __float_as_int(x2) - __float_as_int(y2);
    x = __fsub_rn(x, __fsub_rn(x2, kC2));
    y = __fsub_rn(y, __fsub_rn(y2, kC2));
    c += __float_as_int(__fadd_rn(x, kC3)) - __float_as_int(__fadd_rn(y, kC3));
  }
  // A limb of one token is below 2^21 + 1 in size, and those of b and c may all
  // have one sign: 32 bits hold the sum of 512 tokens whatever they are.
  __device__ __forceinline__ uint64_t value() const {
    return (static_cast<uint64_t>(static_cast<int64_t>(a)) << 40) +
           (static_cast<uint64_t>(static_cast<int64_t>(b)) << 20) +
           static_cast<uint64_t>(static_cast<int64_t>(c));
  }
};

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

// The row a token is drawn from: weight of j is max(p_j - q_j, 0).
template <typename T>
struct Row {
  const T* p;
  const T* q;       // null: nothing is taken off p, except at `spike`
  int spike;        // a draft without probabilities: 1 is taken off there; or -1
  bool wide;        // both rows begin at a multiple of 16 bytes
  __device__ __forceinline__ uint64_t at(int j) const {
    const float x = clean(to_f32(p[j]));
    Limbs w;
    w.add(x, fminf(x, q != nullptr ? clean(to_f32(q[j])) : j == spike ? 1.f : 0.f));
    return w.value();
  }
  // adds tokens j, j + 32, ... (N of them) without the spike; all loads first
  template <int N>
  __device__ __forceinline__ void add(int j, Limbs& w) const {
    T x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = p[j + 32 * i];
    if (q != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = q[j + 32 * i];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float v = clean(to_f32(x[i]));
        w.add(v, fminf(v, fmaxf(to_f32(y[i]), 0.f)));   // a q above 2 is above p, too
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w.add(clean(to_f32(x[i])), 0.f);
    }
  }
  // the same for the 16 bytes of tokens from j on
  static constexpr int kWide = 16 / sizeof(T);
  __device__ __forceinline__ void add_wide(int j, Limbs& w) const {
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p + j));
    uint4 y = make_uint4(0, 0, 0, 0);
    if (q != nullptr) y = __ldcs(reinterpret_cast<const uint4*>(q + j));
    const T* px = reinterpret_cast<const T*>(&x);
    const T* qx = reinterpret_cast<const T*>(&y);
#pragma unroll
    for (int e = 0; e < kWide; ++e) {
      const float v = clean(to_f32(px[e]));
      w.add(v, q != nullptr ? fminf(v, fmaxf(to_f32(qx[e]), 0.f)) : 0.f);
    }
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

constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;

// Sum of the weights of tokens [from, hi), taken by one warp (all lanes get it):
// 16 bytes a lane where the rows' alignment allows it, then, or for rows that begin
// anywhere, one element a lane, kUnroll of them in flight.
template <typename T>
__device__ __forceinline__ uint64_t warp_range_sum(const Row<T>& row, int from, int hi, int lane) {
  int lo = from;
  uint64_t sum = 0;
  if (row.wide) {   // lo is a multiple of 8 tokens
    constexpr int kStep = 32 * Row<T>::kWide;   // of a warp
    while (lo + kStep <= hi) {
      Limbs w;
      for (int i = 0; i < 512 / Row<T>::kWide && lo + kStep <= hi; ++i, lo += kStep)
        row.add_wide(lo + lane * Row<T>::kWide, w);
      sum += w.value();
    }
  }
  int j = lo + lane;
  constexpr int kBatch = kUnroll * 32;
  while (j + kBatch - 32 < hi) {
    Limbs w;
    for (int i = 0; i < 512 / kUnroll && j + kBatch - 32 < hi; ++i, j += kBatch)
      row.template add<kUnroll>(j, w);
    sum += w.value();
  }
  Limbs w;
  for (; j < hi; j += 32) row.template add<1>(j, w);
  sum += w.value();
  if (lane == 0 && from <= row.spike && row.spike < hi) {   // what 1 takes off the spike
    const float x = clean(to_f32(row.p[row.spike]));
    Limbs s;
    s.add(fminf(x, 1.f), 0.f);
    sum -= s.value();
  }
  return warp_sum(sum);
}

// A cluster of CTAs serves one sequence.  Every CTA makes the acceptance tests
// for itself and sums its part of the chosen row, a sub-part a warp; the warps'
// sums go to every CTA of the cluster through distributed shared memory; the
// CTA whose part holds the border narrows it down, re-reading (from L2) one
// warp's sub-part at a time.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 8)
verify_kernel(const VerifyArgs a) {
  __shared__ uint64_t sums[2][kMaxCluster * kVerifyWarps];
  __shared__ uint64_t level[kVerifyWarps];
  __shared__ int first_reject;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
  const int b = blockIdx.x / size;
  int32_t* out = a.out_tokens + static_cast<int64_t>(b) * (a.n + 1);
  const int32_t* drafts = a.draft_tokens + static_cast<int64_t>(b) * a.n;
  const float* u = a.uniforms + static_cast<int64_t>(b) * (a.n + 1);
  const int x0 = tid < a.n ? __ldg(drafts + tid) : 0;   // asked for beside num_drafts
  const float u_draw = __ldg(u + a.n);
  const int nb = a.num_drafts != nullptr ? __ldg(a.num_drafts + b) : a.n;
  if (nb < 0 || nb > a.n) {   // the whole cluster leaves
    if (rank != 0) return;
    for (int i = tid; i <= a.n; i += kVerifyThreads) out[i] = -1;
    if (tid == 0) {
      a.num_accepted[b] = 0;
      atomicOr(a.status, kStatusBadLen);
    }
    return;
  }
  // every CTA of the cluster has begun before another one stores into it
  if (size > 1) cluster_arrive();
  if (tid == 0) first_reject = nb;
  __syncthreads();
  const T* p = static_cast<const T*>(a.p) + static_cast<int64_t>(b) * (a.n + 1) * a.p_stride;
  const T* q = a.q == nullptr ? nullptr
             : static_cast<const T*>(a.q) + static_cast<int64_t>(b) * a.n * a.q_stride;
  for (int i = tid; i < nb; i += kVerifyThreads) {
    const int x = i == tid ? x0 : __ldg(drafts + i);
    bool ok = x >= 0 && x < a.V;
    if (ok) {
      const float px = clean(to_f32(p[i * a.p_stride + x]));
      const float qx = q != nullptr ? clean(to_f32(q[i * a.q_stride + x])) : 1.f;
      ok = static_cast<double>(u[i]) * static_cast<double>(qx) < static_cast<double>(px);
    } else if (rank == 0) {
      atomicOr(a.status, kStatusBadToken);
    }
    if (!ok) atomicMin(&first_reject, i);
  }
  __syncthreads();
  const int r = first_reject;
  Row<T> row;
  row.p = p + r * a.p_stride;
  row.q = r < nb && q != nullptr ? q + r * a.q_stride : nullptr;
  row.spike = r < nb && q == nullptr ? __ldg(drafts + r) : -1;
  row.wide = a.p_stride * sizeof(T) % 16 == 0 && (row.q == nullptr || a.q_stride * sizeof(T) % 16 == 0);
  if (rank == 0) {
    for (int i = tid; i <= a.n; i += kVerifyThreads)
      if (i != r) out[i] = i > r ? -1 : i == tid ? x0 : __ldg(drafts + i);
    if (tid == 0) a.num_accepted[b] = r;
  }
  // part i of the row's size * kVerifyWarps goes to warp i of the cluster
  const int parts = size * kVerifyWarps;
  const int len = ((a.V + parts - 1) / parts + 7) / 8 * 8;
  uint64_t total;
  const uint64_t* all = sums[0];
  for (int pass = 0;; ++pass) {
    const int mine = rank * kVerifyWarps + warp;
    const int lo = min(mine * static_cast<int64_t>(len), static_cast<int64_t>(a.V));
    const uint64_t sum = warp_range_sum(row, lo, min(lo + len, a.V), lane);
    if (size == 1) {
      if (lane == 0) sums[pass][mine] = sum;
      __syncthreads();
    } else {
      if (pass == 0) cluster_wait();
      if (lane < size) st_cluster(&sums[pass][mine], lane, sum);
      cluster_sync();
    }
    all = sums[pass];
    total = 0;
    for (int i = lane; i < parts; i += 32) total += all[i];
    total = warp_sum(total);
    if (total != 0 || pass == 1 || (row.q == nullptr && row.spike < 0)) break;
    row.q = nullptr;    // nothing is left of p - q: drawn from p
    row.spike = -1;
  }
  if (total == 0) {
    if (rank == 0 && tid == 0) out[r] = -1;
    return;
  }
  // the border's place; a u of 1 or more draws the last token that has weight
  const uint64_t thr = threshold(u_draw, total);
  uint64_t want = thr < total ? thr : total - 1;
  // the part that holds it (the same search in every warp of the cluster)
  int part = 0;
  {
    uint64_t before = 0;
    for (int i = 0; i < parts; i += 32) {
      const uint64_t v = i + lane < parts ? all[i + lane] : 0;
      const uint64_t cdf = before + warp_scan(v, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, cdf > want);
      if (hit != 0) {
        const int at = __ffs(hit) - 1;
        part = i + at;
        want -= __shfl_sync(0xffffffffu, cdf - v, at);
        break;
      }
      before = __shfl_sync(0xffffffffu, cdf, 31);
    }
  }
  if (part / kVerifyWarps != rank) return;
  int lo = part * len, hi = min(lo + len, a.V);
  constexpr int kEach = 4;
  while (hi - lo > kEach * kVerifyThreads) {   // a warp's share at a time
    const int step = ((hi - lo + kVerifyWarps - 1) / kVerifyWarps + 7) / 8 * 8;
    const int l0 = min(lo + warp * step, hi);
    const uint64_t sum = warp_range_sum(row, l0, min(l0 + step, hi), lane);
    if (lane == 0) level[warp] = sum;
    __syncthreads();
    int w = 0;
    while (w < kVerifyWarps - 1 && want >= level[w]) want -= level[w++];
    lo += w * step;
    hi = min(lo + step, hi);
    __syncthreads();
  }
  // kEach neighbouring tokens a thread
  uint64_t v[kEach], mine = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = lo + tid * kEach + i;
    v[i] = j < hi ? row.at(j) : 0;
    mine += v[i];
  }
  uint64_t before = warp_scan(mine, lane);
  if (lane == 31) level[warp] = before;
  __syncthreads();
  before -= mine;
  for (int w = 0; w < warp; ++w) before += level[w];
  if (before <= want && want < before + mine) {   // one thread's
    int j = lo + tid * kEach;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (want >= before && want < before + v[i]) out[r] = j + i;
      before += v[i];
    }
  }
}

// CTAs a sequence's row is divided among: up to eight (a portable cluster), as
// long as the GPU holds fewer than four an SM and each keeps 2048 tokens.
int verify_cluster(int B, int V) {
  int c = 1;
  while (c < kMaxCluster && static_cast<int64_t>(B) * c < 4 * device_sm_count() &&
         V / (2 * c) >= 2048)
    c *= 2;
  return c;
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
  const int c = verify_cluster(a.B, a.V);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * c);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = c;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
  return dtype == 0 ? launch<__half>(a, s) : dtype == 1 ? launch<__nv_bfloat16>(a, s)
                                                        : launch<float>(a, s);
}

}  // namespace pa
