// logits.cu -- penalties for repeated tokens, biases and grammar masks on logits,
// and the softmax that draft verification draws from.
//
//   x = logit; seen: x > 0 ? x / r : x r; x -= f c + p (c > 0); x += bias; masked: -inf
//   out = x, or exp((x - max) / T) / sum
//
// One cluster of CTAs holds the rows of a sequence (or one row), its CTAs taking the
// vocabulary's blocks of 128 tokens in turn (the tokens that text repeats are low ones: a
// contiguous share of them would be one CTA's, and the others would wait): their
// counts of the sequence's history in shared memory (one word a token: the output's
// count, and whether the prompt or a bias has it), a row's logits in registers, 32 a
// thread.  So a row is read once and written
// once; only two words a CTA cross the cluster, each CTA's maximum and the sum of
// its exponentials relative to it.  The row after the first of a sequence adds one
// draft to the counts.
//
// Counts are integers, and a token's biases are added in their order, so results
// do not depend on the order of execution.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_cluster.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "request_launch.h"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kPer = 32;                           // logits a thread holds
constexpr int kVec = 4;                            // consecutive ones, where rows are aligned
constexpr int kMaxCluster = 16;
constexpr unsigned kInPrompt = 1u << 31, kHasBias = 1u << 30, kCount = kHasBias - 1u;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* o) { *o = x; }
__device__ __forceinline__ void from_f32(float x, __half* o) { *o = __float2half_rn(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* o) { *o = __float2bfloat16_rn(x); }

__device__ __forceinline__ void st_cluster_f32(void* p, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(in_cluster(p, rank)), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cluster(p, rank)), "r"(v) : "memory");
}

template <typename T>
struct alignas(sizeof(T) * kVec) Pack {
  T v[kVec];
};

// VEC elements of a slice: element j of step k of thread t.
template <bool WIDE, int THREADS>
__device__ __forceinline__ int element(int k, int j, int t) {
  return WIDE ? (k * THREADS + t) * kVec + j : (k * kVec + j) * THREADS + t;
}

template <typename T, bool PROBS, bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
logits_kernel(const LogitsArgs a, int slice, int rows_per_unit) {
  using O = std::conditional_t<PROBS, float, T>;
  constexpr int kSteps = kPer / kVec, kWarps = THREADS / 32;
  extern __shared__ __align__(16) unsigned seen[];   // [slice]
  __shared__ int bias_t[kLogitsMaxBias];
  __shared__ float bias_v[kLogitsMaxBias];
  __shared__ int n_bias;
  __shared__ float red_m[kWarps], red_s[kWarps];
  __shared__ unsigned red_i[kWarps];
  __shared__ float box_m[2][kMaxCluster], box_s[2][kMaxCluster];
  __shared__ unsigned box_i[2][kMaxCluster];
  const pa_logits_spec& sp = a.spec;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(cluster_size());
  const int rank = static_cast<int>(cluster_rank());
  const int units = (a.rows + rows_per_unit - 1) / rows_per_unit;   // of a sequence
  const int unit = blockIdx.x / C;
  const int b = unit / units, i0 = (unit - b * units) * rows_per_unit;
  const int i1 = min(i0 + rows_per_unit, a.rows);
  // this CTA's element e is token ((e / 128) C + rank) 128 + e % 128 (C a power of two)
  const int shift = __ffs(C) - 1;
  auto token = [&](int e) { return ((((e >> 7) << shift) + rank) << 7) + (e & 127); };
  // the element of a token, or -1: another CTA's (or padding)
  auto element_of = [&](int t) {
    return t >= 0 && ((t >> 7) & (C - 1)) == rank ? ((t >> (7 + shift)) << 7) + (t & 127) : -1;
  };
  if (PROBS) cluster_arrive();                     // (this CTA has started)
  // ---- the history's counts in this slice
  for (int j = tid; j < slice / 4; j += THREADS)
    reinterpret_cast<uint4*>(seen)[j] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) n_bias = 0;
  __syncthreads();
  auto add = [&](int t, bool prompt) {
    if (t >= a.V) {
      if (rank == 0) atomicOr(a.status, kStatusBadToken);
      return;
    }
    const int e = element_of(t);
    if (e < 0) return;
    if (prompt) atomicOr(seen + e, kInPrompt);
    else atomicAdd(seen + e, 1u);
  };
  if (sp.history != nullptr) {
    int L = sp.history_lens[b];
    if (L < 0 || L > sp.history_stride) {
      if (tid == 0) atomicOr(a.status, kStatusBadLen);
      L = 0;
    }
    const int P = sp.prompt_lens != nullptr ? sp.prompt_lens[b] : 0;
    const int32_t* h = sp.history + b * sp.history_stride;
    for (int j = tid; j < L; j += THREADS) add(h[j], j < P);
  }
  if (sp.draft_tokens != nullptr)
    for (int j = tid; j < i0; j += THREADS)
      add(sp.draft_tokens[static_cast<int64_t>(b) * (a.rows - 1) + j], false);
  if (sp.bias_tokens != nullptr && warp == 0) {    // this slice's biases, in their order
    int kept = 0;
    for (int j = lane; j - lane < sp.num_bias; j += 32) {
      const bool in = j < sp.num_bias;
      const int t = in ? sp.bias_tokens[static_cast<int64_t>(b) * sp.num_bias + j] : -1;
      if (t >= a.V && rank == 0) atomicOr(a.status, kStatusBadToken);
      const int e = t < a.V ? element_of(t) : -1;
      const bool ours = e >= 0;
      const unsigned m = __ballot_sync(0xffffffffu, ours);
      if (ours) {
        const int at = kept + __popc(m & ((1u << lane) - 1u));
        bias_t[at] = e;
        bias_v[at] = sp.bias_values[static_cast<int64_t>(b) * sp.num_bias + j];
        atomicOr(seen + e, kHasBias);
      }
      kept += __popc(m);
    }
    if (lane == 0) n_bias = kept;
  }
  const float rep = sp.repetition != nullptr ? sp.repetition[b] : 1.f, inv_rep = 1.f / rep;
  const float freq = sp.frequency != nullptr ? sp.frequency[b] : 0.f;
  const float pres = sp.presence != nullptr ? sp.presence[b] : 0.f;
  const float temp = sp.temperature != nullptr ? sp.temperature[b] : 1.f;
  const bool greedy = !(temp > 0.f);
  // exp(d / T) = 2^(c d); c stays finite and above 0, so 0 c and -inf c are what they should be
  const float c = fminf(fmaxf(1.4426950408889634f / temp, 1e-37f), 3.4e38f);
  __syncthreads();
  if (PROBS) cluster_wait();

  for (int i = i0; i < i1; ++i) {
    if (i > i0 && sp.draft_tokens != nullptr) {    // one more draft is output now
      __syncthreads();
      if (tid == 0) add(sp.draft_tokens[static_cast<int64_t>(b) * (a.rows - 1) + i - 1], false);
      __syncthreads();
    }
    const int64_t row = static_cast<int64_t>(b) * a.rows + i;
    const T* in = static_cast<const T*>(a.logits) + row * a.in_stride;
    O* out = static_cast<O*>(a.out) + row * a.out_stride;
    const uint32_t* allowed = sp.allowed != nullptr ? sp.allowed + row * sp.allowed_stride : nullptr;
    float x[kPer];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if constexpr (WIDE) {
        const int t = token(element<WIDE, THREADS>(k, 0, tid));
        if (t + kVec <= a.V) {
          const Pack<T> p = *reinterpret_cast<const Pack<T>*>(in + t);
#pragma unroll
          for (int j = 0; j < kVec; ++j) x[k * kVec + j] = to_f32(p.v[j]);
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int t = token(element<WIDE, THREADS>(k, j, tid));
        x[k * kVec + j] = t < a.V ? to_f32(in[t]) : -INFINITY;
      }
    }
    auto adjust = [&](int e, unsigned w, float v) {   // a token that something is known of
      const unsigned count = w & kCount;
      if (count != 0u || (w & kInPrompt)) {
        // the quotient by the reciprocal, corrected by its remainder
        const float q = v * inv_rep;
        v = v > 0.f ? (v < INFINITY ? fmaf(fmaf(-q, rep, v), inv_rep, q) : v / rep) : v * rep;
      }
      if (count != 0u) v -= fmaf(freq, static_cast<float>(count), pres);
      if (w & kHasBias) {
        float s = 0.f;
        for (int j = 0; j < n_bias; ++j)
          if (bias_t[j] == e) s += bias_v[j];
        v += s;
      }
      return v;
    };
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if constexpr (WIDE) {
        const int e = element<WIDE, THREADS>(k, 0, tid);
        const int t = token(e);
        if (t >= a.V) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(seen + e);
        const unsigned ok = allowed != nullptr ? allowed[t >> 5] >> (t & 31) : ~0u;
        if ((w.x | w.y | w.z | w.w) != 0u) {
          if (w.x != 0u) x[k * kVec] = adjust(e, w.x, x[k * kVec]);
          if (w.y != 0u) x[k * kVec + 1] = adjust(e + 1, w.y, x[k * kVec + 1]);
          if (w.z != 0u) x[k * kVec + 2] = adjust(e + 2, w.z, x[k * kVec + 2]);
          if (w.w != 0u) x[k * kVec + 3] = adjust(e + 3, w.w, x[k * kVec + 3]);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (!((ok >> j) & 1u)) x[k * kVec + j] = -INFINITY;
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const int e = element<WIDE, THREADS>(k, j, tid), q = k * kVec + j;
          const int t = token(e);
          if (t >= a.V) continue;
          const unsigned w = seen[e];
          if (w != 0u) x[q] = adjust(e, w, x[q]);
          if (allowed != nullptr && !((allowed[t >> 5] >> (t & 31)) & 1u)) x[q] = -INFINITY;
        }
      }
    }
    if constexpr (PROBS) {
      // ---- this CTA's maximum, then the exponentials relative to it
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < kPer; ++q) m = fmaxf(m, x[q]);   // (fmaxf passes NaN over)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) red_m[warp] = m;
      __syncthreads();
      m = red_m[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, red_m[w]);
      float sum = 0.f;
      unsigned best = 0xffffffffu;                 // the lowest token at the maximum
      if (greedy) {
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (x[q] == m && m > -INFINITY)
            best = min(best, static_cast<unsigned>(token(element<WIDE, THREADS>(q / kVec, q % kVec, tid))));
        best = __reduce_min_sync(0xffffffffu, best);
      } else {
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const float d = x[q] == m ? 0.f : x[q] - m;
          // m = -inf: nothing is there; a NaN counts as -inf
          x[q] = m > -INFINITY && d <= 0.f ? fast_exp2(d * c) : 0.f;
          sum += x[q];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      if (lane == 0) {
        red_s[warp] = sum;
        red_i[warp] = best;
      }
      __syncthreads();
      sum = 0.f;
      best = 0xffffffffu;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sum += red_s[w];
        best = min(best, red_i[w]);
      }
      // ---- across the cluster (two sets of boxes: a CTA is at most a row ahead)
      const int set = i & 1;
      if (tid < C) {
        st_cluster_f32(&box_m[set][rank], tid, m);
        st_cluster_f32(&box_s[set][rank], tid, sum);
        st_cluster_u32(&box_i[set][rank], tid, best);
      }
      cluster_sync();
      float M = -INFINITY, total = 0.f;
      for (int r = 0; r < C; ++r) M = fmaxf(M, box_m[set][r]);
      if (greedy) {
        best = 0xffffffffu;
        for (int r = 0; r < C; ++r)
          if (box_m[set][r] == M) best = min(best, box_i[set][r]);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          x[q] = static_cast<unsigned>(token(element<WIDE, THREADS>(q / kVec, q % kVec, tid))) == best ? 1.f : 0.f;
      } else {
        auto factor = [&](float mr) {              // 2^(c (mr - M)); all of them -inf: 0
          return mr == M ? (M > -INFINITY ? 1.f : 0.f) : fast_exp2((mr - M) * c);
        };
        for (int r = 0; r < C; ++r) total += box_s[set][r] * factor(box_m[set][r]);
        const float scale = total > 0.f ? factor(m) / total : 0.f;
#pragma unroll
        for (int q = 0; q < kPer; ++q) x[q] *= scale;
      }
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if constexpr (WIDE) {
        const int t = token(element<WIDE, THREADS>(k, 0, tid));
        if (t + kVec <= a.V) {
          Pack<O> p;
#pragma unroll
          for (int j = 0; j < kVec; ++j) from_f32(x[k * kVec + j], &p.v[j]);
          *reinterpret_cast<Pack<O>*>(out + t) = p;
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int t = token(element<WIDE, THREADS>(k, j, tid));
        if (t < a.V) from_f32(x[k * kVec + j], out + t);
      }
    }
  }
}

template <typename T, bool PROBS, bool WIDE, int THREADS>
cudaError_t launch(const LogitsArgs& a, int C, int slice, int rows_per_unit, cudaStream_t s) {
  auto* kern = logits_kernel<T, PROBS, WIDE, THREADS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       THREADS * kPer * 4);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int units = (a.rows + rows_per_unit - 1) / rows_per_unit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(a.B) * units * C));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(slice) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, slice, rows_per_unit);
}

template <typename T>
cudaError_t launch_type(const LogitsArgs& a, bool probs, cudaStream_t s) {
  const size_t out_size = probs ? 4 : sizeof(T);
  // rows that begin at a multiple of kVec elements are read kVec at a time
  const bool wide = (a.in_stride % kVec) == 0 && (a.out_stride % kVec) == 0 &&
                    reinterpret_cast<uintptr_t>(a.out) % (out_size * kVec) == 0;
  int C = 1;
  const int blocks = (a.V + 127) / 128;
  while (C < kMaxCluster &&
         (blocks > C * (512 * kPer / 128) || (C < blocks && static_cast<int64_t>(a.B) * a.rows * C < 152)))
    C *= 2;
  const int slice = (blocks + C - 1) / C * 128;
  const bool big = slice > 512 * kPer;
  const int per_unit = static_cast<int64_t>(a.B) * C >= 608 ? a.rows : 1;
  if (big) {
    if (probs) return wide ? launch<T, true, true, 1024>(a, C, slice, per_unit, s)
                           : launch<T, true, false, 1024>(a, C, slice, per_unit, s);
    return wide ? launch<T, false, true, 1024>(a, C, slice, per_unit, s)
                : launch<T, false, false, 1024>(a, C, slice, per_unit, s);
  }
  if (probs) return wide ? launch<T, true, true, 512>(a, C, slice, per_unit, s)
                         : launch<T, true, false, 512>(a, C, slice, per_unit, s);
  return wide ? launch<T, false, true, 512>(a, C, slice, per_unit, s)
              : launch<T, false, false, 512>(a, C, slice, per_unit, s);
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs& a, int dtype, bool probs, cudaStream_t s) {
  return dtype == PA_F16    ? launch_type<__half>(a, probs, s)
         : dtype == PA_BF16 ? launch_type<__nv_bfloat16>(a, probs, s)
                            : launch_type<float>(a, probs, s);
}

}  // namespace pa
