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
// once; only two words a warp cross the cluster, its maximum and the sum of its
// exponentials relative to it.  The row after the first of a sequence adds one
// draft to the counts.
//
// Where there are rows enough for all SMs and histories are short, a CTA makes a row by
// itself (stream_kernel): the tokens that something is known of, a few thousand at most,
// are in a hash table and a bitmap; they are made first, one by one, and the rest of the
// row streams past them, twice for probabilities (the second time from L2).  Nothing
// waits for other CTAs then.
//
// Bound by memory where there are many rows, by latency where there are few.  Measured on a
// GB300, rows of 128000 bf16 logits to fp32 probabilities, biases and a grammar's mask: 512
// rows with histories of 4096 tokens 147 us, 2.7 TB/s of what is read and written once (a
// copy of those bytes would take 59 us): 35 us are the histories' insertion, the rest two
// rounds of two CTAs an SM.  The same by clusters takes 310 us.  To logits 77 us.  One
// row of 32000 fp32 logits: 6 us.
//
// Counts are integers, a token's biases are added in their order, and what is summed by
// slots of the hash table, whose tokens' places depend on who came first, is summed in whole
// numbers, so results do not depend on the order of execution.
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

// A token's word w (its count, and what else is known) and logit v: the adjusted logit.
// `e` is what the biases' list calls the token.
struct Penalties {
  float rep, inv_rep, freq, pres;
  __device__ explicit Penalties(const pa_logits_spec& sp, int b) {
    rep = sp.repetition != nullptr ? sp.repetition[b] : 1.f;
    inv_rep = 1.f / rep;
    freq = sp.frequency != nullptr ? sp.frequency[b] : 0.f;
    pres = sp.presence != nullptr ? sp.presence[b] : 0.f;
  }
  __device__ float adjust(float v, unsigned w, int e, const int* bias_t, const float* bias_v,
                          int n_bias) const {
    const unsigned count = w & kCount;
    if (count != 0u || (w & kInPrompt)) {
      // the quotient by the reciprocal, corrected by its remainder (where both are finite)
      const float q = v * inv_rep;
      v = v > 0.f ? (q < 1e37f ? fmaf(fmaf(-q, rep, v), inv_rep, q) : v / rep) : v * rep;
    }
    if (count != 0u) v -= fmaf(freq, static_cast<float>(count), pres);
    if (w & kHasBias) {
      float s = 0.f;
      for (int j = 0; j < n_bias; ++j)
        if (bias_t[j] == e) s += bias_v[j];
      v += s;
    }
    return v;
  }
};
// exp(d / T) = 2^(c d); c stays finite and above 0, so 0 c and -inf c are what they should be
__device__ __forceinline__ float exponent_factor(float temp) {
  return fminf(fmaxf(1.4426950408889634f / temp, 1e-37f), 3.4e38f);
}

template <typename T>
struct alignas(sizeof(T) * kVec) Pack {
  T v[kVec];
};

template <typename T, bool PROBS, bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
logits_kernel(const LogitsArgs a, int slice, int rows_per_unit) {
  using O = std::conditional_t<PROBS, float, T>;
  constexpr int kSteps = kPer / kVec, kWarps = THREADS / 32;
  extern __shared__ __align__(16) unsigned seen[];   // [slice]
  __shared__ int bias_t[kLogitsMaxBias];
  __shared__ float bias_v[kLogitsMaxBias];
  __shared__ int n_bias;
  __shared__ unsigned red_i[kWarps];
  // of each warp of the cluster: its maximum and sum, and its lowest token there
  __shared__ float2 box[2][PROBS ? kMaxCluster * kWarps : 1];
  __shared__ unsigned box_i[2][PROBS ? kMaxCluster * kWarps : 1];
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
  // Value q of thread tid is element e_q: q / 4 steps of all threads' four consecutive ones
  // (WIDE) or q steps of all threads; tokens go in equal steps, too.
  auto token = [&](int e) { return ((((e >> 7) << shift) + rank) << 7) + (e & 127); };
  constexpr int kStep = WIDE ? THREADS * kVec : THREADS;
  const int e0 = WIDE ? tid * kVec : tid, t0 = token(e0), t_step = kStep << shift;
  auto element_at = [&](int q) { return WIDE ? e0 + q / kVec * kStep + q % kVec : e0 + q * kStep; };
  auto token_at = [&](int q) { return WIDE ? t0 + q / kVec * t_step + q % kVec : t0 + q * t_step; };
  // the element of a token, or -1: another CTA's (or padding)
  auto element_of = [&](int t) {
    return t >= 0 && ((t >> 7) & (C - 1)) == rank ? ((t >> (7 + shift)) << 7) + (t & 127) : -1;
  };
  if (PROBS) cluster_arrive();                     // (this CTA has started)
  // ---- the history's counts in this slice
  for (int j = tid; j < slice / 4; j += THREADS)
    reinterpret_cast<uint4*>(seen)[j] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) n_bias = 0;
  griddep_wait();                                  // (nothing of memory was touched before)
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
    for (int j0 = tid; j0 < L; j0 += 8 * THREADS) {   // eight loads in flight
      int t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = h[min(j0 + u * THREADS, L - 1)];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u * THREADS < L) add(t[u], j0 + u * THREADS < P);
    }
  }
  if (sp.draft_tokens != nullptr)
    for (int j = tid; j < i0; j += THREADS)
      add(sp.draft_tokens[static_cast<int64_t>(b) * (a.rows - 1) + j], false);
  for (int j0 = 0; j0 < sp.num_bias; j0 += THREADS) {   // this CTA's biases, in their order
    const int j = j0 + tid;
    const int64_t at = static_cast<int64_t>(b) * sp.num_bias + j;
    const int t = j < sp.num_bias ? sp.bias_tokens[at] : -1;
    const float v = j < sp.num_bias ? sp.bias_values[at] : 0.f;
    if (t >= a.V && rank == 0) atomicOr(a.status, kStatusBadToken);
    const int e = t < a.V ? element_of(t) : -1;
    const unsigned m = __ballot_sync(0xffffffffu, e >= 0);
    if (lane == 0) red_i[warp] = __popc(m);
    __syncthreads();
    int to = n_bias + __popc(m & ((1u << lane) - 1u)), all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) to += red_i[w];
      all += red_i[w];
    }
    if (e >= 0) {
      bias_t[to] = e;
      bias_v[to] = v;
      atomicOr(seen + e, kHasBias);
    }
    __syncthreads();
    if (tid == 0) n_bias += all;
    __syncthreads();
  }
  const Penalties pen(sp, b);
  const float temp = sp.temperature != nullptr ? sp.temperature[b] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float c = exponent_factor(temp);
  // A row's logits: all loads at once, none of them behind a branch (what lies behind the
  // row's end is read from its end, and replaced when it is used).
  Pack<T> raw[kSteps];
  auto load = [&](int i) {
    const T* in = static_cast<const T*>(a.logits) + (static_cast<int64_t>(b) * a.rows + i) * a.in_stride;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if constexpr (WIDE) {
        raw[k] = *reinterpret_cast<const Pack<T>*>(in + min(token_at(k * kVec), (a.V - kVec) & ~(kVec - 1)));
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) raw[k].v[j] = in[min(token_at(k * kVec + j), a.V - 1)];
      }
    }
  };
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
    load(i);
    float x[kPer];
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int q = k * kVec + j;
        x[q] = to_f32(raw[k].v[j]);
        if (!WIDE && token_at(q) >= a.V) x[q] = -INFINITY;
      }
    if (WIDE && token_at(kPer - kVec) + kVec > a.V) {   // behind the row's end, or the last few before it
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int t = token_at(q), whole = token_at(q / kVec * kVec) + kVec;
        if (whole > a.V) x[q] = t < a.V ? to_f32(in[t]) : -INFINITY;
      }
    }
    auto adjust = [&](int e, unsigned w, float v) {   // a token that something is known of
      return pen.adjust(v, w, e, bias_t, bias_v, n_bias);
    };
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if constexpr (WIDE) {
        const int e = element_at(k * kVec), t = token_at(k * kVec);
        if (t >= a.V) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(seen + e);
        // (four tokens share a word of the mask)
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
        for (int q = k * kVec; q < (k + 1) * kVec; ++q) {
          const int e = element_at(q), t = token_at(q);
          if (t >= a.V) continue;
          const unsigned w = seen[e];
          if (w != 0u) x[q] = adjust(e, w, x[q]);
          if (allowed != nullptr && !((allowed[t >> 5] >> (t & 31)) & 1u)) x[q] = -INFINITY;
        }
      }
    }
    if constexpr (PROBS) {
      // ---- the warp's maximum, and the exponentials relative to it
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < kPer; ++q) m = fmaxf(m, x[q]);   // (fmaxf passes NaN over)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int set = i & 1;                       // (two sets: a CTA is at most a row ahead)
      float sum = 0.f;
      if (greedy) {                                // the lowest token at the maximum
        unsigned best = 0xffffffffu;
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (x[q] == m && m > -INFINITY) best = min(best, static_cast<unsigned>(token_at(q)));
        best = __reduce_min_sync(0xffffffffu, best);
        if (lane < C) st_cluster_u32(&box_i[set][rank * kWarps + warp], lane, best);
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
      // ---- across the cluster: one barrier a row
      if (lane < C) {
        st_cluster_f32(&box[set][rank * kWarps + warp].x, lane, m);
        st_cluster_f32(&box[set][rank * kWarps + warp].y, lane, sum);
      }
      cluster_sync();
      float M = -INFINITY;
      for (int r = lane; r < C * kWarps; r += 32) M = fmaxf(M, box[set][r].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      if (greedy) {
        unsigned best = 0xffffffffu;
        for (int r = lane; r < C * kWarps; r += 32)
          if (box[set][r].x == M) best = min(best, box_i[set][r]);
        best = __reduce_min_sync(0xffffffffu, best);
#pragma unroll
        for (int q = 0; q < kPer; ++q) x[q] = static_cast<unsigned>(token_at(q)) == best ? 1.f : 0.f;
      } else {
        auto factor = [&](float mr) {              // 2^(c (mr - M)); all of them -inf: 0
          return mr == M ? (M > -INFINITY ? 1.f : 0.f) : fast_exp2((mr - M) * c);
        };
        float total = 0.f;                         // (lane by lane, then across: one order)
        for (int r = lane; r < C * kWarps; r += 32) total += box[set][r].y * factor(box[set][r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const float scale = total > 0.f ? factor(m) / total : 0.f;
#pragma unroll
        for (int q = 0; q < kPer; ++q) x[q] *= scale;
      }
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int t = token_at(k * kVec);
      if (WIDE && t + kVec <= a.V) {
        Pack<O> p;
#pragma unroll
        for (int j = 0; j < kVec; ++j) from_f32(x[k * kVec + j], &p.v[j]);
        *reinterpret_cast<Pack<O>*>(out + t) = p;
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (token_at(k * kVec + j) < a.V) from_f32(x[k * kVec + j], out + token_at(k * kVec + j));
      }
    }
  }
}

// ------------------------------------------------------------- a CTA a row
constexpr int kStreamThreads = 512;
constexpr int kStreamSlots = 8192;                 // of the hash table, at most
constexpr int kStreamKnown = kStreamSlots * 3 / 4;   // tokens that it takes
constexpr int kStreamSteps = 4;                    // loads in flight, of 16 bytes each
template <typename T>
constexpr int kStreamVec = 16 / static_cast<int>(sizeof(T));
template <typename T>
struct alignas(16) Wide {
  T v[kStreamVec<T>];
};

template <typename T, bool PROBS>
__global__ void __launch_bounds__(kStreamThreads, 2)
stream_kernel(const LogitsArgs a, int log_slots) {
  using O = std::conditional_t<PROBS, float, T>;
  constexpr int kVec = kStreamVec<T>, kSteps = kStreamSteps;
  constexpr unsigned kAll = (1u << kVec) - 1u;
  constexpr int kWarps = kStreamThreads / 32, kChunk = kStreamThreads * kVec;
  extern __shared__ __align__(16) unsigned known[];   // a bit a token, then the table
  __shared__ int bias_t[kLogitsMaxBias];
  __shared__ float bias_v[kLogitsMaxBias];
  __shared__ float red_m[kWarps], red_s[kWarps];
  __shared__ unsigned red_i[kWarps];
  __shared__ unsigned long long red_u[kWarps];
  const pa_logits_spec& sp = a.spec;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / a.rows, i = blockIdx.x - b * a.rows;
  const int words = (a.V + 127) / 128 * 4, slots = 1 << log_slots;
  int* keys = reinterpret_cast<int*>(known + words);
  unsigned* vals = reinterpret_cast<unsigned*>(keys + slots);   // words, later the adjusted logits
  for (int j = tid; j < words / 4; j += kStreamThreads)
    reinterpret_cast<uint4*>(known)[j] = make_uint4(0u, 0u, 0u, 0u);
  for (int j = tid; j < slots / 4; j += kStreamThreads) {
    reinterpret_cast<int4*>(keys)[j] = make_int4(-1, -1, -1, -1);
    reinterpret_cast<uint4*>(vals)[j] = make_uint4(0u, 0u, 0u, 0u);
  }
  griddep_wait();                                  // (nothing of memory was touched before)
  __syncthreads();
  // A token's slot (more slots than tokens: one is found).  Most tokens of a text are there
  // already, so a slot is read before it is asked for.
  auto slot_of = [&](int t) {
    unsigned h = (static_cast<unsigned>(t) * 2654435761u) >> (32 - log_slots);
    for (;;) {
      int k = *reinterpret_cast<volatile int*>(keys + h);
      if (k == -1) {
        k = atomicCAS(keys + h, -1, t);
        if (k == -1) atomicOr(known + (t >> 5), 1u << (t & 31));
      }
      if (k == -1 || k == t) return h;
      h = (h + 1) & (slots - 1);
    }
  };
  auto valid = [&](int t) {
    if (t >= a.V) atomicOr(a.status, kStatusBadToken);
    return t >= 0 && t < a.V;
  };
  auto add = [&](int t, bool prompt) {
    if (!valid(t)) return;
    unsigned* v = vals + slot_of(t);
    if (prompt) atomicOr(v, kInPrompt);
    else atomicAdd(v, 1u);
  };
  if (sp.history != nullptr) {
    int L = sp.history_lens[b];
    if (L < 0 || L > sp.history_stride) {
      if (tid == 0) atomicOr(a.status, kStatusBadLen);
      L = 0;
    }
    const int P = sp.prompt_lens != nullptr ? sp.prompt_lens[b] : 0;
    const int32_t* h = sp.history + b * sp.history_stride;
    for (int j0 = tid; j0 < L; j0 += 8 * kStreamThreads) {   // eight loads in flight
      int t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = h[min(j0 + u * kStreamThreads, L - 1)];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u * kStreamThreads < L) add(t[u], j0 + u * kStreamThreads < P);
    }
  }
  if (sp.draft_tokens != nullptr)
    for (int j = tid; j < i; j += kStreamThreads)
      add(sp.draft_tokens[static_cast<int64_t>(b) * (a.rows - 1) + j], false);
  for (int j = tid; j < sp.num_bias; j += kStreamThreads) {
    const int t = sp.bias_tokens[static_cast<int64_t>(b) * sp.num_bias + j];
    bias_t[j] = t;
    bias_v[j] = sp.bias_values[static_cast<int64_t>(b) * sp.num_bias + j];
    if (!valid(t)) continue;
    atomicOr(vals + slot_of(t), kHasBias);
  }
  const Penalties pen(sp, b);
  const float temp = sp.temperature != nullptr ? sp.temperature[b] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float c = exponent_factor(temp);
  const int64_t row = static_cast<int64_t>(b) * a.rows + i;
  const T* in = static_cast<const T*>(a.logits) + row * a.in_stride;
  O* out = static_cast<O*>(a.out) + row * a.out_stride;
  const uint32_t* allowed = sp.allowed != nullptr ? sp.allowed + row * sp.allowed_stride : nullptr;
  __syncthreads();
  // A thread's maximum, and its sum of exponentials relative to it (or lowest token there).
  float m = -INFINITY, sum = 0.f;
  unsigned best = 0xffffffffu;
  auto take = [&](float x, int t) {                // one more value
    if (!(x > -INFINITY)) return;                  // (a NaN counts as -inf)
    if (greedy) {
      if (x > m || (x == m && static_cast<unsigned>(t) < best)) best = t;
      m = fmaxf(m, x);
    } else if (x > m) {
      sum = sum * fast_exp2((m - x) * c) + 1.f;
      m = x;
    } else {
      sum += x == m ? 1.f : fast_exp2((x - m) * c);
    }
  };
  // ---- the known tokens
  for (int j0 = tid; j0 < slots; j0 += 8 * kStreamThreads) {   // eight loads in flight
    int key[8];
    T v[8];
    unsigned ok[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) key[u] = j0 + u * kStreamThreads < slots ? keys[j0 + u * kStreamThreads] : -1;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int t = max(key[u], 0);
      v[u] = in[t];
      ok[u] = allowed != nullptr ? allowed[t >> 5] >> (t & 31) : 1u;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (key[u] < 0) continue;
      unsigned* w = vals + j0 + u * kStreamThreads;
      const float x = ok[u] & 1u ? pen.adjust(to_f32(v[u]), *w, key[u], bias_t, bias_v, sp.num_bias) : -INFINITY;
      *w = __float_as_uint(x);
      if (PROBS && greedy) take(x, key[u]);
      else if (PROBS) m = fmaxf(m, x);             // (passes NaN over)
    }
  }
  if (PROBS && !greedy) {
    // Their sum.  Which slot a token has, and so which thread, depends on who came first; whole
    // numbers add up to the same in any order.  Relative to the largest of them, in units of
    // 2^-40: each is off by half a unit, 6144 of them by 2^-28 of a sum that is 1 at least.
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red_m[warp] = m;
    __syncthreads();
    m = red_m[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, red_m[w]);
    unsigned long long units = 0u;
    if (m > -INFINITY) {
      for (int j = tid; j < slots; j += kStreamThreads) {   // (this thread's own, as above)
        const float x = __uint_as_float(vals[j]);
        if (keys[j] < 0 || !(x > -INFINITY)) continue;
        units += __float2ull_rn((x == m ? 1.f : fast_exp2((x - m) * c)) * 0x1p40f);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
    if (lane == 0) red_u[warp] = units;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) units += red_u[w];
      sum = __ull2float_rn(units) * 0x1p-40f;
    } else {
      m = -INFINITY;
    }
  }
  __syncthreads();                                 // (in place, the rest is written over them)
  // ---- the rest: kSteps loads in flight, none of them behind a branch
  const int last = (a.V - kVec) & ~(kVec - 1);
  auto load = [&](int t0, bool again, Wide<T> (&raw)[kSteps], unsigned (&bits)[kSteps]) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const uint4* at = reinterpret_cast<const uint4*>(in + min(t0 + k * kChunk, last));
      // (a row that is read a second time is not needed any more)
      const uint4 x = again ? __ldcs(at) : *at;
      raw[k] = reinterpret_cast<const Wide<T>&>(x);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {             // bit j: token t + j is there and allowed
      const int t = t0 + k * kChunk, at = min(t, last);
      bits[k] = (allowed != nullptr ? allowed[at >> 5] >> (at & 31) : kAll) & (t <= last ? kAll : 0u);
    }
  };
  if (PROBS) {
    for (int t0 = tid * kVec; t0 < a.V; t0 += kSteps * kChunk) {
      Wide<T> raw[kSteps];
      unsigned bits[kSteps];
      load(t0, false, raw, bits);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int t = t0 + k * kChunk;
        const unsigned ok = bits[k] & ~(known[min(t, last) >> 5] >> (t & 31));
        float x[kVec], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          x[j] = (ok >> j) & 1u ? fmaxf(to_f32(raw[k].v[j]), -INFINITY) : -INFINITY;
          top = fmaxf(top, x[j]);
        }
        if (greedy || top == INFINITY) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) take(x[j], t + j);
          continue;
        }
        if (top > m) {
          sum *= fast_exp2((m - top) * c);
          m = top;
        }
        if (m > -INFINITY) {
          float part[2] = {0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kVec; ++j) part[j & 1] += fast_exp2((x[j] - m) * c);
          sum += part[0] + part[1];
        }
      }
    }
    for (int t = last + kVec + tid; t < a.V; t += kStreamThreads) {   // the last few, one by one
      const bool ok = !((known[t >> 5] >> (t & 31)) & 1u) &&
                      (allowed == nullptr || ((allowed[t >> 5] >> (t & 31)) & 1u));
      if (ok) take(to_f32(in[t]), t);
    }
    // ---- over the CTA, in one order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, sum, o);
      const unsigned ob = __shfl_xor_sync(0xffffffffu, best, o);
      const float top = fmaxf(m, om);
      if (greedy) best = m == om ? min(best, ob) : om > m ? ob : best;
      else if (top > -INFINITY)
        sum = sum * (m == top ? 1.f : fast_exp2((m - top) * c)) + os * (om == top ? 1.f : fast_exp2((om - top) * c));
      m = top;
    }
    if (lane == 0) {
      red_m[warp] = m;
      red_s[warp] = sum;
      red_i[warp] = best;
    }
    __syncthreads();
    m = red_m[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, red_m[w]);
    sum = 0.f;
    best = 0xffffffffu;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (red_m[w] == m) best = min(best, red_i[w]);
      if (m > -INFINITY) sum += red_s[w] * (red_m[w] == m ? 1.f : fast_exp2((red_m[w] - m) * c));
    }
  }
  const float scale = PROBS && sum > 0.f ? 1.f / sum : 0.f;
  auto result = [&](float x, int t) {              // of an adjusted logit (-inf: masked)
    if (!PROBS) return x;
    if (greedy) return static_cast<unsigned>(t) == best ? 1.f : 0.f;
    if (!(x > -INFINITY)) return 0.f;              // (a NaN counts as -inf)
    return x == m ? scale : fast_exp2((x - m) * c) * scale;
  };
  const bool plain = !greedy && fabsf(m) < INFINITY;   // exp(0) at the maximum, 0 at -inf
  for (int t0 = tid * kVec; t0 < a.V; t0 += kSteps * kChunk) {
    Wide<T> raw[kSteps];
    unsigned bits[kSteps];
    load(t0, PROBS, raw, bits);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int t = t0 + k * kChunk;
      if (t > last) continue;
      struct alignas(16) {
        O v[kVec];
      } r;
      if (PROBS && plain) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {           // (fmaxf: a NaN counts as -inf)
          const float x = (bits[k] >> j) & 1u ? fmaxf(to_f32(raw[k].v[j]), -INFINITY) : -INFINITY;
          from_f32(fast_exp2((x - m) * c) * scale, &r.v[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          from_f32(result((bits[k] >> j) & 1u ? to_f32(raw[k].v[j]) : -INFINITY, t + j), &r.v[j]);
      }
      // (past what the other rows read again)
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(r) / 16); ++j)
        __stcs(reinterpret_cast<uint4*>(out + t) + j, reinterpret_cast<const uint4*>(&r)[j]);
    }
  }
  for (int t = last + kVec + tid; t < a.V; t += kStreamThreads) {
    const bool ok = allowed == nullptr || ((allowed[t >> 5] >> (t & 31)) & 1u);
    from_f32(result(ok ? to_f32(in[t]) : -INFINITY, t), out + t);
  }
  __syncthreads();                                 // the known tokens over what stands there now
  for (int j = tid; j < slots; j += kStreamThreads)
    if (keys[j] >= 0) from_f32(result(__uint_as_float(vals[j]), keys[j]), out + keys[j]);
}

template <typename T, bool PROBS>
cudaError_t launch_stream(const LogitsArgs& a, int64_t known, cudaStream_t s) {
  auto* kern = stream_kernel<T, PROBS>;
  int log_slots = 6;
  while ((1 << log_slots) * 3 / 4 < known) ++log_slots;
  const size_t smem = static_cast<size_t>((a.V + 127) / 128) * 16 + (size_t{8} << log_slots);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (kLogitsMaxVocab + 127) / 128 * 16 + kStreamSlots * 8);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(static_cast<unsigned>(a.B * a.rows)), kStreamThreads, smem, s, a, log_slots);
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
  cudaLaunchAttribute attr[2];
  attr[0] = after_previous();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, slice, rows_per_unit);
}

template <typename T>
cudaError_t launch_type(const LogitsArgs& a, bool probs, cudaStream_t s) {
  const size_t out_size = probs ? 4 : sizeof(T);
  // rows that begin at a multiple of kVec elements are read kVec at a time
  const bool wide = a.V >= kVec && (a.in_stride % kVec) == 0 && (a.out_stride % kVec) == 0 &&
                    reinterpret_cast<uintptr_t>(a.out) % (out_size * kVec) == 0;
  // tokens that something may be known of in a row
  const int64_t known = (a.spec.history != nullptr ? a.spec.history_stride : 0) + a.spec.num_bias + a.rows;
  // From a row for every second SM on (third, for logits) a CTA makes a row by itself.  Rows of
  // 128000 bf16 logits with histories of 4096 tokens, by clusters and by a CTA a row: to
  // probabilities 64 rows 50 and 57 us, 96 rows 72 and 58; to logits 32 rows 19 and 30 us,
  // 64 rows 35 and 30.
  const bool aligned = a.V >= kStreamVec<T> && a.in_stride * sizeof(T) % 16 == 0 && a.out_stride * out_size % 16 == 0;
  if (aligned && static_cast<int64_t>(a.B) * a.rows >= (probs ? 76 : 48) && known <= kStreamKnown)
    return probs ? launch_stream<T, true>(a, known, s) : launch_stream<T, false>(a, known, s);
  // as few CTAs a row as hold it, more where there are not enough rows for the SMs
  const int blocks = (a.V + 127) / 128;
  const bool large = blocks > kMaxCluster * (512 * kPer / 128);
  const int most = (large ? 1024 : 512) * kPer / 128;   // blocks a CTA
  int C = 1;
  while (C < kMaxCluster &&
         (blocks > C * most || (C < blocks && static_cast<int64_t>(a.B) * a.rows * C < 152)))
    C *= 2;
  const int slice = (blocks + C - 1) / C * 128;
  // a unit is a sequence's rows, whose counts differ by a draft each, or one row
  const int per_unit = static_cast<int64_t>(a.B) * C >= 608 ? a.rows : 1;
  if (large) {
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
