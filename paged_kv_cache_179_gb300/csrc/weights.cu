// weights.cu -- the attention weight each cached token receives.
//
//   W[b][h][t] = old(t) + sum_r softmax_t(scale q_r . K_t)
// over the query rows r of (sequence b, kv head h): n_q tokens times the query
// group.  The weight of a token needs the softmax statistics of the whole
// context, so one cooperative launch works in two phases with a grid barrier
// between them:
//   score:  every page's logits by mma.sync (a page's 16 tokens are the 16 rows
//           of the MMA's A, the query rows its 8 columns) and, per partition and
//           row, the running (reference, sum);
//   finish: per row the statistics of the whole context, joined from those of
//           its partitions, then each token's weights summed over the rows.
// K is read once: 2 D bytes a token and kv head (D for E4M3) are the floor.  A
// warp keeps the logits of its first pages in shared memory (200 KB an SM) and
// those behind them in the workspace, where they mostly stay in L2.
//
// Work split: the pages of all (sequence, kv head) units form one line, divided
// evenly among the warps.  A warp's part of a unit is a partition.  Units and
// warps both grow along the line, so unit + warp numbers every partition
// uniquely, and a unit's partitions are consecutive.
//
// K goes from global memory straight into the MMA's registers.  A dot product
// does not care in which order the dimensions are summed, so lane (r, c) of a
// quad takes the 16-byte chunks c, c + 4, ... of rows r and r + 8, and q's
// fragments are loaded with the same permutation.
#include <mutex>

#include "pa_e4m3.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kPrefix = kWeightsMaxBatch + 1;
constexpr int kMaxWarps = 12;
// Warps of a CTA, CTAs an SM, and the pages whose logits a warp keeps in shared
// memory: up to 16 query rows keep 16 warps an SM; the fragments of 32 take 64
// registers, which leaves room for 12.
template <int NT>
struct Shape {
  static constexpr int kWarps = NT == 4 ? 12 : 8;
  static constexpr int kCtas = NT == 4 ? 1 : 2;
  static constexpr int kKept = NT == 1 ? 25 : NT == 2 ? 12 : 9;
  static constexpr int kPage = NT * 32;   // float4s of a page's logits
  static constexpr int kSmem = kWarps * kKept * kPage * 16;
};

// ------------------------------------------------------------ the line of pages
struct Line {
  int64_t n;        // pages of all units
  int workers;      // warps that have pages: each has at least one
};
__device__ __forceinline__ Line make_line(const WeightsArgs& a, const int* cum, int warps) {
  const int64_t n = static_cast<int64_t>(cum[a.B]) * a.Hkv;
  return Line{n, static_cast<int>(n < warps ? n : warps)};
}
// The pages worker w takes: [start(w), start(w + 1)).
__device__ __forceinline__ int64_t part_start(const Line& l, int w) {
  return l.n * w / l.workers;
}
// The worker that takes page x of the line.
__device__ __forceinline__ int part_of(const Line& l, int64_t x) {
  return static_cast<int>(((x + 1) * l.workers - 1) / l.n);
}

__device__ __forceinline__ int checked_len(const WeightsArgs& a, int b, bool report) {
  const int L = __ldg(a.context_lens + b);
  if (L < 0 || L > a.max_context_len || L > static_cast<int64_t>(a.mbs) * 16) {
    if (report) atomicOr(a.status, kStatusBadLen);
    return 0;
  }
  return L;
}

// cum[b] = pages of the sequences before b, cum[B] = all; by the whole CTA.
template <int WARPS>
__device__ __forceinline__ void prefix_pages(const WeightsArgs& a, int* cum, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int base = 0; base < a.B; base += WARPS * 32) {
    const int b = base + tid;
    const int v = b < a.B ? (checked_len(a, b, blockIdx.x == 0) + 15) / 16 : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += warp_sums[w];
      carry += warp_sums[w];
    }
    if (b < a.B) cum[b] = before + s - v;
    __syncthreads();
  }
  if (tid == 0) cum[a.B] = carry;
  __syncthreads();
}

// A place on the line: unit (b, h) and page within it.
struct Place {
  int b, h, page, pages;   // pages: of the unit
  int64_t unit_start;      // the unit's first page on the line
};
__device__ __forceinline__ Place find(const int* cum, int B, int Hkv, int64_t x) {
  int lo = 0, hi = B;      // the last b with cum[b] * Hkv <= x that has pages
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (static_cast<int64_t>(cum[mid]) * Hkv <= x) lo = mid;
    else hi = mid;
  }
  Place p;
  p.b = lo;
  p.pages = cum[lo + 1] - cum[lo];
  const int64_t in_seq = x - static_cast<int64_t>(cum[lo]) * Hkv;
  p.h = static_cast<int>(in_seq / p.pages);
  p.page = static_cast<int>(in_seq - static_cast<int64_t>(p.h) * p.pages);
  p.unit_start = x - p.page;
  return p;
}

// ------------------------------------------------------------------ workspace
// logits: per page of the line and tile of 8 query rows, one float4 a lane (the
// MMA's result fragment); statistics: per partition and row (max, sum), log2 units.
// barrier: the grid barrier's count and generation; the count is 0 between calls.
struct Work {
  uint32_t* barrier;
  float4* logits;
  float2* stats;
};
constexpr size_t kBarrierBytes = 256;
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// ----------------------------------------------------------------- K fragments
// KV: 0 fp16, 1 bf16, 2 E4M3 with fp16 q, 3 E4M3 with bf16 q.  E4M3 codes become
// fp16, exactly; a bf16 row of q then enters the fp16 product scaled by the power
// of two that brings its largest element into [2^14, 2^15).  Its 8 bits fit
// fp16's 11, and what falls below fp16's smallest step is 2^-39 of the largest.
template <int KV>
struct Kind {
  static constexpr bool kE4m3 = KV >= 2;
  static constexpr bool kBf16 = KV == 1;        // of the product
  static constexpr bool kScaledQ = KV == 3;
};

// The lane's part of one page: NLD 16-byte chunks of row r, then of row r + 8.
template <int D, int KV>
struct Page {
  static constexpr int NLD = D / (Kind<KV>::kE4m3 ? 64 : 32);
  uint4 lo[NLD], hi[NLD];
  float scale;     // of an E4M3 page
  __device__ __forceinline__ void load(const WeightsArgs& a, int id, int h, int lane) {
    constexpr int row_chunks = NLD * 4;
    const int64_t tile = static_cast<int64_t>(id) * a.Hkv + h;
    const uint4* p = static_cast<const uint4*>(a.k_cache) + tile * (16 * row_chunks) +
                     (lane >> 2) * row_chunks + (lane & 3);
#pragma unroll
    for (int j = 0; j < NLD; ++j) {
      lo[j] = __ldcs(p + 4 * j);
      hi[j] = __ldcs(p + 8 * row_chunks + 4 * j);
    }
    if constexpr (Kind<KV>::kE4m3) scale = __ldg(a.k_scale + tile);
  }
};

// The lane's part of 8 query rows: the elements its K chunks hold, of row lane / 4.
template <int D, int KV>
struct Query {
  uint32_t w[D / 16][2];   // b0, b1 of each of the D / 16 MMA steps
  // returns what the scores have to be multiplied by (1 unless q was scaled)
  __device__ __forceinline__ float load(const uint16_t* row, bool live, int lane) {
    constexpr int per = Kind<KV>::kE4m3 ? 16 : 8;    // elements of a K chunk
    constexpr int NLD = D / (4 * per);
#pragma unroll
    for (int j = 0; j < NLD; ++j) {
#pragma unroll
      for (int x = 0; x < per / 8; ++x) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live)
          v = __ldg(reinterpret_cast<const uint4*>(row + ((lane & 3) + 4 * j) * per + 8 * x));
        const int s = (j * per + 8 * x) / 4;         // two steps per 8 elements
        w[s][0] = v.x;
        w[s][1] = v.y;
        w[s + 1][0] = v.z;
        w[s + 1][1] = v.w;
      }
    }
    if constexpr (Kind<KV>::kScaledQ) {
      float amax = 0.f;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 v = bits2_to_float2<true>(w[s][i]);
          amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = max(static_cast<int>(__float_as_uint(amax) >> 23), 15);   // biased exponent
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 127 + 14 - e) << 23);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 v = bits2_to_float2<true>(w[s][i]);
          w[s][i] = pack2<false>(v.x * up, v.y * up);
        }
      return __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
    }
    return 1.f;
  }
};

template <int D, int KV, int NT>
__device__ __forceinline__ void page_scores(float (&acc)[NT][4], const Page<D, KV>& k,
                                            const Query<D, KV> (&q)[NT]) {
  constexpr bool BF16 = Kind<KV>::kBf16;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
#pragma unroll
  for (int j = 0; j < Page<D, KV>::NLD; ++j) {
    const uint32_t lo[4] = {k.lo[j].x, k.lo[j].y, k.lo[j].z, k.lo[j].w};
    const uint32_t hi[4] = {k.hi[j].x, k.hi[j].y, k.hi[j].z, k.hi[j].w};
    if constexpr (Kind<KV>::kE4m3) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = e4m3x2_to_f16x2(lo[i] & 0xffffu), a2 = e4m3x2_to_f16x2(lo[i] >> 16);
        const uint32_t a1 = e4m3x2_to_f16x2(hi[i] & 0xffffu), a3 = e4m3x2_to_f16x2(hi[i] >> 16);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma16816<BF16>(acc[t], a0, a1, a2, a3, q[t].w[4 * j + i][0], q[t].w[4 * j + i][1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma16816<BF16>(acc[t], lo[2 * i], hi[2 * i], lo[2 * i + 1], hi[2 * i + 1],
                         q[t].w[2 * j + i][0], q[t].w[2 * j + i][1]);
    }
  }
}

// (reference, sum) of a row in log2 units: sum = sum over its tokens of
// 2^(s - reference).  An empty row is (kNoScore, 0); 2^(-inf - kNoScore) is 0.
constexpr float kNoScore = -3.402823466e38f;
__device__ __forceinline__ void stat_join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  l = l * fast_exp2(m - top) + l2 * fast_exp2(m2 - top);
  m = top;
}

// ------------------------------------------------------------------ the kernel
// Grid barrier among the `n` CTAs that have work, by one thread of each.  What a
// CTA wrote before it (and a __syncthreads) is seen after it by the others.
// False: the wait reached its limit.  A count above what a finished call can leave
// is reported, and nobody is kept waiting for it.
__device__ __forceinline__ bool grid_barrier(uint32_t* words, uint32_t n, unsigned* status,
                                             uint64_t limit_ns) {
  __threadfence();
  const uint32_t gen = ld_acquire_b32(words + 1);
  const uint32_t old = atomicAdd(words, 1u);
  if (old > n - 1) {
    atomicOr(status, kStatusWsDirty);
    return true;
  }
  if (old == n - 1) {
    atomicExch(words, 0u);
    __threadfence();
    st_release_gpu_b32(words + 1, gen + 1);
    return true;
  }
  if (ld_acquire_b32(words + 1) != gen) return true;
  const uint64_t t0 = global_ns();
  while (ld_acquire_b32(words + 1) == gen) {
    if (global_ns() - t0 >= limit_ns) {
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

// What a warp keeps of one partition.
template <int NT>
struct Partition {
  float m[NT][2], l[NT][2];   // of the lane's two columns of each tile, over its own tokens

  // The scores of one page: into the workspace and the statistics.  The
  // reference moves only when a score exceeds it by 2^8, so that few pages pay
  // for a rescale; a sum of up to 2^8 a token is as exact as one of 1.
  __device__ __forceinline__ void take(const float (&s)[NT][4], float4* out) {
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      out[t * 32] = make_float4(s[t][0], s[t][1], s[t][2], s[t][3]);
#pragma unroll
      for (int c = 0; c < 2; ++c) grow |= fmaxf(s[t][c], s[t][c + 2]) > m[t][c] + 8.f;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float top = fmaxf(m[t][c], fmaxf(s[t][c], s[t][c + 2]));
          l[t][c] *= fast_exp2(m[t][c] - top);
          m[t][c] = top;
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        l[t][c] += fast_exp2(s[t][c] - m[t][c]) + fast_exp2(s[t][c + 2] - m[t][c]);
  }
};

// The scores of pages [x, end) of the line, by one warp.
template <int D, int KV, int NT, typename LogitsAt>
__device__ __forceinline__ void score_pages(const WeightsArgs& a, const Work& ws, const int* cum,
                                            int64_t x, int64_t end, int w, int lane, int rows,
                                            const LogitsAt& logits_at) {
  constexpr int R = 8 * NT;
  while (x < end) {
    const Place at = find(cum, a.B, a.Hkv, x);
    const int L = __ldg(a.context_lens + at.b);
    const int n = static_cast<int>(min(static_cast<int64_t>(at.pages - at.page), end - x));
    const int32_t* table = a.block_tables + static_cast<int64_t>(at.b) * a.mbs + at.page;
    // block ids, 32 pages at a time, one a lane; -1 outside the pool
    auto ids_from = [&](int i) {
      int id = i + lane < n ? __ldg(table + i + lane) : -1;
      if (i + lane < n && (id < 0 || id >= a.num_blocks)) {
        atomicOr(a.status, kStatusBadBlock);
        id = -1;
      }
      return id;
    };
    int ids = ids_from(0);
    auto id_of = [&](int i) { return __shfl_sync(0xffffffffu, ids, i & 31); };
    Page<D, KV> buf[2];
    int id0 = id_of(0), id1 = -1;
    buf[0].load(a, max(id0, 0), at.h, lane);
    Query<D, KV> q[NT];
    float f[NT][2];   // score -> log2 units, for the lane's columns
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + (lane >> 2);
      const int i = r / a.group, g = r - i * a.group;
      const uint16_t* row = static_cast<const uint16_t*>(a.q) +
          ((static_cast<int64_t>(at.b) * a.q_tokens + a.q_first + i) * a.Hq +
           at.h * a.group + g) * D;
      const float back = q[t].load(row, r < rows, lane) * a.scale_log2;
      f[t][0] = __shfl_sync(0xffffffffu, back, (lane & 3) * 8);
      f[t][1] = __shfl_sync(0xffffffffu, back, (lane & 3) * 8 + 4);
    }
    // tokens from here on are not attended by some row; padding rows (q = 0)
    // are left out by the finish launch
    const int all_see = L - a.q_tokens + a.q_first + 1;
    Partition<NT> part;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) part.m[t][c] = kNoScore, part.l[t][c] = 0.f;
    auto step = [&](const Page<D, KV>& k, int id, int i) {
      float s[NT][4];
      page_scores<D, KV, NT>(s, k, q);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[t][j] *= Kind<KV>::kE4m3 ? f[t][j & 1] * k.scale : f[t][j & 1];
      const int first = (at.page + i) * 16;
      if (first + 16 > all_see || id < 0) {
        const int tok = first + (lane >> 2);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int col = 8 * t + 2 * (lane & 3) + (j & 1);
            if (id < 0 || tok + (j & 2 ? 8 : 0) >= all_see + col / a.group) s[t][j] = -INFINITY;
          }
      }
      part.take(s, logits_at(x + i));
    };
    for (int i = 0; i < n; i += 2) {
      if (i + 1 < n) {
        id1 = id_of(i + 1);
        buf[1].load(a, max(id1, 0), at.h, lane);
      }
      step(buf[0], id0, i);
      if (i + 1 >= n) break;
      if (i + 2 < n) {
        if (((i + 2) & 31) == 0) ids = ids_from(i + 2);
        id0 = id_of(i + 2);
        buf[0].load(a, max(id0, 0), at.h, lane);
      }
      step(buf[1], id1, i + 1);
    }
    // the partition's statistics: over the 8 lanes that hold the same columns
    const int64_t index = static_cast<int64_t>(at.b) * a.Hkv + at.h + w;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          stat_join(part.m[t][c], part.l[t][c], __shfl_xor_sync(0xffffffffu, part.m[t][c], o),
                    __shfl_xor_sync(0xffffffffu, part.l[t][c], o));
      if (lane < 4)
        *reinterpret_cast<float4*>(ws.stats + index * R + 8 * t + 2 * lane) =
            make_float4(part.m[t][0], part.l[t][0], part.m[t][1], part.l[t][1]);
    }
    x += n;
  }
}

// Joins the partitions [0, n) of a unit at st (R rows each): by one warp, lane
// i taking row i % R of every 32 / R-th partition.
template <int R>
__device__ __forceinline__ float2 join_by_warp(const float2* st, int n, int lane) {
  float m = kNoScore, l = 0.f;
  for (int i = lane; i < n * R; i += 32) {
    const float2 v = __ldcg(st + i);
    stat_join(m, l, v.x, v.y);
  }
#pragma unroll
  for (int o = R; o < 32; o <<= 1)
    stat_join(m, l, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
  return make_float2(m, l);   // of row lane % R
}

// A unit of more partitions than this is joined by a whole CTA, once for its
// warps: at most two such units (its first and its last) reach into a CTA's pages.
constexpr int kWarpJoin = 16;

template <int D, int KV, int NT>
__global__ void __launch_bounds__(Shape<NT>::kWarps * 32, Shape<NT>::kCtas)
weights_kernel(const __grid_constant__ WeightsArgs a, Work ws) {
  using S = Shape<NT>;
  constexpr int R = 8 * NT;
  constexpr int kThreads = S::kWarps * 32;
  extern __shared__ float4 kept_logits[];
  __shared__ int cum[kPrefix];
  __shared__ int warp_sums[S::kWarps];
  __shared__ float2 joined[2][R];
  __shared__ float2 scratch[kThreads];
  __shared__ bool passed;
  const int tid = threadIdx.x, lane = tid & 31;
  const int w_first = blockIdx.x * S::kWarps, w = w_first + (tid >> 5);
  prefix_pages<S::kWarps>(a, cum, warp_sums);
  const Line line = make_line(a, cum, static_cast<int>(gridDim.x) * S::kWarps);
  if (w_first >= line.workers) return;   // the whole CTA
  const int rows = a.n_q * a.group;
  const int64_t start = part_start(line, min(w, line.workers));
  const int64_t end = part_start(line, min(w + 1, line.workers));
  // the logits of page x: of the warp's first kKept in shared memory
  float4* kept = kept_logits + (tid >> 5) * (S::kKept * S::kPage) + lane;
  auto logits_at = [&](int64_t x) {
    return x - start < S::kKept ? kept + (x - start) * S::kPage : ws.logits + x * S::kPage + lane;
  };
  score_pages<D, KV, NT>(a, ws, cum, start, end, w, lane, rows, logits_at);

  // ---- all statistics are written
  __syncthreads();
  const uint32_t ctas = static_cast<uint32_t>((line.workers + S::kWarps - 1) / S::kWarps);
  if (ctas > 1) {
    if (tid == 0) passed = grid_barrier(ws.barrier, ctas, a.status, a.wait_limit_ns);
    __syncthreads();
    if (!passed) return;
  }
  // units of many partitions are joined by the whole CTA
  int long_unit[2] = {-1, -1};
  {
    const int w_last = min(w_first + S::kWarps, line.workers);
    const int64_t ends[2] = {part_start(line, w_first), part_start(line, w_last) - 1};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const Place at = find(cum, a.B, a.Hkv, ends[e]);
      const int unit = at.b * a.Hkv + at.h;
      if (e == 1 && unit == long_unit[0]) break;
      const int w0 = part_of(line, at.unit_start);
      const int n = part_of(line, at.unit_start + at.pages - 1) - w0 + 1;
      if (n <= kWarpJoin) continue;
      long_unit[e] = unit;
      const float2* st = ws.stats + (static_cast<int64_t>(unit) + w0) * R;
      float m = kNoScore, l = 0.f;
      for (int i = tid; i < n * R; i += kThreads) {
        const float2 v = __ldcg(st + i);
        stat_join(m, l, v.x, v.y);
      }
      scratch[tid] = make_float2(m, l);
      __syncthreads();
      if (tid < R) {
        for (int i = tid + R; i < kThreads; i += R) stat_join(m, l, scratch[i].x, scratch[i].y);
        joined[e][tid] = make_float2(m, l);
      }
      __syncthreads();
    }
  }
  int64_t x = end;
  while (x > start) {   // from the end: the logits written last are the likeliest in L2
    const Place at = find(cum, a.B, a.Hkv, x - 1);
    const int L = __ldg(a.context_lens + at.b);
    const int n = static_cast<int>(min(static_cast<int64_t>(at.page) + 1, x - start));
    const int unit = at.b * a.Hkv + at.h;
    float2 st;
    if (unit == long_unit[0]) {
      st = joined[0][lane % R];
    } else if (unit == long_unit[1]) {
      st = joined[1][lane % R];
    } else {
      const int w0 = part_of(line, at.unit_start);
      st = join_by_warp<R>(ws.stats + (static_cast<int64_t>(unit) + w0) * R,
                           part_of(line, at.unit_start + at.pages - 1) - w0 + 1, lane);
    }
    // an empty row's and a padding row's tokens get 0
    const float inv = lane % R < rows && (st.y > 0.f || st.y != st.y) ? 1.f / st.y : 0.f;
    float top[NT][2], f[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * t + 2 * (lane & 3) + c;
        top[t][c] = __shfl_sync(0xffffffffu, st.x, r);
        f[t][c] = __shfl_sync(0xffffffffu, inv, r);
      }
    float* weights = a.weights + static_cast<int64_t>(unit) * a.stride;
    // a few pages at a time: their old weights and logits are asked for together
    constexpr int kGroup = NT == 4 ? 2 : 4;
    for (int i = 0; i < n; i += kGroup) {
      float4 s[kGroup][NT];
      float old[kGroup];
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        old[j] = 0.f;
        if (i + j >= n) continue;
        const int tok = (at.page - i - j) * 16 + (lane >> 2) + (lane & 1) * 8;
        if ((lane & 2) == 0 && a.decay != 0.f && tok < L - a.fresh) old[j] = weights[tok];
        const float4* in = logits_at(x - 1 - i - j);
#pragma unroll
        for (int t = 0; t < NT; ++t) s[j][t] = in[t * 32];
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        if (i + j >= n) break;
        const int tok = (at.page - i - j) * 16 + (lane >> 2) + (lane & 1) * 8;
        float lo = 0.f, hi = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          lo += fast_exp2(s[j][t].x - top[t][0]) * f[t][0] + fast_exp2(s[j][t].y - top[t][1]) * f[t][1];
          hi += fast_exp2(s[j][t].z - top[t][0]) * f[t][0] + fast_exp2(s[j][t].w - top[t][1]) * f[t][1];
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          lo += __shfl_xor_sync(0xffffffffu, lo, o);
          hi += __shfl_xor_sync(0xffffffffu, hi, o);
        }
        if ((lane & 2) == 0 && tok < L) weights[tok] = a.decay * old[j] + (lane & 1 ? hi : lo);
      }
    }
    x -= n;
  }
}

int tiles_of(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

// CTAs of a launch of `warps` warps each, `ctas` of them an SM; fewer when there
// cannot be as many pages as warps.
int weights_grid(const WeightsArgs& a, int warps, int ctas) {
  const int64_t pages = static_cast<int64_t>(a.B) * a.Hkv *
                        ((static_cast<int64_t>(a.max_context_len) + 15) / 16);
  const int64_t want = (pages + warps - 1) / warps;
  const int most = ctas * device_sm_count();
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

template <int D, int KV, int NT>
cudaError_t launch_tiles(const WeightsArgs& a, const Work& ws, cudaStream_t s) {
  using S = Shape<NT>;
  auto* kernel = weights_kernel<D, KV, NT>;
  {
    // more than 48 KB of shared memory has to be asked for, once per device
    static std::mutex mu;
    static bool raised[kMaxDevices] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!raised[dev]) {
      if (cudaError_t e = cudaFuncSetAttribute(
              kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem))
        return e;
      raised[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(weights_grid(a, S::kWarps, S::kCtas));
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeCooperative;   // the CTAs wait for one another
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, ws);
}

template <int D, int KV>
cudaError_t launch_pass(const WeightsArgs& a, int nt, const Work& ws, cudaStream_t s) {
  return nt == 1 ? launch_tiles<D, KV, 1>(a, ws, s) : nt == 2 ? launch_tiles<D, KV, 2>(a, ws, s)
                                                              : launch_tiles<D, KV, 4>(a, ws, s);
}

}  // namespace

size_t weights_workspace_bytes(int B, int Hkv, int max_context_len, int rows) {
  const size_t nt = tiles_of(rows);
  if (B > kWeightsMaxBatch) B = kWeightsMaxBatch;
  const size_t units = static_cast<size_t>(B) * Hkv;
  const size_t pages = units * ((static_cast<size_t>(max_context_len) + 15) / 16);
  const size_t parts = units + static_cast<size_t>(2 * device_sm_count()) * kMaxWarps;
  return kBarrierBytes + align256(pages * nt * 32 * sizeof(float4)) +
         align256(parts * nt * 8 * sizeof(float2));
}

cudaError_t launch_weights(const WeightsArgs& a0, bool fp8, bool bf16, cudaStream_t s) {
  const int per_pass = a0.q_tokens * a0.group <= kWeightsMaxRows ? a0.q_tokens
                                                                 : kWeightsMaxRows / a0.group;
  for (int b0 = 0; b0 < a0.B; b0 += kWeightsMaxBatch) {
    WeightsArgs a = a0;
    a.B = a0.B - b0 < kWeightsMaxBatch ? a0.B - b0 : kWeightsMaxBatch;
    a.weights = a0.weights + static_cast<int64_t>(b0) * a.Hkv * a.stride;
    a.q = static_cast<const uint16_t*>(a0.q) + static_cast<int64_t>(b0) * a.q_tokens * a.Hq * a.D;
    a.block_tables = a0.block_tables + static_cast<int64_t>(b0) * a.mbs;
    a.context_lens = a0.context_lens + b0;
    for (int t0 = 0; t0 < a.q_tokens; t0 += per_pass) {
      a.q_first = t0;
      a.n_q = a.q_tokens - t0 < per_pass ? a.q_tokens - t0 : per_pass;
      if (t0 > 0) {   // later passes add to what the first has left
        a.decay = 1.f;
        a.fresh = 0;
      }
      const int nt = tiles_of(a.n_q * a.group);
      const size_t pages = static_cast<size_t>(a.B) * a.Hkv * ((static_cast<size_t>(a.max_context_len) + 15) / 16);
      Work ws;
      uint8_t* base = static_cast<uint8_t*>(a.workspace);
      ws.barrier = reinterpret_cast<uint32_t*>(base);
      base += kBarrierBytes;
      ws.logits = reinterpret_cast<float4*>(base);
      ws.stats = reinterpret_cast<float2*>(base + align256(pages * nt * 32 * sizeof(float4)));
      const int kv = (fp8 ? 2 : 0) + (bf16 ? 1 : 0);
      cudaError_t e;
      if (a.D == 128)
        e = kv == 0 ? launch_pass<128, 0>(a, nt, ws, s) : kv == 1 ? launch_pass<128, 1>(a, nt, ws, s)
          : kv == 2 ? launch_pass<128, 2>(a, nt, ws, s) : launch_pass<128, 3>(a, nt, ws, s);
      else
        e = kv == 0 ? launch_pass<64, 0>(a, nt, ws, s) : kv == 1 ? launch_pass<64, 1>(a, nt, ws, s)
          : kv == 2 ? launch_pass<64, 2>(a, nt, ws, s) : launch_pass<64, 3>(a, nt, ws, s);
      if (e) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace pa
