// weights.cu -- the attention weight each cached token receives.
//
//   W[b][h][t] = old(t) + sum_r softmax_t(scale q_r . K_t)
// over the query rows r of (sequence b, kv head h): n_q tokens times the query
// group.  The weight of a token needs the softmax statistics of the whole
// context, so there are two launches:
//   score:  every page's logits by mma.sync (a page's 16 tokens are the 16 rows
//           of the MMA's A, the query rows its 8 columns), written to the
//           workspace, and per partition and row the running (max, sum);
//   finish: per row the statistics of the whole context, joined from those of
//           its partitions, then each token's weights summed over the rows.
// K is read once: 2 D bytes a token and kv head (D for E4M3) are the floor; the
// logits (4 bytes a query row and token, written and read) stay in L2 when they
// fit there.
//
// Work split: the pages of all (sequence, kv head) units form one line, divided
// evenly among the warps of both launches.  A warp's part of a unit is a
// partition.  Units and warps both grow along the line, so unit + warp numbers
// every partition uniquely, and a unit's partitions are consecutive.
//
// K goes from global memory straight into the MMA's registers.  A dot product
// does not care in which order the dimensions are summed, so lane (r, c) of a
// quad takes the 16-byte chunks c, c + 4, ... of rows r and r + 8, and q's
// fragments are loaded with the same permutation.
#include <climits>

#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPrefix = kWeightsMaxBatch + 1;

// ------------------------------------------------------------ the line of pages
struct Line {
  int64_t n;        // pages of all units
  int workers;      // warps that have pages: each has at least one
};
__device__ __forceinline__ Line make_line(const WeightsArgs& a, const int* cum) {
  const int64_t n = static_cast<int64_t>(cum[a.B]) * a.Hkv;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
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
__device__ __forceinline__ void prefix_pages(const WeightsArgs& a, int* cum, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int base = 0; base < a.B; base += kThreads) {
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
    for (int w = 0; w < kWarps; ++w) {
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
struct Work {
  float4* logits;
  float2* stats;
};
__device__ __host__ __forceinline__ size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// ----------------------------------------------------------------- K fragments
// KV: 0 fp16, 1 bf16, 2 E4M3 with fp16 q, 3 E4M3 with bf16 q
template <int KV>
struct Kind {
  static constexpr bool kE4m3 = KV >= 2;
  static constexpr bool kBf16 = KV == 1 || KV == 3;
};

// Two E4M3 codes as two values of the activations' type; exact.
template <bool BF16>
__device__ __forceinline__ uint32_t codes2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  if constexpr (BF16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack2<true>(f.x, f.y);
  } else {
    return h;
  }
}

// The lane's part of one page: NLD 16-byte chunks of row r, then of row r + 8.
template <int D, int KV>
struct Page {
  static constexpr int NLD = D / (Kind<KV>::kE4m3 ? 64 : 32);
  uint4 lo[NLD], hi[NLD];
  __device__ __forceinline__ void load(const void* page, int lane) {
    constexpr int row_chunks = NLD * 4;
    const uint4* p = static_cast<const uint4*>(page) + (lane >> 2) * row_chunks + (lane & 3);
#pragma unroll
    for (int j = 0; j < NLD; ++j) {
      lo[j] = __ldcs(p + 4 * j);
      hi[j] = __ldcs(p + 8 * row_chunks + 4 * j);
    }
  }
};

// The lane's part of 8 query rows: the elements its K chunks hold, of row lane / 4.
template <int D, int KV>
struct Query {
  uint32_t w[D / 16][2];   // b0, b1 of each of the D / 16 MMA steps
  __device__ __forceinline__ void load(const uint16_t* row, bool live, int lane) {
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
        const uint32_t a0 = codes2<BF16>(lo[i] & 0xffffu), a2 = codes2<BF16>(lo[i] >> 16);
        const uint32_t a1 = codes2<BF16>(hi[i] & 0xffffu), a3 = codes2<BF16>(hi[i] >> 16);
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

// Running (max, sum) of a row in log2 units; an empty row is (-inf, 0).
__device__ __forceinline__ void stat_join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  const float base = top == -INFINITY ? 0.f : top;
  l = l * fast_exp2(m - base) + l2 * fast_exp2(m2 - base);
  m = top;
}

// ------------------------------------------------------------------- launch 1
template <int D, int KV, int NT>
__global__ void __launch_bounds__(kThreads, NT == 4 ? 1 : 2)
weights_score_kernel(const __grid_constant__ WeightsArgs a, Work ws) {
  __shared__ int cum[kPrefix];
  __shared__ int warp_sums[kWarps];
  constexpr int R = 8 * NT;
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  prefix_pages(a, cum, warp_sums);
  const Line line = make_line(a, cum);
  if (w >= line.workers) return;
  int64_t x = part_start(line, w);
  const int64_t end = part_start(line, w + 1);
  const int rows = a.n_q * a.group;
  const int64_t page_bytes = 16 * D * (Kind<KV>::kE4m3 ? 1 : 2);
  while (x < end) {
    const Place at = find(cum, a.B, a.Hkv, x);
    const int L = __ldg(a.context_lens + at.b);
    const int stop = static_cast<int>(min(static_cast<int64_t>(at.pages), at.page + (end - x)));
    // q, and for the lane's two columns of each tile the first position not attended
    Query<D, KV> q[NT];
    int bound[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + (lane >> 2);
      const int i = r / a.group, g = r - i * a.group;
      const uint16_t* row = static_cast<const uint16_t*>(a.q) +
          ((static_cast<int64_t>(at.b) * a.q_tokens + a.q_first + i) * a.Hq +
           at.h * a.group + g) * D;
      q[t].load(row, r < rows, lane);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * t + 2 * (lane & 3) + c;
        bound[t][c] = col < rows ? L - a.q_tokens + a.q_first + col / a.group + 1 : 0;
      }
    }
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) m[t][c] = -INFINITY, l[t][c] = 0.f;
    const int32_t* table = a.block_tables + static_cast<int64_t>(at.b) * a.mbs;
    float4* out = ws.logits + (at.unit_start * NT) * 32 + lane;
    for (int page = at.page; page < stop; ++page) {
      const int id = __ldg(table + page);
      const bool good = id >= 0 && id < a.num_blocks;
      if (!good && lane == 0) atomicOr(a.status, kStatusBadBlock);
      const int64_t tile = static_cast<int64_t>(good ? id : 0) * a.Hkv + at.h;
      Page<D, KV> k;
      k.load(static_cast<const uint8_t*>(a.k_cache) + tile * page_bytes, lane);
      float f = a.scale_log2;
      if constexpr (Kind<KV>::kE4m3) f *= __ldg(a.k_scale + tile);
      float s[NT][4];
      page_scores<D, KV, NT>(s, k, q);
      const int tok = page * 16 + (lane >> 2);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool seen = good && tok + (i & 2 ? 8 : 0) < bound[t][i & 1];
          s[t][i] = seen ? s[t][i] * f : -INFINITY;
        }
        out[(static_cast<int64_t>(page) * NT + t) * 32] =
            make_float4(s[t][0], s[t][1], s[t][2], s[t][3]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float top = fmaxf(m[t][c], fmaxf(s[t][c], s[t][c + 2]));
          const float base = top == -INFINITY ? 0.f : top;
          l[t][c] = l[t][c] * fast_exp2(m[t][c] - base) + fast_exp2(s[t][c] - base) +
                    fast_exp2(s[t][c + 2] - base);
          m[t][c] = top;
        }
      }
    }
    // the partition's statistics: over the 8 lanes that hold the same columns
    const int64_t part = static_cast<int64_t>(at.b) * a.Hkv + at.h + w;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          stat_join(m[t][c], l[t][c], __shfl_xor_sync(0xffffffffu, m[t][c], o),
                    __shfl_xor_sync(0xffffffffu, l[t][c], o));
      if (lane < 4) {
        float2* st = ws.stats + part * R + 8 * t + 2 * lane;
        st[0] = make_float2(m[t][0], l[t][0]);
        st[1] = make_float2(m[t][1], l[t][1]);
      }
    }
    x += stop - at.page;
  }
}

// ------------------------------------------------------------------- launch 2
template <int NT>
__global__ void __launch_bounds__(kThreads, 2)
weights_finish_kernel(const __grid_constant__ WeightsArgs a, Work ws) {
  __shared__ int cum[kPrefix];
  __shared__ int warp_sums[kWarps];
  constexpr int R = 8 * NT;
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * kWarps + (threadIdx.x >> 5);
  prefix_pages(a, cum, warp_sums);
  const Line line = make_line(a, cum);
  if (w >= line.workers) return;
  int64_t x = part_start(line, w);
  const int64_t end = part_start(line, w + 1);
  while (x < end) {
    const Place at = find(cum, a.B, a.Hkv, x);
    const int L = __ldg(a.context_lens + at.b);
    const int stop = static_cast<int>(min(static_cast<int64_t>(at.pages), at.page + (end - x)));
    const int64_t unit = static_cast<int64_t>(at.b) * a.Hkv + at.h;
    // the unit's statistics: lane holds row lane % R of every 32 / R-th partition
    const int w0 = part_of(line, at.unit_start), w1 = part_of(line, at.unit_start + at.pages - 1);
    const float2* st = ws.stats + (unit + w0) * R;
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < (w1 - w0 + 1) * R; i += 32) {
      const float2 v = st[i];
      stat_join(m, l, v.x, v.y);
    }
#pragma unroll
    for (int o = R; o < 32; o <<= 1)
      stat_join(m, l, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, l, o));
    // an empty row gives every token 0: its logits are -inf
    const float base = m == -INFINITY ? 0.f : m;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    float top[NT][2], f[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * t + 2 * (lane & 3) + c;
        top[t][c] = __shfl_sync(0xffffffffu, base, r);
        f[t][c] = __shfl_sync(0xffffffffu, inv, r);
      }
    float* weights = a.weights + unit * a.stride;
    const float4* in = ws.logits + (at.unit_start * NT) * 32 + lane;
    for (int page = at.page; page < stop; ++page) {
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float4 s = in[(static_cast<int64_t>(page) * NT + t) * 32];
        lo += fast_exp2(s.x - top[t][0]) * f[t][0] + fast_exp2(s.y - top[t][1]) * f[t][1];
        hi += fast_exp2(s.z - top[t][0]) * f[t][0] + fast_exp2(s.w - top[t][1]) * f[t][1];
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
        hi += __shfl_xor_sync(0xffffffffu, hi, o);
      }
      const int tok = page * 16 + (lane >> 2) + (lane & 1) * 8;
      if ((lane & 2) == 0 && tok < L) {
        const float old = a.decay != 0.f && tok < L - a.fresh ? a.decay * weights[tok] : 0.f;
        weights[tok] = old + (lane & 1 ? hi : lo);
      }
    }
    x += stop - at.page;
  }
}

int tiles_of(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

template <int D, int KV>
cudaError_t launch_pass(const WeightsArgs& a, int nt, int grid, const Work& ws, cudaStream_t s) {
  if (nt == 1) {
    weights_score_kernel<D, KV, 1><<<grid, kThreads, 0, s>>>(a, ws);
    weights_finish_kernel<1><<<grid, kThreads, 0, s>>>(a, ws);
  } else if (nt == 2) {
    weights_score_kernel<D, KV, 2><<<grid, kThreads, 0, s>>>(a, ws);
    weights_finish_kernel<2><<<grid, kThreads, 0, s>>>(a, ws);
  } else {
    weights_score_kernel<D, KV, 4><<<grid, kThreads, 0, s>>>(a, ws);
    weights_finish_kernel<4><<<grid, kThreads, 0, s>>>(a, ws);
  }
  return cudaGetLastError();
}

// CTAs of a launch: two a SM, fewer when there are fewer pages than warps.
int weights_grid(int B, int Hkv, int max_context_len) {
  const int64_t pages = static_cast<int64_t>(B) * Hkv * ((static_cast<int64_t>(max_context_len) + 15) / 16);
  const int64_t want = (pages + kWarps - 1) / kWarps;
  const int most = 2 * device_sm_count();
  return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

}  // namespace

size_t weights_workspace_bytes(int B, int Hkv, int max_context_len, int rows) {
  const size_t nt = tiles_of(rows);
  if (B > kWeightsMaxBatch) B = kWeightsMaxBatch;
  const size_t units = static_cast<size_t>(B) * Hkv;
  const size_t pages = units * ((static_cast<size_t>(max_context_len) + 15) / 16);
  const size_t parts = units + static_cast<size_t>(weights_grid(B, Hkv, max_context_len)) * kWarps;
  return align256(pages * nt * 32 * sizeof(float4)) + align256(parts * nt * 8 * sizeof(float2));
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
      const int grid = weights_grid(a.B, a.Hkv, a.max_context_len);
      const size_t pages = static_cast<size_t>(a.B) * a.Hkv * ((static_cast<size_t>(a.max_context_len) + 15) / 16);
      Work ws;
      ws.logits = static_cast<float4*>(a.workspace);
      ws.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(a.workspace) +
                                           align256(pages * nt * 32 * sizeof(float4)));
      const int kv = (fp8 ? 2 : 0) + (bf16 ? 1 : 0);
      cudaError_t e;
      if (a.D == 128)
        e = kv == 0 ? launch_pass<128, 0>(a, nt, grid, ws, s) : kv == 1 ? launch_pass<128, 1>(a, nt, grid, ws, s)
          : kv == 2 ? launch_pass<128, 2>(a, nt, grid, ws, s) : launch_pass<128, 3>(a, nt, grid, ws, s);
      else
        e = kv == 0 ? launch_pass<64, 0>(a, nt, grid, ws, s) : kv == 1 ? launch_pass<64, 1>(a, nt, grid, ws, s)
          : kv == 2 ? launch_pass<64, 2>(a, nt, grid, ws, s) : launch_pass<64, 3>(a, nt, grid, ws, s);
      if (e) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace pa
