// weights.cu -- the attention weight each cached token receives.
//
//   W[b][h][t] = old(t) + sum_r softmax_t(scale q_r . K_t)
// over the query rows r of (sequence b, kv head h): n_q tokens times the query
// group.  The weight of a token needs the softmax statistics of the whole
// context, so one launch works in two phases:
//   score:  every page's logits by mma.sync (a page's 16 tokens are the 16 rows
//           of the MMA's A, the query rows its 8 columns) and, per partition and
//           row, the running (reference, sum);
//   finish: per row the statistics of the whole context, joined from those of
//           its partitions, then each token's weights summed over the rows.
// Short contexts take a cluster of CTAs for each unit (sequence, kv head), which joins
// its statistics through distributed shared memory.  Long ones take a cooperative
// launch over all units' pages, whose warps wait between the phases for the warps
// that share their first and their last unit, so that slow SMs do not hold up others.
// K is read once: 2 D bytes a token and kv head (D for E4M3) are the floor.  A
// warp keeps the logits of its first pages in shared memory and those behind
// them in the workspace, where they mostly stay in L2; the old weights come into
// shared memory while K is read.
//
// Work split of the cooperative launch: the pages of all units form one line, divided
// evenly among the warps.  A warp's part of a unit is a partition.  Units and
// warps both grow along the line, so unit + warp numbers every partition
// uniquely, and a unit's partitions are consecutive.
//
// Measured on a GB300 (28 q and 4 kv heads of 128): 54 to 59 us for 128 fp16 sequences,
// median 1024 tokens (212 MB, 53 to 58 % of the measured copy bandwidth), of which the first
// phase, at 5.8 TB/s, takes 37, the wait for the slowest neighbours and the joining 3,
// the second phase 5 and the launch the rest; 34 us for 100 sequences of up to 2048
// tokens by clusters; 71 to 73 us for two 115k-token E4M3 contexts with 28 rows (122 MB):
// 42 to score, bound by each warp's own chain (2500 cycles a page, the tensor pipe busy
// for 260 of them, three warps a scheduler), 12 of it for the logits, which are as large
// as K; 5 to wait and join; 15 for the second phase.  What was slower in that case:
// three or four pages on their way a warp instead of two 79 and 80 us against 78.7, two
// pages scored at once 85, 14 or 16 warps (with fewer pages kept) 87 and 85 against 81.
// Before q's fragments moved to shared memory (84 us): the logits computed again in the
// second phase 85 to 90 us, K through a ring in shared memory 81 to 90 us (and 87 to 90
// us for the 128 sequences), two fp32 values an instruction 86 us.
//
// K goes from global memory straight into the MMA's registers.  A dot product
// does not care in which order the dimensions are summed, so lane (r, c) of a
// quad takes the 32-byte chunks c, c + 4, ... of rows r and r + 8, and q's
// fragments are loaded with the same permutation.
#include <mutex>

#include "pa_cluster.cuh"
#include "pa_e4m3.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kPrefix = kWeightsMaxBatch + 1;
constexpr int kMaxWarps = 12;
constexpr int kOld = 32;   // pages a warp whose old weights are copied ahead
// Warps of a CTA, CTAs an SM, and what a warp's share of shared memory holds: the
// logits of kKept pages, the old weights of kOld and, at head_dim 128, the query's MMA
// fragments.  Up to 16 query rows keep 16 warps an SM; 32 need the registers of 12.
// The fragments of 8, 16 and 32 rows of 128 take 16, 32 and 64 registers, or shared
// memory that would keep 4 more pages.  Registers against shared memory: 57.6 and 56.8
// us for 7 rows (128 16-bit contexts), 53.6 and 45.9 for 14 and 73.8 and 55.8 for 28
// (24 contexts of up to 8000 tokens), 87.5 and 78.7 for 28 rows over two E4M3 contexts
// of 115k; at head_dim 64 they are half as large, and 32 rows take 47.2 us against 50.6.
template <int D, int NT>
struct Shape {
  static constexpr bool kSharedQ = D == 128;
  static constexpr int kWarps = NT == 4 ? 12 : 8;
  static constexpr int kCtas = NT == 4 ? 1 : 2;
  static constexpr int kKept = (NT == 1 ? 22 : NT == 2 ? 11 : 8) - (kSharedQ ? 4 : 0);
  static constexpr int kPage = NT * 32;        // float4s of a page's logits
  static constexpr int kOldAt = kKept * kPage * 16;      // bytes
  static constexpr int kQueryAt = kOldAt + kOld * 64;
  static constexpr int kWarpBytes = kQueryAt + (kSharedQ ? NT * 8 * D * 2 : 0);
  static constexpr int kSmem = kWarps * kWarpBytes;
};

// ------------------------------------------------------------ the line of pages
struct Line {
  int64_t n;        // pages of all units
  int workers;      // warps that have pages: each has at least one
  bool small;       // (n + 1) * workers fits 32 bits: the short division will do
};
__device__ __forceinline__ Line make_line(const WeightsArgs& a, const int* cum, int warps) {
  const int64_t n = static_cast<int64_t>(cum[a.B]) * a.Hkv;
  const int workers = static_cast<int>(n < warps ? n : warps);
  return Line{n, workers, (n + 1) * workers < (INT64_C(1) << 32)};
}
// The pages worker w takes: [start(w), start(w + 1)).
__device__ __forceinline__ int64_t part_start(const Line& l, int w) {
  if (l.small)
    return static_cast<uint32_t>(l.n) * static_cast<uint32_t>(w) / static_cast<uint32_t>(l.workers);
  return l.n * w / l.workers;
}
// The worker that takes page x of the line.
__device__ __forceinline__ int part_of(const Line& l, int64_t x) {
  if (l.small)
    return static_cast<int>((static_cast<uint32_t>(x + 1) * static_cast<uint32_t>(l.workers) - 1u) /
                            static_cast<uint32_t>(l.n));
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
  // fewer than 2^31 pages a sequence; all its heads' may be more
  p.h = in_seq < (INT64_C(1) << 32)
            ? static_cast<int>(static_cast<uint32_t>(in_seq) / static_cast<uint32_t>(p.pages))
            : static_cast<int>(in_seq / p.pages);
  p.page = static_cast<int>(in_seq - static_cast<int64_t>(p.h) * p.pages);
  p.unit_start = x - p.page;
  return p;
}

// ------------------------------------------------------------------ workspace
// sync[0]: CTAs done, 0 between calls; sync[1]: the number of the last call;
// sync[2 + w]: the call in which warp w has last written its statistics.
// logits: per page of the line and tile of 8 query rows, [token][row] (a token's
// two halves swapped by bit 2 of the token: no bank conflicts in shared memory);
// of 32 rows, most of which go to the workspace, as the MMA's result fragment, one
// float4 a lane.
// statistics: per partition and row (reference, sum), log2 units.
struct Work {
  uint32_t* sync;
  float* logits;
  float2* stats;
};
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// 4-byte asynchronous copy global -> shared.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

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

// 32 bytes of global memory that are read once.
struct Bytes32 {
  uint32_t w[8];
};
__device__ __forceinline__ Bytes32 load32(const void* p, bool aligned) {
  Bytes32 v;
  if (!aligned) {   // a pool that starts at 16 bytes
    const uint4 x = __ldcs(static_cast<const uint4*>(p));
    const uint4 y = __ldcs(static_cast<const uint4*>(p) + 1);
    return Bytes32{{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}};
  }
  asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]),
                 "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
               : "l"(p));
  return v;
}

// The lane's part of one page: 32-byte chunks c, c + 4, ... of row r, then of row
// r + 8, so that the quad of a row reads whole 128-byte lines.
template <int D, int KV>
struct Page {
  static constexpr int kRow = D * (Kind<KV>::kE4m3 ? 1 : 2);   // bytes
  static constexpr int NLD = kRow < 128 ? 1 : kRow / 128;
  Bytes32 lo[NLD], hi[NLD];
  float scale;     // of an E4M3 page
  __device__ __forceinline__ void load(const WeightsArgs& a, int id, int h, int lane) {
    const int64_t tile = static_cast<int64_t>(id) * a.Hkv + h;
    const uint8_t* p = static_cast<const uint8_t*>(a.k_cache) + tile * (16 * kRow) +
                       (lane >> 2) * kRow;
    if constexpr (kRow < 128) {   // 64-byte rows: 16 bytes a lane
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p + (lane & 3) * 16));
      const uint4 y = __ldcs(reinterpret_cast<const uint4*>(p + 8 * kRow + (lane & 3) * 16));
      lo[0] = Bytes32{{x.x, x.y, x.z, x.w, 0, 0, 0, 0}};
      hi[0] = Bytes32{{y.x, y.y, y.z, y.w, 0, 0, 0, 0}};
    } else {
#pragma unroll
      for (int j = 0; j < NLD; ++j) {
        lo[j] = load32(p + ((lane & 3) + 4 * j) * 32, a.wide);
        hi[j] = load32(p + 8 * kRow + ((lane & 3) + 4 * j) * 32, a.wide);
      }
    }
    if constexpr (Kind<KV>::kE4m3) scale = __ldg(a.k_scale + tile);
  }
};

// The lane's part of 8 query rows: the elements its K chunks hold, of row lane / 4.
template <int D, int KV>
struct Query {
  uint32_t w[D / 16][2];   // b0, b1 of each of the D / 16 MMA steps
  __device__ __forceinline__ void load(const uint16_t* row, int lane) {
    // elements of a K chunk: its bytes over an element's
    constexpr int kRow = Page<D, KV>::kRow;
    constexpr int per = (kRow < 128 ? 16 : 32) / (Kind<KV>::kE4m3 ? 1 : 2);
#pragma unroll
    for (int j = 0; j < D / (4 * per); ++j) {
#pragma unroll
      for (int x = 0; x < per / 8; ++x) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + ((lane & 3) + 4 * j) * per + 8 * x));
        const int s = (j * per + 8 * x) / 4;         // two steps per 8 elements
        w[s][0] = v.x;
        w[s][1] = v.y;
        w[s + 1][0] = v.z;
        w[s + 1][1] = v.w;
      }
    }
  }
  // Returns what the scores have to be multiplied by (1 unless q was scaled).
  __device__ __forceinline__ float scale() {
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

// The query rows of a unit as MMA fragments, in registers or in shared memory, where
// the lane's 16 bytes of tile t and steps 2 s and 2 s + 1 stand at (t * D / 32 + s) * 32
// (each lane reads only what it has written).
template <int D, int KV, int NT>
struct Rows {
  static constexpr bool kShared = Shape<D, NT>::kSharedQ;
  Query<D, KV> q[kShared ? 1 : NT];
  uint4* shared;
  __device__ __forceinline__ void put(int t, const Query<D, KV>& x) {
    if constexpr (kShared) {
#pragma unroll
      for (int s = 0; s < D / 32; ++s)
        shared[(t * (D / 32) + s) * 32] =
            make_uint4(x.w[2 * s][0], x.w[2 * s][1], x.w[2 * s + 1][0], x.w[2 * s + 1][1]);
    } else {
      q[t] = x;
    }
  }
};

template <int D, int KV, int NT>
__device__ __forceinline__ void page_scores(float (&acc)[NT][4], const Page<D, KV>& k,
                                            const Rows<D, KV, NT>& rows) {
  constexpr bool BF16 = Kind<KV>::kBf16;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  // a step takes 4 elements a lane: two words of 16-bit values, one of codes
  constexpr int kSteps = (Page<D, KV>::kRow < 128 ? 4 : 8) / (Kind<KV>::kE4m3 ? 1 : 2);   // of a chunk
  auto fragment = [&](int st, uint32_t (&a)[4]) {
    const uint32_t* lo = k.lo[st / kSteps].w;
    const uint32_t* hi = k.hi[st / kSteps].w;
    const int i = st % kSteps;
    if constexpr (Kind<KV>::kE4m3) {
      a[0] = e4m3x2_to_f16x2(lo[i] & 0xffffu), a[2] = e4m3x2_to_f16x2(lo[i] >> 16);
      a[1] = e4m3x2_to_f16x2(hi[i] & 0xffffu), a[3] = e4m3x2_to_f16x2(hi[i] >> 16);
    } else {
      a[0] = lo[2 * i], a[1] = hi[2 * i], a[2] = lo[2 * i + 1], a[3] = hi[2 * i + 1];
    }
  };
  if constexpr (Rows<D, KV, NT>::kShared) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      uint32_t a0[4], a1[4];
      fragment(2 * s, a0);
      fragment(2 * s + 1, a1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 b = rows.shared[(t * (D / 32) + s) * 32];
        mma16816<BF16>(acc[t], a0[0], a0[1], a0[2], a0[3], b.x, b.y);
        mma16816<BF16>(acc[t], a1[0], a1[1], a1[2], a1[3], b.z, b.w);
      }
    }
  } else {
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      uint32_t f[4];
      fragment(st, f);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma16816<BF16>(acc[t], f[0], f[1], f[2], f[3], rows.q[t].w[st][0], rows.q[t].w[st][1]);
    }
  }
}

// Two fp32 values an instruction.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 exp2_2(F2 a) {
  const float2 x = unpack(a);
  return pack(fast_exp2(x.x), fast_exp2(x.y));
}

// (reference, sum) of a row in log2 units: sum = sum over its tokens of
// 2^(s - reference).  An empty row is (kNoScore, 0); 2^(-inf - kNoScore) is 0.
constexpr float kNoScore = -3.402823466e38f;
__device__ __forceinline__ void stat_join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  l = l * fast_exp2(m - top) + l2 * fast_exp2(m2 - top);
  m = top;
}

// What p (in this CTA's shared memory) holds in CTA `rank`'s.
__device__ __forceinline__ float2 ld_cluster2(const float2* p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(in_cluster(p, rank)));
  return v;
}

// ------------------------------------------------------------------ the kernel
// Waits until warps [w0, w0 + n) have written their statistics in call `call`;
// by the threads `first`, first + step, ... of a warp or CTA, each for its share.
// False: the wait reached its limit.
__device__ __forceinline__ bool await_warps(const Work& ws, int w0, int n, uint32_t call, int first,
                                            int step, unsigned* status, uint64_t limit_ns) {
  for (int i = first; i < n; i += step) {
    const uint32_t* flag = ws.sync + 2 + w0 + i;
    if (ld_acquire_b32(flag) == call) continue;
    const uint64_t t0 = global_ns();
    while (ld_acquire_b32(flag) != call) {
      if (global_ns() - t0 >= limit_ns) {
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
  return true;
}

// Where the score of (token of the page, row 2 c of tile t) stands among a page's.
__device__ __forceinline__ int logit_at(int t, int tok, int c) {
  return t * 128 + tok * 8 + (((c >> 1) ^ ((tok >> 2) & 1)) << 2) + (c & 1) * 2;
}

// One warp's pages of one unit: n pages from page at.page on.  Calls take(scores,
// scale of the page, i, skip) for each (i counts from at.page; skip: its block is
// outside the pool).  asked: the block id of page `lane`.
template <int D, int KV, int NT, typename Take>
__device__ __forceinline__ void for_pages(const WeightsArgs& a, const Place& at, int n, int lane,
                                          const Rows<D, KV, NT>& q, int asked, const Take& take) {
  using P = Page<D, KV>;
  // pages in registers, the one at work among them: up to 64 registers
  constexpr int kAhead = P::kRow >= 256 || NT == 4 ? 2 : NT == 1 ? 4 : 3;
  const int32_t* table = a.block_tables + static_cast<int64_t>(at.b) * a.mbs + at.page;
  // block ids, 32 pages at a time, one a lane; -1 outside the pool
  auto ids_from = [&](int j) {
    int id = j == 0 ? asked : j + lane < n ? __ldg(table + j + lane) : -1;
    if (j + lane < n && (id < 0 || id >= a.num_blocks)) {
      atomicOr(a.status, kStatusBadBlock);
      id = -1;
    }
    return id;
  };
  int ids = ids_from(0);
  P buf[kAhead];
  uint32_t bad = 0;   // of the last 32 pages asked for: outside the pool
  auto ask = [&](int j, P& into) {
    if (j < n) {
      if ((j & 31) == 0 && j > 0) ids = ids_from(j);
      const int id = __shfl_sync(0xffffffffu, ids, j & 31);
      bad = id < 0 ? bad | 1u << (j & 31) : bad & ~(1u << (j & 31));
      into.load(a, max(id, 0), at.h, lane);
    }
  };
  auto step = [&](const P& k, int j) {
    float s[NT][4];
    page_scores<D, KV, NT>(s, k, q);
    take(s, Kind<KV>::kE4m3 ? k.scale : 1.f, j, (bad >> (j & 31) & 1) != 0);
  };
#pragma unroll
  for (int j = 0; j < kAhead - 1; ++j) ask(j, buf[j]);
  for (int i = 0; i < n; i += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i + j >= n) break;
      ask(i + j + kAhead - 1, buf[(j + kAhead - 1) % kAhead]);
      step(buf[j], i + j);
    }
  }
}

// The query rows of a unit and what turns their scores into log2 units, for the
// lane's two columns of each tile.  Columns behind the rows hold the last row again:
// they get weight 0 in the second phase, and a score of theirs is infinite or not a
// number (which no weight makes 0) only where a row's own is.
template <int D, int KV, int NT>
__device__ __forceinline__ void load_rows(const WeightsArgs& a, const Place& at, int rows, int lane,
                                          Rows<D, KV, NT>& to, float (&f)[NT][2]) {
  Query<D, KV> q[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = min(8 * t + (lane >> 2), rows - 1);
    const int i = r / a.group, g = r - i * a.group;
    const uint16_t* row = static_cast<const uint16_t*>(a.q) +
        ((static_cast<int64_t>(at.b) * a.q_tokens + a.q_first + i) * a.Hq +
         at.h * a.group + g) * D;
    q[t].load(row, lane);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float back = q[t].scale() * a.scale_log2;
    to.put(t, q[t]);
    f[t][0] = __shfl_sync(0xffffffffu, back, (lane & 3) * 8);
    f[t][1] = __shfl_sync(0xffffffffu, back, (lane & 3) * 8 + 4);
  }
}

// Scores of tokens that a row does not attend become -inf: those from all_see +
// (its query's number) on, and all of a skipped page.
template <int NT>
__device__ __forceinline__ void mask(float (&s)[NT][4], int first, int all_see, bool skip, int group,
                                     int n_q, int lane) {
  if (first + 16 <= all_see && !skip) return;
  const int tok = first + (lane >> 2);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = 8 * t + 2 * (lane & 3) + (j & 1);
      if (skip || tok + (j & 2 ? 8 : 0) >= all_see + min(col / group, n_q - 1)) s[t][j] = -INFINITY;
    }
}

// The logits of one warp's pages of one unit, n from page at.page on (the first of
// them page x of the line, of which the warp's own begin at `start`), and their
// statistics: R pairs at `stats`.
template <int D, int KV, int NT, typename LogitsAt>
__device__ __forceinline__ void score_segment(const WeightsArgs& a, const Place& at, int L, int n,
                                              int64_t x, int64_t start, int lane, int rows,
                                              uint8_t* mine, float2* stats,
                                              const LogitsAt& logits_at) {
  float* old_weights = reinterpret_cast<float*>(mine + Shape<D, NT>::kOldAt);
  Rows<D, KV, NT> q;
  q.shared = reinterpret_cast<uint4*>(mine + Shape<D, NT>::kQueryAt) + lane;
  float f[NT][2];
  // the first block ids are on their way while the rows are loaded (0.3 to 1.6 us)
  const int asked = lane < n ? __ldg(a.block_tables + static_cast<int64_t>(at.b) * a.mbs + at.page + lane) : -1;
  load_rows<D, KV, NT>(a, at, rows, lane, q, f);
  const int all_see = L - a.q_tokens + a.q_first + 1;
  const float* weights = a.weights + (static_cast<int64_t>(at.b) * a.Hkv + at.h) * a.stride;
  const int old_end = a.decay != 0.f ? L - a.fresh : 0;   // tokens with an old weight
  // the reference and the sum of the lane's columns over its own tokens
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) m[t][c] = kNoScore, l[t][c] = 0.f;
  auto take = [&](float (&s)[NT][4], float page_scale, int i, bool skip) {
    const int first = (at.page + i) * 16;
    if (x - start + i < kOld && lane < 16 && first + lane < old_end)
      cp_async4(smem_u32(old_weights + (x - start + i) * 16 + lane), weights + first + lane);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[t][j] *= Kind<KV>::kE4m3 ? f[t][j & 1] * page_scale : f[t][j & 1];
    mask<NT>(s, first, all_see, skip, a.group, a.n_q, lane);
    float* out = logits_at(x + i);
    // The reference moves only when a score exceeds it by 2^8, so that few pages
    // pay for a rescale; a sum of up to 2^8 a token is as exact as one of 1.
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (NT == 4) {
        *reinterpret_cast<float4*>(out + (t * 32 + lane) * 4) =
            make_float4(s[t][0], s[t][1], s[t][2], s[t][3]);
      } else {
        *reinterpret_cast<float2*>(out + logit_at(t, lane >> 2, lane & 3)) =
            make_float2(s[t][0], s[t][1]);
        *reinterpret_cast<float2*>(out + logit_at(t, (lane >> 2) + 8, lane & 3)) =
            make_float2(s[t][2], s[t][3]);
      }
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
  };
  for_pages<D, KV, NT>(a, at, n, lane, q, asked, take);
  // the partition's statistics: over the 8 lanes that hold the same columns
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        stat_join(m[t][c], l[t][c], __shfl_xor_sync(0xffffffffu, m[t][c], o),
                  __shfl_xor_sync(0xffffffffu, l[t][c], o));
    if (lane < 4)
      *reinterpret_cast<float4*>(stats + 8 * t + 2 * lane) =
          make_float4(m[t][0], l[t][0], m[t][1], l[t][1]);
  }
}

// One warp's pages [start, end) of the line.
template <int D, int KV, int NT, typename LogitsAt>
__device__ __forceinline__ void score_pages(const WeightsArgs& a, const Work& ws, const int* cum,
                                            int64_t start, int64_t end, int w, int lane, int rows,
                                            uint8_t* mine, const LogitsAt& logits_at) {
  int64_t x = start;
  while (x < end) {
    const Place at = find(cum, a.B, a.Hkv, x);
    const int L = __ldg(a.context_lens + at.b);
    const int n = static_cast<int>(min(static_cast<int64_t>(at.pages - at.page), end - x));
    const int64_t partition = static_cast<int64_t>(at.b) * a.Hkv + at.h + w;
    score_segment<D, KV, NT>(a, at, L, n, x, start, lane, rows, mine,
                             ws.stats + partition * (8 * NT), logits_at);
    x += n;
  }
}

// The weights of one segment from its logits: pages [x0, x0 + n) of the line, from
// page `first` on of the unit.  st: reference and 1 / sum of row lane % R.  From
// the end (the logits written last are the likeliest in L2), a few pages at a
// time, whose logits are asked for together.
template <int NT, typename LogitsAt>
__device__ __forceinline__ void finish_pages(const WeightsArgs& a, float* weights, int L, int first,
                                             int n, int64_t x0, int64_t start, float2 st, int lane,
                                             const float* old_weights, const LogitsAt& logits_at) {
  const int old_end = a.decay != 0.f ? L - a.fresh : 0;
  auto old_of = [&](int page, int in_page) {
    return x0 + page - start < kOld ? old_weights[(x0 + page - start) * 16 + in_page]
                                               : weights[(first + page) * 16 + in_page];
  };
  // a token a lane, two pages a step
  constexpr int R = 8 * NT;
  constexpr int kGroup = NT == 1 ? 4 : 2;
  F2 minus_top[R / 2], f[R / 2];
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    minus_top[i] = pack(-__shfl_sync(0xffffffffu, st.x, 2 * i), -__shfl_sync(0xffffffffu, st.x, 2 * i + 1));
    f[i] = pack(__shfl_sync(0xffffffffu, st.y, 2 * i), __shfl_sync(0xffffffffu, st.y, 2 * i + 1));
  }
  for (int i = (n - 1) / 2; i >= 0; i -= kGroup) {
    float4 s[kGroup][2 * NT];
    float old[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      const int page = 2 * (i - j) + (lane >> 4);
      old[j] = 0.f;
      if (i - j >= 0 && page < n) {
        const float* in = logits_at(x0 + page);
#pragma unroll
        for (int h = 0; h < 2 * NT; ++h)
          s[j][h] = *reinterpret_cast<const float4*>(in + logit_at(h / 2, lane & 15, h % 2 * 2));
        if ((first + page) * 16 + (lane & 15) < old_end) old[j] = old_of(page, lane & 15);
      }
    }
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      const int page = 2 * (i - j) + (lane >> 4);
      const int tok = (first + page) * 16 + (lane & 15);
      if (i - j < 0 || page >= n || tok >= L) continue;
      F2 sum = pack(0.f, 0.f);
#pragma unroll
      for (int h = 0; h < 2 * NT; ++h) {
        sum = fma2(exp2_2(pack(s[j][h].x, s[j][h].y) + minus_top[2 * h]), f[2 * h], sum);
        sum = fma2(exp2_2(pack(s[j][h].z, s[j][h].w) + minus_top[2 * h + 1]), f[2 * h + 1], sum);
      }
      weights[tok] = a.decay * old[j] + (unpack(sum).x + unpack(sum).y);
    }
  }
}

// 32 rows: from the fragments, a lane's two columns of each tile and a quad's sum.
template <typename LogitsAt>
__device__ __forceinline__ void finish_pages4(const WeightsArgs& a, float* weights, int L, int first,
                                              int n, int64_t x0, int64_t start, float2 st, int lane,
                                              const float* old_weights, const LogitsAt& logits_at) {
  const int old_end = a.decay != 0.f ? L - a.fresh : 0;
  constexpr int kGroup = 3;
  F2 minus_top[4], f[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int r = 8 * t + 2 * (lane & 3);
    minus_top[t] = pack(-__shfl_sync(0xffffffffu, st.x, r), -__shfl_sync(0xffffffffu, st.x, r + 1));
    f[t] = pack(__shfl_sync(0xffffffffu, st.y, r), __shfl_sync(0xffffffffu, st.y, r + 1));
  }
  const int in_page = (lane >> 2) + (lane & 1) * 8;   // the token whose sum the lane will hold
  for (int i = n - 1; i >= 0; i -= kGroup) {
    float4 s[kGroup][4];
    float old[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      old[j] = 0.f;
      if (i - j < 0) continue;
      const float4* in = reinterpret_cast<const float4*>(logits_at(x0 + i - j)) + lane;
#pragma unroll
      for (int t = 0; t < 4; ++t) s[j][t] = in[t * 32];
      if ((lane & 2) == 0 && (first + i - j) * 16 + in_page < old_end)
        old[j] = x0 + i - j - start < kOld
                     ? old_weights[(x0 + i - j - start) * 16 + in_page]
                     : weights[(first + i - j) * 16 + in_page];
    }
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      if (i - j < 0) break;
      F2 lo = pack(0.f, 0.f), hi = lo;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        lo = fma2(exp2_2(pack(s[j][t].x, s[j][t].y) + minus_top[t]), f[t], lo);
        hi = fma2(exp2_2(pack(s[j][t].z, s[j][t].w) + minus_top[t]), f[t], hi);
      }
      float x = unpack(lo).x + unpack(lo).y, y = unpack(hi).x + unpack(hi).y;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
      }
      const int tok = (first + i - j) * 16 + in_page;
      if ((lane & 2) == 0 && tok < L) weights[tok] = a.decay * old[j] + (lane & 1 ? y : x);
    }
  }
}

// Joins values first, first + step, ... below n of st, eight of them on their way at a
// time (one after the other: 1 us more for units of 228 partitions of 32 rows).
__device__ __forceinline__ float2 join_strided(const float2* st, int first, int n, int step) {
  constexpr int kBatch = 8;
  float m = kNoScore, l = 0.f;
  for (int i = first; i < n; i += kBatch * step) {
    float2 v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      v[j] = i + j * step < n ? __ldcg(st + i + j * step) : make_float2(kNoScore, 0.f);
    float top = m;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) top = fmaxf(top, v[j].x);
    l *= fast_exp2(m - top);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) l += v[j].y * fast_exp2(v[j].x - top);
    m = top;
  }
  return make_float2(m, l);
}

// Joins the partitions [0, n) of a unit at st (R rows each): by one warp, lane
// i taking row i % R of every 32 / R-th partition.
template <int R>
__device__ __forceinline__ float2 join_by_warp(const float2* st, int n, int lane) {
  float2 v = join_strided(st, lane, n * R, 32);
#pragma unroll
  for (int o = R; o < 32; o <<= 1)
    stat_join(v.x, v.y, __shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
  return v;   // of row lane % R
}

// A unit of more partitions than this is joined by a whole CTA, once for its
// warps: at most two such units (its first and its last) reach into a CTA's pages.
constexpr int kWarpJoin = 16;

template <int D, int KV, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kWarps * 32, Shape<D, NT>::kCtas)
weights_kernel(const __grid_constant__ WeightsArgs a, Work ws) {
  using S = Shape<D, NT>;
  constexpr int R = 8 * NT;
  constexpr int kThreads = S::kWarps * 32;
  extern __shared__ __align__(16) uint8_t warp_smem[];
  __shared__ int cum[kPrefix];
  __shared__ int warp_sums[S::kWarps];
  __shared__ float2 joined[2][R];
  __shared__ float2 scratch[kThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  const int w_first = blockIdx.x * S::kWarps, w = w_first + (tid >> 5);
  const uint32_t call = ld_relaxed_b32(ws.sync + 1) + 1;   // changed only when all CTAs are done
  prefix_pages<S::kWarps>(a, cum, warp_sums);
  const Line line = make_line(a, cum, static_cast<int>(gridDim.x) * S::kWarps);
  if (w_first >= line.workers) return;   // the whole CTA
  const int w_last = min(w_first + S::kWarps, line.workers);
  const int rows = a.n_q * a.group;
  const int64_t start = part_start(line, min(w, line.workers));
  const int64_t end = part_start(line, min(w + 1, line.workers));
  uint8_t* mine = warp_smem + (tid >> 5) * S::kWarpBytes;
  float* kept = reinterpret_cast<float*>(mine);
  float* old_weights = reinterpret_cast<float*>(mine + S::kOldAt);
  // the logits of page x: of the warp's first kKept in shared memory
  auto logits_at = [&](int64_t x) {
    return x - start < S::kKept ? kept + (x - start) * (S::kPage * 4) : ws.logits + x * (S::kPage * 4);
  };
  score_pages<D, KV, NT>(a, ws, cum, start, end, w, lane, rows, mine, logits_at);
  __syncwarp();   // the release covers what the other lanes have written
  if (lane == 0 && w < line.workers && w != a.silent_warp) st_release_gpu_b32(ws.sync + 2 + w, call);
  cp_async_wait_all();   // the old weights, each lane's own copies
  __syncwarp();

  // units of many partitions are joined by the whole CTA
  int long_unit[2] = {-1, -1};
  bool ok = true;
  {
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
      ok = await_warps(ws, w0, n, call, tid, kThreads, a.status, a.wait_limit_ns);
      ok = __syncthreads_and(ok);
      if (!ok) break;
      const float2* st = ws.stats + (static_cast<int64_t>(unit) + w0) * R;
      float2 v = join_strided(st, tid, n * R, kThreads);
      scratch[tid] = v;
      __syncthreads();
      if (tid < R) {
        for (int i = tid + R; i < kThreads; i += R) stat_join(v.x, v.y, scratch[i].x, scratch[i].y);
        joined[e][tid] = v;
      }
      __syncthreads();
    }
  }
  int64_t x = ok ? end : start;
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
      const int parts = part_of(line, at.unit_start + at.pages - 1) - w0 + 1;
      const bool there = await_warps(ws, w0, parts, call, lane, 32, a.status, a.wait_limit_ns);
      if (!__all_sync(0xffffffffu, there)) break;
      __syncwarp();   // what any lane has waited for is seen by all
      st = join_by_warp<R>(ws.stats + (static_cast<int64_t>(unit) + w0) * R, parts, lane);
    }
    // an empty row's and a padding row's tokens get 0
    st.y = lane % R < rows && (st.y > 0.f || st.y != st.y) ? 1.f / st.y : 0.f;
    float* weights = a.weights + static_cast<int64_t>(unit) * a.stride;
    if constexpr (NT == 4)
      finish_pages4(a, weights, L, at.page - n + 1, n, x - n, start, st, lane, old_weights, logits_at);
    else
      finish_pages<NT>(a, weights, L, at.page - n + 1, n, x - n, start, st, lane, old_weights,
                       logits_at);
    x -= n;
  }
  // the last CTA closes the call
  __syncthreads();
  if (tid == 0) {
    const uint32_t ctas = static_cast<uint32_t>((line.workers + S::kWarps - 1) / S::kWarps);
    __threadfence();
    const uint32_t done = atomicAdd(ws.sync, 1u);
    if (done == ctas - 1) {
      atomicExch(ws.sync, 0u);
      atomicExch(ws.sync + 1, call);
    } else if (done >= ctas) {
      atomicOr(a.status, kStatusWsDirty);   // a count that no call leaves
    }
  }
}

// The other kernel: one cluster of CTAs per (kv head, sequence), whose warps divide
// its pages and join their statistics through distributed shared memory; the
// hardware deals the clusters out, and none waits for another.  A warp's logits
// behind the first kKept pages go to the workspace.
constexpr int kMaxCluster = 8;

template <int D, int KV, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kWarps * 32, Shape<D, NT>::kCtas)
weights_unit_kernel(const __grid_constant__ WeightsArgs a, float* spilled, int64_t unit_pages) {
  using S = Shape<D, NT>;
  constexpr int R = 8 * NT;
  extern __shared__ __align__(16) uint8_t warp_smem[];
  __shared__ __align__(16) float2 stats[S::kWarps][R];
  __shared__ __align__(8) float2 cta_stats[R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
  const int h = blockIdx.x / size, b = blockIdx.y;
  const int L = checked_len(a, b, blockIdx.x == 0 && tid == 0);
  if (L == 0) return;   // the whole cluster
  const int pages = (L + 15) / 16, rows = a.n_q * a.group;
  const int w = rank * S::kWarps + warp, warps = size * S::kWarps;
  const int start = static_cast<int>(static_cast<int64_t>(pages) * w / warps);
  const int n = static_cast<int>(static_cast<int64_t>(pages) * (w + 1) / warps) - start;
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  uint8_t* mine = warp_smem + warp * S::kWarpBytes;
  float* kept = reinterpret_cast<float*>(mine);
  float* old_weights = reinterpret_cast<float*>(mine + S::kOldAt);
  float* behind = spilled + unit * unit_pages * (S::kPage * 4);
  auto logits_at = [&](int64_t x) {
    return x - start < S::kKept ? kept + (x - start) * (S::kPage * 4) : behind + x * (S::kPage * 4);
  };
  const Place at{b, h, start, pages, 0};
  if (n > 0)
    score_segment<D, KV, NT>(a, at, L, n, start, start, lane, rows, mine, stats[warp], logits_at);
  else
    for (int r = lane; r < R; r += 32) stats[warp][r] = make_float2(kNoScore, 0.f);
  cp_async_wait_all();
  __syncthreads();
  float2 st = stats[0][lane % R];
#pragma unroll
  for (int i = 1; i < S::kWarps; ++i)
    stat_join(st.x, st.y, stats[i][lane % R].x, stats[i][lane % R].y);
  if (size > 1) {
    if (tid < R) cta_stats[tid] = st;
    cluster_sync();
    float2 all[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      all[r] = r < size ? ld_cluster2(&cta_stats[lane % R], r) : make_float2(kNoScore, 0.f);
    st = all[0];
#pragma unroll
    for (int r = 1; r < kMaxCluster; ++r) stat_join(st.x, st.y, all[r].x, all[r].y);
    cluster_arrive();   // nobody's statistics are read any more, once all have arrived
  }
  st.y = lane % R < rows && (st.y > 0.f || st.y != st.y) ? 1.f / st.y : 0.f;
  float* weights = a.weights + unit * a.stride;
  if constexpr (NT == 4)
    finish_pages4(a, weights, L, start, n, start, start, st, lane, old_weights, logits_at);
  else
    finish_pages<NT>(a, weights, L, start, n, start, start, st, lane, old_weights, logits_at);
  if (size > 1) cluster_wait();
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

// CTAs a unit is divided among by the cluster kernel, 0 for the cooperative one.
// Up to 4096 tokens a cluster a unit: with 400 units of up to 512 and 2048 tokens 14.7
// and 33.6 us against 23.6 and 45.6, with 96 units 8.3 and 15.1 against 14.2 and 22.2,
// with 4 units 6.3 and 7.9 against 12.4 (fp16, head_dim 128, 7 rows); longer units
// divide too unevenly when their lengths differ (512 units, median 1024, bound 8192:
// 69 us against 57).  Two CTAs and more while all fit the GPU at once and each warp
// has a page, or while a warp has more than 16.
int unit_cluster(const WeightsArgs& a, int warps, int ctas) {
  const int64_t pages = (static_cast<int64_t>(a.max_context_len) + 15) / 16;
  if (pages > kWeightsClusterPages) return 0;
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv, slots = static_cast<int64_t>(ctas) * device_sm_count();
  int c = 1;
  while (c < kMaxCluster && ((units * 2 * c <= slots && pages > warps * c) || pages > 16 * warps * c)) c *= 2;
  return c;
}

template <int D, int KV, int NT>
cudaError_t launch_tiles(const WeightsArgs& a, const Work& ws, cudaStream_t s) {
  using S = Shape<D, NT>;
  const int cluster = unit_cluster(a, S::kWarps, S::kCtas);
  auto* kernel = weights_kernel<D, KV, NT>;
  auto* unit_kernel = weights_unit_kernel<D, KV, NT>;
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
      if (cudaError_t e = cudaFuncSetAttribute(
              unit_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem))
        return e;
      raised[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cluster > 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(a.Hkv) * cluster, a.B);
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    const int64_t unit_pages = (static_cast<int64_t>(a.max_context_len) + 15) / 16;
    return cudaLaunchKernelEx(&cfg, unit_kernel, a, ws.logits, unit_pages);
  }
  cfg.gridDim = dim3(weights_grid(a, S::kWarps, S::kCtas));
  attr.id = cudaLaunchAttributeCooperative;   // the CTAs wait for one another
  attr.val.cooperative = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, ws);
}

template <int D, int KV>
cudaError_t launch_pass(const WeightsArgs& a, int nt, const Work& ws, cudaStream_t s) {
  return nt == 1 ? launch_tiles<D, KV, 1>(a, ws, s) : nt == 2 ? launch_tiles<D, KV, 2>(a, ws, s)
                                                              : launch_tiles<D, KV, 4>(a, ws, s);
}

// The words at the start of a workspace: the same ones for every call.
size_t sync_bytes() { return align256((2 + 2 * device_sm_count() * kMaxWarps) * sizeof(uint32_t)); }

}  // namespace

size_t weights_workspace_bytes(int B, int Hkv, int max_context_len, int rows) {
  const size_t nt = tiles_of(rows);
  if (B > kWeightsMaxBatch) B = kWeightsMaxBatch;
  const size_t units = static_cast<size_t>(B) * Hkv;
  const size_t pages = units * ((static_cast<size_t>(max_context_len) + 15) / 16);
  const size_t parts = units + static_cast<size_t>(2 * device_sm_count()) * kMaxWarps;
  return sync_bytes() + align256(pages * nt * 32 * sizeof(float4)) +
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
      ws.sync = reinterpret_cast<uint32_t*>(base);
      base += sync_bytes();
      ws.logits = reinterpret_cast<float*>(base);
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
