// evict.cu -- a cache cut to a budget by accumulated attention weight.
//
// For each (sequence, kv head) of a sequence longer than `keep`: the first f
// tokens, the last r, and of those between them the k = keep - f - r heaviest
// (of equal weights the lowest index).  Two launches, the second a programmatic
// dependent of the first (or one, for small caches):
//   select: the k-th largest weight by radix selection on order-preserving
//           32-bit keys, then the kept positions in order, with their weights;
//   move:   the kept tokens' K and V rows gathered into the spare blocks.
// Bytes: the weights once (4 a token), the kept rows of K and V read once and
// written once.  Measured on a GB300: 29 us for 48 sequences of 1100 to 4096 tokens
// cut to 1024 (2 fp16 kv heads of 128, 102 MB): 8.5 us to select, 16 us to move at 93
// % of the measured copy bandwidth, the rest launches; 43 us for 8 E4M3 sequences of
// 20000 to 32768 cut to 4099 (4 kv heads of 128, 72 MB): 18 us to select, 23 us to
// move, bound by the re-encoding's instructions (1050 a page and pool); 12 to 13 us for
// four small sequences in one launch.
#include <mutex>

#include "pa_cluster.cuh"
#include "pa_e4m3.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

// ------------------------------------------------- distributed shared memory
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_cluster(p, rank)));
  return v;
}
__device__ __forceinline__ int4 ld_cluster4(const int* p, uint32_t rank) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(in_cluster(p, rank)));
  return v;
}

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

// ------------------------------------------------------------------ one page
// Four E4M3 codes c of a row with page scale s become codes under page scale S:
// E4M3(fl(fl(c s) / S)), both roundings to fp32, without dividing.  That quotient
// is within 2^-23 of c s / S, and c r with r = fl(s fl(1 / S)) (1 -+ 2^-21) is below
// and above it for certain (four roundings of 2^-24 are half of 2^-21); rounding to
// a code is monotone, so where both give the same code it is the right one.  About
// 3 pages in 100 have a code where they differ and are divided out.
__device__ __forceinline__ float2 mul2(float2 x, float f) {   // one instruction
  uint64_t a, b, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(b) : "f"(f));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  float2 out;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(out.x), "=f"(out.y) : "l"(r));
  return out;
}
__device__ __forceinline__ uint32_t recode4(uint32_t codes, float r_lo, float r_hi, uint32_t& differ) {
  const uint32_t h0 = e4m3x2_to_f16x2(codes & 0xffffu), h1 = e4m3x2_to_f16x2(codes >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  const float2 xl = mul2(x, r_lo), yl = mul2(y, r_lo), xh = mul2(x, r_hi), yh = mul2(y, r_hi);
  const uint32_t lo = f32x2_to_e4m3x2(xl.x, xl.y) | f32x2_to_e4m3x2(yl.x, yl.y) << 16;
  const uint32_t hi = f32x2_to_e4m3x2(xh.x, xh.y) | f32x2_to_e4m3x2(yh.x, yh.y) << 16;
  differ |= lo ^ hi;
  return lo;
}

// The largest magnitude among four codes.
__device__ __forceinline__ float amax4(uint32_t codes) {
  const uint32_t h0 = e4m3x2_to_f16x2(codes & 0xffffu), h1 = e4m3x2_to_f16x2(codes >> 16);
  const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&h0)),
                            __habs2(*reinterpret_cast<const __half2*>(&h1)));
  const float2 f = __half22float2(m);
  return fmaxf(f.x, f.y);
}

// One warp moves the E4M3 rows of K (kv 0) or V (1) of one destination page.  The
// page's scale is that of the rows it now holds, so all of them are read before any
// is written.
template <int D>
__device__ __forceinline__ void move_page_e4m3(const EvictArgs& a, int b, int h, int page, int kv,
                                               int dst, int lane) {
  if (dst < 0 || dst >= a.num_blocks) {
    if (lane == 0) atomicOr(a.status, kStatusBadBlock);
    return;
  }
  const int rows = min(16, a.keep - page * 16);
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
  uint32_t codes[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int64_t r = __shfl_sync(0xffffffffu, src_row, j);
    codes[j] = r >= 0 ? load_row_codes<D>(pool + r * D, lane) : 0u;
  }
  // fl(c s) grows with c, so a row's largest value is its largest code's
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    amax = fmaxf(amax, __fmul_rn(amax4(codes[j]), __shfl_sync(0xffffffffu, src_scale, j)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = e4m3_page_scale(amax);
  const int64_t tile = static_cast<int64_t>(dst) * a.Hkv + h;
  if (lane == 0) scales[tile] = scale;
  const unsigned live_rows = __ballot_sync(0xffffffffu, src_row >= 0);
  uint8_t* to = pool + tile * 16 * D;
  // lane j: row j's factor; out of range (or not a number): divided out
  const float factor = src_scale * __fdiv_rn(1.f, scale);
  uint32_t differ = src_row >= 0 && !(factor < 0x1p20f) ? 1u : 0u;
  if (!(scale > 0x1p-100f && scale < 0x1p100f)) differ = 1u;
  uint32_t out[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float r = __shfl_sync(0xffffffffu, factor, j);
    out[j] = recode4(codes[j], r * (1.f - 0x1p-21f), r * (1.f + 0x1p-21f), differ);
  }
  if (__any_sync(0xffffffffu, differ != 0)) {
#pragma unroll 1
    for (int j = 0; j < rows; ++j) {
      const float s = __shfl_sync(0xffffffffu, src_scale, j);
      uint32_t c = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) c = i == j ? codes[i] : c;
      c = e4m3x2_rescale(c & 0xffffu, s, scale) | e4m3x2_rescale(c >> 16, s, scale) << 16;
      if (live_rows >> j & 1) store_row_codes<D>(to + j * D, lane, c);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (live_rows >> j & 1) store_row_codes<D>(to + j * D, lane, out[j]);
}

// ------------------------------------------------------------------- select
// One cluster of CTAs per (kv head, sequence): each takes a contiguous part of the
// candidates, each warp of it a contiguous part of that, so that positions come
// out in order with scans over the parts' counts and ballots inside a warp.  A
// part of up to kKeys candidates stays in the threads' registers (ONE); longer
// ones are read again, from L2, in every step.
//
// Radix selection in digits of 11, 11 and 10 bits.  The first digit's histogram
// sees every key, and the weights' few exponents would make the lanes of a warp
// add to the same few bins: four copies, one for every fourth lane.  Once the bin
// that is found holds at most kListed keys, they are listed and each thread counts
// the larger ones of one, instead of more digits (the count grows with the square:
// 256 keys take what a digit takes, 490 took 5 us more).  The CTAs'
// histograms and lists are joined through distributed shared memory; every CTA
// does the whole search for itself.
constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kPer = 16;                                 // keys a thread
constexpr int kKeys = kSelectThreads * kPer;             // a CTA
constexpr int kMaxSelectCluster = 8;
constexpr int kBins = 2048;
constexpr int kCopies = 4;
constexpr int kListed = 256;             // keys that are ranked directly
constexpr int64_t kMoveAlong = 16384;    // elements of K that a CTA moves along with its selection
constexpr int kSelectSmem = (kCopies + 3) * kBins * 4;   // the copies, and each digit's histogram

// Exclusive sum of v over the CTA's threads.
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
  int before = lane < warp ? warp_sums[lane & (kSelectWarps - 1)] : 0;
  before = __reduce_add_sync(0xffffffffu, before);
  __syncthreads();
  return before + s - v;
}

// MOVE: 1 (16-bit pools) or 2 (E4M3), the unit's own CTAs move its rows, too.
template <bool ONE, int MOVE>
__global__ void __launch_bounds__(kSelectThreads, 2)
evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) int smem[];   // read and written 16 bytes at a time
  int* copies = smem;                    // [bin][copy]
  int* hist = smem + kCopies * kBins;    // [digit][bin], of this CTA
  __shared__ int warp_sums[kSelectWarps];
  __shared__ int warp_gt[kSelectWarps], warp_eq[kSelectWarps];
  __shared__ int cta_gt, cta_eq, s_bin, s_left, s_count, s_listed;
  if (MOVE == 0) griddep_launch_dependents();   // the move may do its prologue
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
  const int h = blockIdx.x / size, b = blockIdx.y;
  const int L = checked_len(a, b, h == 0 && rank == 0 && tid == 0);
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  const bool cut = L > a.keep;
  const int tid_all = rank * kSelectThreads + tid, threads_all = size * kSelectThreads;
  if (h == 0) {
    if (tid_all == 0) a.new_lens[b] = cut ? a.keep : L;
    if (a.tables_out != nullptr)
      for (int i = tid_all; i < a.spare_blocks; i += threads_all)
        a.tables_out[static_cast<int64_t>(b) * a.spare_blocks + i] =
            cut ? a.spare[static_cast<int64_t>(b) * a.spare_blocks + i]
                : i < a.mbs ? a.block_tables[static_cast<int64_t>(b) * a.mbs + i] : -1;
  }
  const float* w = a.weights + unit * a.stride;
  float* w_out = a.weights_out != nullptr ? a.weights_out + unit * a.out_stride : nullptr;
  int32_t* kept = a.kept + unit * a.keep;
  // the protected ends, or, uncut, everything
  const int head = cut ? a.first : L, tail = cut ? a.recent : 0;
  for (int i = tid_all; i < head + tail; i += threads_all) {
    const int t = i < head ? i : L - tail + (i - head);
    const int pos = i < head ? i : a.keep - tail + (i - head);
    kept[pos] = t;
    if (w_out != nullptr) w_out[pos] = w[t];
  }
  if (!cut) return;                            // the whole cluster
  const int k = a.keep - a.first - a.recent;   // how many of the m candidates stay; k < m
  if (k > 0) {
    const int m = L - a.first - a.recent;
    const float* cand = w + a.first;
    const int share = ((m + size - 1) / size + 31) / 32 * 32;
    const int cta_lo = static_cast<int>(min(static_cast<int64_t>(rank) * share, static_cast<int64_t>(m)));
    const int cta_hi = min(cta_lo + share, m);
    const int part = ((cta_hi - cta_lo + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int lo = min(cta_lo + warp * part, cta_hi), hi = min(lo + part, cta_hi);

    uint32_t key[kPer];
    auto load = [&](int i0) {   // the keys of candidates i0 + 32 j + lane
      float v[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = i0 + 32 * j + lane < hi ? __ldg(cand + i0 + 32 * j + lane) : 0.f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) key[j] = weight_key(v[j]);
    };
    // f(key, candidate, whether it is one), warp by warp in order
    auto for_keys = [&](auto f) {
      if constexpr (ONE) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) f(key[j], lo + 32 * j + lane, lo + 32 * j + lane < hi);
      } else {
        for (int i0 = lo; i0 < hi; i0 += 32 * kPer) {
          load(i0);
#pragma unroll
          for (int j = 0; j < kPer; ++j) f(key[j], i0 + 32 * j + lane, i0 + 32 * j + lane < hi);
        }
      }
    };
    if constexpr (ONE) load(lo);
    uint32_t prefix = 0;   // the k-th largest key's digits so far
    int left = k;          // how many of the keys with that prefix stay
    // The k-th largest key itself, from a list of the `count` keys that have the
    // prefix in the bits `found`: the one that has fewer than `left` larger ones.
    auto rank_listed = [&](uint32_t found, int count) {
      uint32_t* list = reinterpret_cast<uint32_t*>(hist + 2 * kBins);   // this CTA's, then all keys
      uint32_t* all = list + kListed;
      for_keys([&](uint32_t x, int, bool in) {
        const unsigned hit = __ballot_sync(0xffffffffu, in && (x & found) == prefix);
        if (hit == 0) return;
        int at = 0;
        if (lane == 0) at = atomicAdd(&s_listed, __popc(hit));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(hit & ((1u << lane) - 1));
        if (hit >> lane & 1) list[at] = x;
      });
      if (size > 1) cluster_sync();
      else __syncthreads();
      uint32_t x = 0;
      if (tid < count) {
        int listed[kMaxSelectCluster], r = 0, i = tid;
#pragma unroll
        for (int j = 0; j < kMaxSelectCluster; ++j) listed[j] = j < size ? ld_cluster(&s_listed, j) : 0;
#pragma unroll
        for (int j = 0; j < kMaxSelectCluster - 1; ++j)
          if (r == j && i >= listed[j]) i -= listed[j], ++r;
        x = static_cast<uint32_t>(ld_cluster(reinterpret_cast<int*>(list + i), r));
      }
      if (tid < kListed) all[tid] = x;   // those behind the count are 0: larger than none
      __syncthreads();
      if (tid < count) {
        int larger = 0, same = 0;
        for (int i = 0; i < count; i += 4) {
          const uint4 y = *reinterpret_cast<const uint4*>(all + i);
          larger += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
          same += (y.x == x) + (y.y == x) + (y.z == x) + (y.w == x);
        }
        if (larger < left && left <= larger + same) {   // every thread with this key
          s_bin = static_cast<int>(x);
          s_left = left - larger;
        }
      }
      __syncthreads();
      prefix = static_cast<uint32_t>(s_bin);
      left = s_left;
    };
    if (tid == 0) s_listed = 0;
    const bool few = m <= kListed;   // all of them are ranked directly
    if (!few)
      for (int i = tid; i < (kCopies + 3) * kBins / 4; i += kSelectThreads)
        reinterpret_cast<int4*>(smem)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (few) rank_listed(0u, m);
#pragma unroll
    for (int digit = 0; digit < 3; ++digit) {
      if (few) break;
      const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
      const int bins = digit == 2 ? 1024 : 2048;
      int* mine = hist + digit * kBins;
      if (digit == 0) {
        for_keys([&](uint32_t x, int, bool in) {
          if (in) atomicAdd(&copies[(x >> 21) * kCopies + (lane & (kCopies - 1))], 1);
        });
        __syncthreads();
        for (int i = tid; i < kBins; i += kSelectThreads) {
          const int4 c = reinterpret_cast<const int4*>(copies)[i];
          mine[i] = c.x + c.y + c.z + c.w;
        }
      } else {
        const uint32_t mask = digit == 1 ? 0xffe00000u : 0xfffffc00u;
        for_keys([&](uint32_t x, int, bool in) {
          if (in && (x & mask) == prefix) atomicAdd(&mine[(x >> shift) & (bins - 1)], 1);
        });
      }
      if (size > 1) cluster_sync();
      else __syncthreads();
      // the bin, from the largest down, in which the left-th key lies
      // (four bins a thread, every CTA's asked for before any is used)
      constexpr int kEach = 4;
      static_assert(kEach * kSelectThreads == kBins, "");
      int c[kEach] = {}, sum = 0;
      const int low = bins - kEach * (tid + 1);   // the thread's lowest bin
      if (low >= 0) {
        int4 part[kMaxSelectCluster];
#pragma unroll
        for (int r = 0; r < kMaxSelectCluster; ++r)
          part[r] = r < size ? ld_cluster4(mine + low, r) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < kMaxSelectCluster; ++r)
          c[0] += part[r].w, c[1] += part[r].z, c[2] += part[r].y, c[3] += part[r].x;
        sum = c[0] + c[1] + c[2] + c[3];
      }
      int over = block_scan(sum, warp_sums);
      if (over < left && over + sum >= left) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          if (over < left && over + c[j] >= left) {
            s_bin = bins - 1 - (tid * kEach + j);
            s_left = left - over;
            s_count = c[j];
          }
          over += c[j];
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(s_bin) << shift;
      left = s_left;
      const int count = s_count;
      __syncthreads();
      if (digit < 2 && count <= kListed) {
        rank_listed(digit == 0 ? 0xffe00000u : 0xfffffc00u, count);
        break;
      }
    }
    // every part's larger keys and ties, then the positions in order
    int gt = 0, eq = 0;
    for_keys([&](uint32_t x, int, bool in) {
      gt += in && x > prefix;
      eq += in && x == prefix;
    });
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) warp_gt[warp] = gt, warp_eq[warp] = eq;
    __syncthreads();
    int pos = lane < warp ? warp_gt[lane & (kSelectWarps - 1)] : 0;
    int ties = lane < warp ? warp_eq[lane & (kSelectWarps - 1)] : 0;
    pos = __reduce_add_sync(0xffffffffu, pos);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (size > 1) {
      if (tid == kSelectThreads - 1) cta_gt = pos + gt, cta_eq = ties + eq;
      cluster_sync();
      int gts[kMaxSelectCluster], eqs[kMaxSelectCluster];
#pragma unroll
      for (int r = 0; r < kMaxSelectCluster; ++r) {
        gts[r] = r < rank ? ld_cluster(&cta_gt, r) : 0;
        eqs[r] = r < rank ? ld_cluster(&cta_eq, r) : 0;
      }
#pragma unroll
      for (int r = 0; r < kMaxSelectCluster; ++r) pos += gts[r], ties += eqs[r];
    }
    pos += a.first + min(ties, left);
    const unsigned below = (1u << lane) - 1;
    for_keys([&](uint32_t x, int i, bool in) {
      const unsigned tied = __ballot_sync(0xffffffffu, in && x == prefix);
      const bool stay = in && (x > prefix || (x == prefix && ties + __popc(tied & below) < left));
      const unsigned staying = __ballot_sync(0xffffffffu, stay);
      if (stay) {
        const int at = pos + __popc(staying & below);
        kept[at] = a.first + i;
        if (w_out != nullptr) w_out[at] = __ldg(cand + i);
      }
      pos += __popc(staying);
      ties += __popc(tied);
    });
  }
  // nobody's shared memory is read any more, and all kept positions are seen
  if (size > 1) cluster_sync();
  else __syncthreads();
  if constexpr (MOVE != 0) {
    const int32_t* spare = a.spare + static_cast<int64_t>(b) * a.spare_blocks;
    if constexpr (MOVE == 1) {
      const int chunks = a.D / 8;
      const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.mbs;
      for (int i = tid_all; i < a.keep * chunks; i += threads_all) {
        const int row = i / chunks, c = i - row * chunks;
        const int t = kept[row];
        const int src = __ldg(table + t / 16), dst = __ldg(spare + row / 16);
        if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
          atomicOr(a.status, kStatusBadBlock);
          continue;
        }
        const int64_t from = ((static_cast<int64_t>(src) * a.Hkv + h) * 16 + t % 16) * chunks + c;
        const int64_t to = ((static_cast<int64_t>(dst) * a.Hkv + h) * 16 + row % 16) * chunks + c;
        static_cast<uint4*>(a.k_cache)[to] = static_cast<const uint4*>(a.k_cache)[from];
        static_cast<uint4*>(a.v_cache)[to] = static_cast<const uint4*>(a.v_cache)[from];
      }
    } else {
      for (int i = tid_all >> 5; i < ((a.keep - 1) / 16 + 1) * 2; i += threads_all >> 5) {
        const int dst = __ldg(spare + (i >> 1));
        if (a.D == 128) move_page_e4m3<128>(a, b, h, i >> 1, i & 1, dst, lane);
        else move_page_e4m3<64>(a, b, h, i >> 1, i & 1, dst, lane);
      }
    }
  }
}

// --------------------------------------------------------------------- move
// A thread moves one 16-byte chunk of K and of V of kDeep pages; all its loads are
// made before the stores.
constexpr int kMoveThreads = 256;
constexpr int kDeep = 4;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int C = D / 8;                          // 16-byte chunks a row
  constexpr int kPages = kMoveThreads / (16 * C);   // that the CTA's threads cover at once
  const int h = blockIdx.y, b = blockIdx.z;
  const int L = checked_len(a, b, false);
  const int row = threadIdx.x / C % 16, c = threadIdx.x % C;
  const int page0 = blockIdx.x * kDeep * kPages + threadIdx.x / (16 * C);
  const int32_t* spare = a.spare + static_cast<int64_t>(b) * a.spare_blocks;
  int dst[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int page = page0 + j * kPages;
    dst[j] = -1;
    if (L > a.keep && page * 16 + row < a.keep) {
      dst[j] = __ldg(spare + page);
      if (dst[j] < 0 || dst[j] >= a.num_blocks) {
        atomicOr(a.status, kStatusBadBlock);
        dst[j] = -1;
      }
    }
  }
  griddep_wait();   // the kept positions are written
  const int32_t* kept = a.kept + (static_cast<int64_t>(b) * a.Hkv + h) * a.keep;
  const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.mbs;
  int t[kDeep], src[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) t[j] = dst[j] >= 0 ? kept[(page0 + j * kPages) * 16 + row] : 0;
#pragma unroll
  for (int j = 0; j < kDeep; ++j) src[j] = dst[j] >= 0 ? __ldg(table + t[j] / 16) : 0;
  uint4 kv[kDeep][2];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    if (src[j] < 0 || src[j] >= a.num_blocks) {
      atomicOr(a.status, kStatusBadBlock);
      dst[j] = -1;
    }
    if (dst[j] < 0) continue;
    const int64_t from = ((static_cast<int64_t>(src[j]) * a.Hkv + h) * 16 + t[j] % 16) * C + c;
    kv[j][0] = __ldcs(static_cast<const uint4*>(a.k_cache) + from);
    kv[j][1] = __ldcs(static_cast<const uint4*>(a.v_cache) + from);
  }
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    if (dst[j] < 0) continue;
    const int64_t to = ((static_cast<int64_t>(dst[j]) * a.Hkv + h) * 16 + row) * C + c;
    static_cast<uint4*>(a.k_cache)[to] = kv[j][0];
    static_cast<uint4*>(a.v_cache)[to] = kv[j][1];
  }
}

// E4M3: one warp per (destination page, kv head, sequence, K|V).
constexpr int kMoveE4m3Warps = 4;

template <int D>
__global__ void __launch_bounds__(kMoveE4m3Warps * 32, 12)
evict_move_e4m3_kernel(const __grid_constant__ EvictArgs a) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int page = blockIdx.x * (kMoveE4m3Warps / 2) + (threadIdx.x >> 6);
  const bool live = checked_len(a, b, false) > a.keep && page * 16 < a.keep;
  const int dst = live ? __ldg(a.spare + static_cast<int64_t>(b) * a.spare_blocks + page) : 0;
  griddep_wait();   // the kept positions are written
  if (live) move_page_e4m3<D>(a, b, h, page, threadIdx.x >> 5 & 1, dst, threadIdx.x & 31);
}

template <bool ONE, int MOVE>
cudaError_t launch_select(const EvictArgs& a, int cluster, cudaStream_t s) {
  {
    // more than 48 KB of shared memory has to be asked for, once per device
    static std::mutex mu;
    static bool raised[kMaxDevices] = {};
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!raised[dev]) {
      if (cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<ONE, MOVE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectSmem))
        return e;
      raised[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.Hkv) * cluster, a.B);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = kSelectSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<ONE, MOVE>, a);
}

template <typename Kernel>
cudaError_t launch_move(Kernel* kernel, const EvictArgs& a, int pages, int threads, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(((a.keep - 1) / 16 + pages) / pages, a.Hkv, a.B);
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
  // as many CTAs a unit as hold its candidates in registers, up to a portable cluster
  int cluster = 1;
  while (cluster < kMaxSelectCluster && a.max_context_len > cluster * kKeys) cluster *= 2;
  const bool one = a.max_context_len <= cluster * kKeys;
  // A unit's CTAs move what is soon moved; more is worth a launch of its own, which
  // all SMs share.  At head_dim 128, one launch against two: with 64 rows 1 to 2 us
  // less; with 128 rows the same for 4 units, 2 us less for 128; with 256 rows 2.5 us
  // more for 4 units, 4 us more for 128.
  if (static_cast<int64_t>(a.keep) * a.D <= kMoveAlong * cluster)
    return fp8 ? (one ? launch_select<true, 2>(a, cluster, s) : launch_select<false, 2>(a, cluster, s))
               : (one ? launch_select<true, 1>(a, cluster, s) : launch_select<false, 1>(a, cluster, s));
  if (cudaError_t e = one ? launch_select<true, 0>(a, cluster, s) : launch_select<false, 0>(a, cluster, s))
    return e;
  if (a.keep >= a.max_context_len) return cudaSuccess;   // nothing can be cut
  if (fp8)
    return launch_move(a.D == 128 ? evict_move_e4m3_kernel<128> : evict_move_e4m3_kernel<64>, a,
                       kMoveE4m3Warps / 2, kMoveE4m3Warps * 32, s);
  return a.D == 128 ? launch_move(evict_move_kernel<128>, a, kDeep, kMoveThreads, s)
                    : launch_move(evict_move_kernel<64>, a, 2 * kDeep, kMoveThreads, s);
}

}  // namespace pa
