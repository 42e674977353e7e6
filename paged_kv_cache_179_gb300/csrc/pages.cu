// pages.cu -- the pool's pages by reference counts: taken, given back, shared by
// forks, moved together.
//
// The counts are the only record of which pages are free, so every call that
// takes or moves pages ranks them by one pass over the counts:
//   rank(p) = number of free (or live) pages below p.
// A cluster of CTAs does that: each warp counts its own contiguous part, the CTAs'
// totals are exchanged through distributed shared memory, and a second pass
// (from L2 now) has every page's rank without a second launch or a workspace.
// The page of rank k goes to the item whose needs' prefix sum holds k, found by
// bisection: the lowest free pages, in the items' order, whatever order the
// warps run in.
//
// Latency bounds them, the pages' copies excepted: the counts of a pool of 577k pages are
// 2.3 MB, read once from memory and, where pages are taken, again from L2.  Measured on
// a GB300: 64 rows given back and 256 served from that pool 20 us (two launches; 85 with
// contiguous parts of the pool for the warps and one load in flight); the same in a pool
// of 64 pages 8 us; 96 forks with their copies, after 96 rows are given back, 14 us;
// compaction of 16384 pages, half of them live (132 MB of copies and tables), 28 us,
// 4.7 TB/s; of 49001 E4M3 pages (341 MB) 62 us, 5.5 TB/s, 81 % of a plain copy's rate.
#include <algorithm>
#include <climits>

#include "pa_cluster.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "request_launch.h"

namespace pa {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanCtas = 16;                      // a cluster, for larger pools
// Up to so many pages one CTA ranks by itself, without a cluster's barriers.  64 rows served
// and given back, by one CTA and by a cluster: 11.7 and 13.0 us in 4096 pages, 12.0 and 13.1
// in 16384, 15.4 and 13.4 in 32768.  A compaction that moves nothing: 6.0 and 6.5 us of 4096
// pages, 8.2 and 6.5 of 8192.  (Clusters of 8 take 14.5 us instead of 10.7 for 131072.)
constexpr int kOneCtaTake = 16384, kOneCtaCompact = 4096;
// Where items' pages go is kept in shared memory for up to this many items.
constexpr int kKeptItems = 8192;
constexpr unsigned kMany = (1u << 30) + 1u;        // sums of needs saturate above any pool

__device__ __forceinline__ void st_cluster_u32(void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cluster(p, rank)), "r"(v) : "memory");
}

// The counts of pages 4g .. 4g + 3; those behind the pool's end are `behind`.
__device__ __forceinline__ int4 counts_at(const int32_t* ref, int g, int num_blocks, int behind) {
  const int p = 4 * g;
  if (p + 4 <= num_blocks) return *reinterpret_cast<const int4*>(ref + p);
  int4 c = make_int4(behind, behind, behind, behind);
  if (p < num_blocks) c.x = ref[p];
  if (p + 1 < num_blocks) c.y = ref[p + 1];
  if (p + 2 < num_blocks) c.z = ref[p + 2];
  return c;
}
// Bit i: page 4g + i is free / live.
__device__ __forceinline__ unsigned free_bits(int4 c) {
  return (c.x <= 0) | (c.y <= 0) << 1 | (c.z <= 0) << 2 | (c.w <= 0) << 3;
}
__device__ __forceinline__ unsigned live_bits(int4 c) {
  return (c.x > 0) | (c.y > 0) << 1 | (c.z > 0) << 2 | (c.w > 0) << 3;
}

// Pages of this warp's part whose bits_of(counts) are set.
template <typename F>
__device__ __forceinline__ unsigned count_part(const int32_t* ref, int num_blocks, int behind, int g0,
                                               int g1, int lane, F bits_of) {
  unsigned n = 0;
  for (int g = g0; g < g1; g += 128) {             // four loads in flight
    int4 c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      c[u] = g + 32 * u + lane < g1 ? counts_at(ref, g + 32 * u + lane, num_blocks, behind)
                                    : make_int4(behind, behind, behind, behind);
#pragma unroll
    for (int u = 0; u < 4; ++u) n += __popc(bits_of(c[u]));
  }
  return __reduce_add_sync(0xffffffffu, n);
}

// This warp's part of the groups of four pages: an equal contiguous share.
struct Part {
  int g0, g1;
};
template <int CTAS>
__device__ __forceinline__ Part my_part(int num_blocks, uint32_t rank, int warp) {
  const int groups = (num_blocks + 3) / 4;
  const int parts = CTAS * kScanWarps;
  const int per = (groups + parts - 1) / parts;
  const int64_t w = static_cast<int64_t>(rank) * kScanWarps + warp;
  const int g0 = static_cast<int>(min(w * per, static_cast<int64_t>(groups)));
  return Part{g0, min(g0 + per, groups)};
}

// What the warps count, summed: each warp's own `n` in; out, the sum over all
// warps before it and the sum over all of them.  `box` [kScanCtas] and `mine`
// [kScanWarps] in shared memory; a cluster barrier inside.  All CTAs of the cluster
// have started (one reaches into the others' shared memory).
struct Before {
  unsigned before, total;
};
template <int CTAS>
__device__ __forceinline__ Before cluster_prefix(unsigned n, unsigned* mine, unsigned* box, int warp,
                                                 int lane, uint32_t rank) {
  if (lane == 0) mine[warp] = n;
  __syncthreads();
  unsigned sum = mine[lane];                       // kScanWarps == 32
  unsigned inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  const unsigned all = __shfl_sync(0xffffffffu, inc, 31);
  const unsigned in_cta = __shfl_sync(0xffffffffu, inc - sum, warp);
  if (CTAS == 1) return Before{in_cta, all};
  if (warp == 0 && lane < CTAS) st_cluster_u32(box + rank, lane, all);
  cluster_sync();
  Before b{in_cta, 0u};
#pragma unroll
  for (int r = 0; r < CTAS; ++r) {
    const unsigned v = box[r];
    b.before += static_cast<uint32_t>(r) < rank ? v : 0u;
    b.total += v;
  }
  return b;
}

__device__ __forceinline__ unsigned warp_sum(unsigned v) {
  return __reduce_add_sync(0xffffffffu, v);
}
__device__ __forceinline__ unsigned warp_prefix(unsigned v, int lane) {   // exclusive
  unsigned inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  return inc - v;
}

// ---------------------------------------------------------------------- taking
// The free pages that a call takes are the lowest ones, a small part of the pool: the
// warps take chunks of the pages in turn, so that all of them have some of it.
constexpr int kMaxChunks = 4096;
constexpr int kChunkGroups = 128;                  // groups of four pages: 512 pages, or more in large pools
// What item i needs: pages (-1: it is passed over), in which row, from which
// entry of its table on, and how many the row holds with them.
struct Need {
  int pages, row, entry, holds;
};
template <bool FORK>
__device__ __forceinline__ Need need_of(const TakeArgs& a, int i, bool report) {
  Need n{-1, a.rows[i], 0, 0};
  unsigned bad = 0u;
  if (n.row < 0 || n.row >= a.num_rows) {
    bad = kStatusBadRow;
  } else if (FORK) {
    const int src = a.src_rows[i];
    if (src < 0 || src >= a.num_rows || src == n.row) {
      bad = kStatusBadRow;
    } else {
      const int L = a.lens[src], have = a.num_pages[src];
      if (have < 0 || have > a.mbs || L < 0 || L > static_cast<int64_t>(have) * 16) {
        bad = kStatusBadLen;
      } else {
        n.pages = (L & 15) != 0;
        n.entry = L >> 4;
        n.holds = n.entry + n.pages;
      }
    }
  } else {
    const int L = a.lens[i], have = a.num_pages[n.row];
    const int want = static_cast<int>((static_cast<int64_t>(L) + 15) >> 4);
    if (have < 0 || have > a.mbs || L < 0 || want > a.mbs) {
      bad = kStatusBadLen;
    } else {
      n.pages = max(want - have, 0);
      n.entry = have;
      n.holds = max(want, have);
    }
  }
  if (bad && report) atomicOr(a.status, bad);
  return n;
}

template <bool FORK, int CTAS>
__global__ void __launch_bounds__(kScanThreads, 1) take_kernel(const TakeArgs a) {
  // [items + 1]: needs before each item; then, of up to kKeptItems, the place in the tables
  // of the page of rank 0 of each item (-1: passed over)
  extern __shared__ __align__(16) int first[];
  __shared__ unsigned before[kMaxChunks + 1];      // free pages in, then before, each chunk
  __shared__ unsigned sums[2][kScanWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CTAS > 1 ? cluster_rank() : 0u;
  griddep_launch_dependents();
  griddep_wait();
  if (CTAS > 1) cluster_sync();                    // all CTAs have started
  const bool kept = a.items <= kKeptItems;
  int64_t* place = reinterpret_cast<int64_t*>(first + (a.items + 4) / 4 * 4);
  // ---- the free pages of each chunk
  const int groups = (a.num_blocks + 3) / 4;
  const int per_chunk = max(kChunkGroups, ((groups + kMaxChunks - 1) / kMaxChunks + 31) / 32 * 32);
  const int chunks = (groups + per_chunk - 1) / per_chunk;
  constexpr int kWarpsInAll = CTAS * kScanWarps;
  const int me = warp * CTAS + static_cast<int>(rank);
  for (int k = me; k < chunks; k += kWarpsInAll) {
    const int g0 = k * per_chunk;
    const unsigned n = count_part(a.ref_counts, a.num_blocks, 1, g0, min(g0 + per_chunk, groups), lane, free_bits);
    if (CTAS == 1) {
      if (lane == 0) before[k] = n;
    } else if (lane < CTAS) {
      st_cluster_u32(before + k, lane, n);
    }
  }
  // ---- the needs and their prefix sums, by every CTA for itself
  const int per = (a.items + kScanThreads - 1) / kScanThreads;
  const int i0 = min(a.items, tid * per), i1 = min(a.items, i0 + per);
  auto place_of = [&](const Need& n) { return static_cast<int64_t>(n.row) * a.mbs + n.entry; };
  unsigned sum = 0;
  for (int i = i0; i < i1; ++i) {
    const Need n = need_of<FORK>(a, i, rank == 0);
    first[i] = max(n.pages, 0);
    if (kept) place[i] = n.pages < 0 ? -1 : place_of(n);
    sum = min(sum + first[i], kMany);
  }
  if (CTAS > 1) cluster_sync();
  else __syncthreads();
  // ---- both prefix sums: a thread's share first
  constexpr int kMine = kMaxChunks / kScanThreads;
  unsigned free_n = 0;
#pragma unroll
  for (int j = 0; j < kMine; ++j) free_n += tid * kMine + j < chunks ? before[tid * kMine + j] : 0u;
  unsigned inc = sum, inc_free = free_n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(0xffffffffu, inc, o), u = __shfl_up_sync(0xffffffffu, inc_free, o);
    if (lane >= o) {
      inc = min(inc + t, kMany);
      inc_free += u;
    }
  }
  if (lane == 31) {
    sums[0][warp] = inc;
    sums[1][warp] = inc_free;
  }
  const unsigned up = __shfl_up_sync(0xffffffffu, inc, 1);
  __syncthreads();
  unsigned ex = lane > 0 ? up : 0u, ex_free = inc_free - free_n, total = 0;
  for (int w = 0; w < kScanWarps; ++w) {
    if (w < warp) {
      ex = min(ex + sums[0][w], kMany);
      ex_free += sums[1][w];
    }
    total += sums[1][w];
  }
  for (int i = i0; i < i1; ++i) {
    const unsigned pages = first[i];
    first[i] = ex;
    ex = min(ex + pages, kMany);
  }
  if (tid == kScanThreads - 1) first[a.items] = ex;
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (tid * kMine + j < chunks) {
      const unsigned n = before[tid * kMine + j];
      before[tid * kMine + j] = ex_free;
      ex_free += n;
    }
  __syncthreads();
  // ---- items are granted while their last page's rank is there
  auto last_at_most = [&](int v) {                 // the last j with first[j] <= v
    int l = 0, r = a.items + 1;
    while (r - l > 1) {
      const int m = (l + r) >> 1;
      if (first[m] <= v) l = m;
      else r = m;
    }
    return l;
  };
  const unsigned limit = first[last_at_most(static_cast<int>(total))];
  for (int chunk = me; chunk < chunks; chunk += kWarpsInAll) {
    unsigned k0 = before[chunk];
    const int g1 = min((chunk + 1) * per_chunk, groups);
    auto counts = [&](int g) {
      return g + lane < g1 ? counts_at(a.ref_counts, g + lane, a.num_blocks, 1) : make_int4(1, 1, 1, 1);
    };
    if (k0 >= limit) break;                        // (so do those behind)
    int4 c = counts(chunk * per_chunk);
    for (int g = chunk * per_chunk; g < g1 && k0 < limit; g += 32) {
      unsigned bits = free_bits(c);
      if (g + 32 < g1) c = counts(g + 32);         // on their way
      const unsigned mine_n = __popc(bits);
      unsigned k = k0 + warp_prefix(mine_n, lane);
      if (bits != 0u && k < limit) {
        int i = last_at_most(static_cast<int>(k));   // this lane's pages have ranks k, k + 1, ..
        for (; bits != 0u && k < limit; bits &= bits - 1, ++k) {
          while (first[i + 1] <= static_cast<int>(k)) ++i;
          const int page = 4 * (g + lane) + __ffs(bits) - 1;
          const int64_t to = kept ? place[i] : place_of(need_of<FORK>(a, i, false));
          a.block_tables[to + (k - first[i])] = page;
          a.ref_counts[page] = 1;
        }
      }
      k0 += warp_sum(mine_n);
    }
  }
  // ---- what the items hold now, once no CTA reads num_pages any more
  if (CTAS > 1) cluster_sync();
  else __syncthreads();
  if (rank != 0) return;
  for (int i = tid; i < a.items; i += kScanThreads) {
    // (a kept item's need is the difference of the prefix sums, unless those have saturated,
    // and then it is not granted)
    const bool passed_over = kept ? place[i] < 0 : need_of<FORK>(a, i, false).pages < 0;
    const bool ok = !passed_over && static_cast<unsigned>(first[i + 1]) <= total;
    if (!FORK && ok) a.num_pages[a.rows[i]] = need_of<FORK>(a, i, false).holds;
    a.granted[i] = ok;
  }
}

template <bool FORK, int CTAS>
cudaError_t launch_take(const TakeArgs& a, cudaStream_t s) {
  auto* kern = take_kernel<FORK, CTAS>;
  const size_t smem = (static_cast<size_t>(a.items) + 4) / 4 * 16 +
                      (a.items <= kKeptItems ? static_cast<size_t>(a.items) * 8 : 0);
  if (smem > 30 * 1024) {                          // (the default limit is 48 KB with the static arrays)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (kPagesMaxItems + 4) * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CTAS);
  cfg.blockDim = dim3(kScanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0] = after_previous();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CTAS > 1 ? 2 : 1;
  if (CTAS > 1) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kern, a);
}
template <bool FORK>
cudaError_t launch_take(const TakeArgs& a, cudaStream_t s) {
  static_assert(kKeptItems * 12 + 16 <= (kPagesMaxItems + 4) * 4, "one limit serves both layouts");
  return a.num_blocks <= kOneCtaTake ? launch_take<FORK, 1>(a, s) : launch_take<FORK, kScanCtas>(a, s);
}

// -------------------------------------------------------------------- giving back
constexpr int kFreeThreads = 1024;
__global__ void __launch_bounds__(kFreeThreads)
free_kernel(int32_t* tables, int mbs, int32_t* num_pages, int num_rows, const int32_t* rows,
            int32_t* ref, int num_blocks, unsigned* status) {
  __shared__ int held;
  griddep_launch_dependents();
  griddep_wait();
  const int row = rows[blockIdx.x];
  if (row < 0 || row >= num_rows) {
    if (threadIdx.x == 0) atomicOr(status, kStatusBadRow);
    return;
  }
  if (threadIdx.x == 0) {
    const int n = num_pages[row];
    const bool ok = n >= 0 && n <= mbs;
    // the exchange: a row that is listed twice is freed by one of its CTAs
    held = ok ? atomicExch(num_pages + row, 0) : 0;
    if (!ok) atomicOr(status, kStatusBadLen);
  }
  __syncthreads();
  int32_t* t = tables + static_cast<int64_t>(row) * mbs;
  for (int j = threadIdx.x; j < held; j += kFreeThreads) {
    const int id = t[j];
    t[j] = -1;
    bool bad = id < 0 || id >= num_blocks;
    if (!bad && atomicSub(ref + id, 1) <= 0) {     // it was free: back to what it was
      atomicAdd(ref + id, 1);
      bad = true;
    }
    if (bad) atomicOr(status, kStatusBadBlock);
  }
}

// ------------------------------------------------------------------------- copies
constexpr int kPieceChunks = 256;                  // 16-byte chunks a warp has in flight: 4 KB

// Piece `piece` of a page of one pool, by a warp.
__device__ __forceinline__ void copy_piece(uint4* pool, int64_t chunks, int src, int dst, int piece,
                                           int lane) {
  const uint4* from = pool + src * chunks;
  uint4* to = pool + dst * chunks;
  const int64_t c0 = static_cast<int64_t>(piece) * kPieceChunks + lane;
  uint4 r[kPieceChunks / 32];
#pragma unroll
  for (int j = 0; j < kPieceChunks / 32; ++j)
    if (c0 + 32 * j < chunks) r[j] = __ldcs(from + c0 + 32 * j);
#pragma unroll
  for (int j = 0; j < kPieceChunks / 32; ++j)
    if (c0 + 32 * j < chunks) __stcs(to + c0 + 32 * j, r[j]);
}
__device__ __forceinline__ void copy_scales(const PagePools& p, int src, int dst, int lane) {
  for (int h = lane; h < p.Hkv; h += 32) {
    p.k_scale[static_cast<int64_t>(dst) * p.Hkv + h] = p.k_scale[static_cast<int64_t>(src) * p.Hkv + h];
    p.v_scale[static_cast<int64_t>(dst) * p.Hkv + h] = p.v_scale[static_cast<int64_t>(src) * p.Hkv + h];
  }
}

constexpr int kForkThreads = 256;
// One CTA a pair, after its part-full page was taken: the shared pages' ids and
// counts, then the copy.
__global__ void __launch_bounds__(kForkThreads)
fork_kernel(const TakeArgs a, int32_t* context_lens, const PagePools p) {
  griddep_launch_dependents();
  griddep_wait();
  const int i = blockIdx.x;
  if (!a.granted[i]) return;
  const int src = a.src_rows[i], dst = a.rows[i], L = context_lens[src];
  const int full = L >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t* from = a.block_tables + static_cast<int64_t>(src) * a.mbs;
  int32_t* to = a.block_tables + static_cast<int64_t>(dst) * a.mbs;
  if (L & 15) {
    const int old = from[full], mine = to[full];
    // (`mine` is what the launch before took, unless another pair changed src meanwhile)
    if (old < 0 || old >= a.num_blocks || mine < 0 || mine >= a.num_blocks) {
      if (threadIdx.x == 0) atomicOr(a.status, kStatusBadBlock);
    } else {
      const int64_t chunks = p.page_bytes / 16;
      const int pieces = static_cast<int>((chunks + kPieceChunks - 1) / kPieceChunks);
      for (int u = warp; u < 2 * pieces; u += kForkThreads / 32)
        copy_piece(static_cast<uint4*>(u < pieces ? p.k_cache : p.v_cache), chunks, old, mine,
                   u < pieces ? u : u - pieces, lane);
      if (p.k_scale != nullptr && warp == 0) copy_scales(p, old, mine, lane);
    }
  }
  for (int j = threadIdx.x; j < full; j += kForkThreads) {
    const int id = from[j];
    to[j] = id;
    if (id >= 0 && id < a.num_blocks) atomicAdd(a.ref_counts + id, 1);
    else atomicOr(a.status, kStatusBadBlock);
  }
  if (threadIdx.x == 0) {
    a.num_pages[dst] = full + ((L & 15) != 0);
    context_lens[dst] = L;
  }
}

// --------------------------------------------------------------------- compaction
// Workspace: the number of moves, then the free pages below num_live in order
// (`holes`) and the live pages by their rank, as far as they move (`movers`).
struct CompactSpace {
  int32_t* moves;
  int32_t* holes;
  int32_t* movers;
};
__host__ __device__ inline int64_t holes_room(int num_blocks) {
  return (static_cast<int64_t>(num_blocks) + 63) / 64 * 64;
}
__host__ __device__ inline CompactSpace compact_space(void* ws, int num_blocks) {
  int32_t* w = static_cast<int32_t*>(ws);
  return CompactSpace{w, w + 64, w + 64 + holes_room(num_blocks)};
}

// Ranks the live pages; writes num_live, moved_to, ref_counts_out and the lists.
template <int CTAS>
__global__ void __launch_bounds__(kScanThreads, 1) compact_plan_kernel(const CompactArgs a) {
  __shared__ unsigned mine[kScanWarps], box[2][kScanCtas];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS > 1 ? cluster_rank() : 0u;
  if (CTAS > 1) cluster_arrive();                  // (this CTA has started)
  const CompactSpace ws = compact_space(a.workspace, a.num_blocks);
  const Part part = my_part<CTAS>(a.num_blocks, rank, warp);
  const unsigned n = count_part(a.ref_counts, a.num_blocks, 0, part.g0, part.g1, lane, live_bits);
  if (CTAS > 1) cluster_wait();
  const Before at = cluster_prefix<CTAS>(n, mine, box[0], warp, lane, rank);
  const int live = static_cast<int>(at.total);
  // ---- pages that stay, holes (rank: free pages below) and movers (live ones below)
  unsigned k0 = at.before, holes = 0;
  for (int g = part.g0; g < part.g1; g += 32) {
    const bool here = g + lane < part.g1;
    const int4 c = counts_at(a.ref_counts, min(g + lane, part.g1 - 1), a.num_blocks, 0);
    const unsigned bits = here ? live_bits(c) : 0u;
    unsigned k = k0 + warp_prefix(__popc(bits), lane);
    const int cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int page = 4 * (g + lane) + j;
      if (!here || page >= a.num_blocks) continue;
      const bool used = (bits >> j) & 1u;
      if (used && page >= live) {
        ws.movers[k] = page;
      } else {
        a.moved_to[page] = used ? page : -1;
        if (!used && page < live) {
          ws.holes[page - static_cast<int>(k)] = page;
          ++holes;
        } else if (a.ref_counts_out != a.ref_counts) {
          a.ref_counts_out[page] = cs[j];
        }
      }
      k += used;
    }
    k0 += warp_sum(__popc(bits));
  }
  holes = warp_sum(holes);
  __syncthreads();                                 // `mine` has been read by all
  const int moves = static_cast<int>(cluster_prefix<CTAS>(holes, mine, box[1], warp, lane, rank).total);
  if (CTAS == 1) __syncthreads();
  // (the barrier inside: the lists are whole) movers take the holes, in order
  for (int m = static_cast<int>(rank) * kScanThreads + threadIdx.x; m < moves;
       m += CTAS * kScanThreads) {
    const int src = ws.movers[live - moves + m], dst = ws.holes[m];
    const int count = a.ref_counts[src];
    a.moved_to[src] = dst;
    a.ref_counts_out[dst] = count;
    a.ref_counts_out[src] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    *a.num_live = live;
    *ws.moves = moves;
  }
}

constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads)
compact_move_kernel(const CompactArgs a, const PagePools p) {
  griddep_wait();
  const CompactSpace ws = compact_space(a.workspace, a.num_blocks);
  const int moves = *ws.moves, live = *a.num_live;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t chunks = p.page_bytes / 16;
  const int pieces = static_cast<int>((chunks + kPieceChunks - 1) / kPieceChunks);
  const int64_t units = static_cast<int64_t>(moves) * 2 * pieces;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kMoveThreads / 32) + warp; u < units;
       u += static_cast<int64_t>(gridDim.x) * (kMoveThreads / 32)) {
    const int m = static_cast<int>(u / (2 * pieces)), r = static_cast<int>(u - static_cast<int64_t>(m) * 2 * pieces);
    const int src = ws.movers[live - moves + m], dst = ws.holes[m];
    copy_piece(static_cast<uint4*>(r < pieces ? p.k_cache : p.v_cache), chunks, src, dst,
               r < pieces ? r : r - pieces, lane);
    if (r == 0 && p.k_scale != nullptr) copy_scales(p, src, dst, lane);
  }
  for (int row = blockIdx.x; row < a.num_rows; row += gridDim.x) {
    const int held = a.num_pages[row];
    const bool ok = held >= 0 && held <= a.mbs;
    if (!ok && threadIdx.x == 0) atomicOr(a.status, kStatusBadLen);
    const int32_t* t = a.block_tables + static_cast<int64_t>(row) * a.mbs;
    int32_t* o = a.tables_out + static_cast<int64_t>(row) * a.mbs;
    for (int j = threadIdx.x; j < a.mbs; j += kMoveThreads) {
      int id = t[j];
      if (ok && j < held) {
        const bool in = id >= 0 && id < a.num_blocks;
        if (in) id = a.moved_to[id];
        if (!in || id < 0) atomicOr(a.status, kStatusBadBlock);
      }
      o[j] = id;
    }
  }
}

}  // namespace

cudaError_t launch_alloc_pages(const TakeArgs& a, cudaStream_t s) { return launch_take<false>(a, s); }

cudaError_t launch_free_pages(int32_t* tables, int mbs, int32_t* num_pages, int num_rows,
                              const int32_t* rows, int items, int32_t* ref_counts, int num_blocks,
                              unsigned* status, cudaStream_t s) {
  return launch_after(free_kernel, dim3(static_cast<unsigned>(items)), kFreeThreads, 0, s, tables, mbs, num_pages,
                      num_rows, rows, ref_counts, num_blocks, status);
}

cudaError_t launch_fork_pages(const TakeArgs& a, int32_t* context_lens, const PagePools& p,
                              cudaStream_t s) {
  if (const cudaError_t e = launch_take<true>(a, s)) return e;
  return launch_after(fork_kernel, dim3(static_cast<unsigned>(a.items)), kForkThreads, 0, s, a, context_lens, p);
}

size_t compact_workspace_bytes(int num_blocks) {
  return static_cast<size_t>(64 + 2 * holes_room(num_blocks)) * 4;
}

cudaError_t launch_compact_pages(const CompactArgs& a, const PagePools& p, cudaStream_t s) {
  const bool one = a.num_blocks <= kOneCtaCompact;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(one ? 1 : kScanCtas);
  cfg.blockDim = dim3(kScanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0] = after_previous();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kScanCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = one ? 1 : 2;
  auto* plan = one ? compact_plan_kernel<1> : compact_plan_kernel<kScanCtas>;
  if (!one) {
    const cudaError_t e = cudaFuncSetAttribute(plan, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, plan, a)) return e;
  return launch_after(compact_move_kernel, dim3(static_cast<unsigned>(device_sm_count()) * 8), kMoveThreads, 0, s, a, p);
}

}  // namespace pa
