// prefill.cu -- attention of prompts over the paged cache, on the fifth-generation
// tensor cores (tcgen05.mma, accumulators in tensor memory).
//
//   out[t][hq] = sum_j softmax_j(scale q[t][hq] . K_j) V_j,  j up to t's own position
//
// The query rows of one (sequence, kv head) are its tokens times the group's heads:
// all of them read the same keys.  An item is 2 subtiles of floor(128 / group) tokens
// (up to 128 rows each) of one of them, and the 128-token tiles of keys that they see.
// Per tile and subtile:
//   S[128 rows][128 tokens]  = Q . K^T       (both K-major in shared memory)
//   O[128 rows][D]          += P . V         (P in tensor memory, in S's place)
//
// Roles of a CTA, one an SM:
//   warps 0-3, 4-7   the softmax of one subtile each, a thread a row, whose 128 scores it
//                    holds in registers; P goes back to tensor memory as 16-bit pairs;
//   warp 8           walks the CTA's pieces, copies Q and K (TMA), of E4M3 pools V too;
//   warps 9, 10      the products of one subtile each.  Its Q.K of the next tile follows its
//                    P.V in the same queue, so S needs no second buffer.  The subtiles
//                    take turns, tile by tile: the tensor cores work on one while the
//                    other's softmax runs;
//   warp 11          copies V; or, warps 11-15, of E4M3 pools: codes to f16 (exact)
//                    between two shared-memory rings.
//
// The softmax offset of a row is the maximum of an early tile's scores (the first of which
// it sees a number) and moves only when weights grow out of the products' range (kMaxSum):
// any standing offset gives the same softmax.  So once a warp's rows have theirs, most
// tiles need no maximum: their weights are made at once, their sum shows whether they may
// stand, and O is scaled in tensor memory hardly ever.  The weights of a tile's first half
// are announced alone, and its product begins.
//
// What bounds it: a product of 128 x 128 x 16 takes 64 cycles (measured, alone; 65 to 80
// with the softmax beside it), so a tile of both subtiles takes 2048 of the tensor
// cores, and 1200 of each exponential unit.  Measured on a GB300 (28/4 heads of 128,
// bf16): one prompt of 16384 tokens 1.19 ms, 1.62 PFLOP/s, 85 % of the measured bf16
// rate; with one loop for whole tiles and edges together it took 1.31 ms, with both
// subtiles' products in one queue unordered 1.95 (either in step, or one ahead until the
// ring had no place for its keys), with one thread issuing both subtiles' 3.8.
// Over E4M3 pools the codes' way through the converting warps is close behind: the next
// 450 tokens of two prompts over 115k cached ones take 1.13 ms when calls follow one another,
// 1.31 PFLOP/s, 69 %.  With a window of 4096 that prompt takes 0.57 ms, 1.48 PFLOP/s (its
// items are shorter), over an E4M3 pool 0.76.
//
// Page scales: K's multiply the scores of their 16 columns, V's the weights (relative
// to a power of two that follows the largest that the row has seen, so that P stays in
// f16's range and a page that the row does not see has no say).
//
// The batch's items, each as long as its tiles, are laid end to end and cut into one
// share a CTA; a cut within kSnap tiles of an item's border moves there.  An item that
// is cut all the same leaves its parts (O, maximum, sum) in the workspace, which a
// second launch joins in their order.
//
// A tile that some row of the subtile sees in part is an edge: masks are applied, V's
// rows without data (behind the context, pages with a bad id) are zeroed, and when a
// value of V is not finite, which a weight of 0 does not take away, the subtile's
// threads add up that tile's visible rows themselves.
//
// Every wait is bounded in time: a wait that gives up sets kStatusTimeout and a
// CTA-wide flag, at which every role leaves; copies and products in flight are waited
// for and tensor memory is freed first.
#include <climits>
#include <type_traits>

#include <cudaTypedefs.h>

#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "pa_tc.cuh"
#include "request_launch.h"

namespace pa {
namespace {

constexpr int kTile = 128;                 // tokens of a tile, rows of a subtile
constexpr int kPages = kTile / 16;
constexpr float kSlack = 8.f;              // log2 units
// Weights (and with a page scale up to twice the reference their products) are in f16's
// range while 64 of them add up to no more than this.
constexpr float kMaxSum = 32000.f;
constexpr int kSnap = 4;                   // tiles
// What an item costs besides its tiles (its queries, a pipeline that fills and drains, edges,
// the result), in tiles: what it adds to the shares.
constexpr int kItemCost = 8;
constexpr int kMaxSeqs = 512;              // sequences a launch sorts
constexpr int kDescs = 4;                  // pieces known ahead
constexpr int kMetas = 8;                  // tiles whose pages' validity and scales are kept
constexpr int kCopyWarp = 8, kMmaWarp = 9, kConvWarp = 11;
constexpr int kHeader = 16;                // ints a CTA's header in the workspace

struct Args {
  PrefillArgs a;
  CUtensorMap tm_q, tm_k, tm_v;
  float* ws_acc;                           // [grid][2 parts][2 subtiles][D / 4][128 rows][4]
  float2* ws_ml;                           // [grid][2][256]: offset (log2 units), sum
  int* ws_head;                            // [grid][kHeader]
  float sl2;                               // scale log2(e), not 0
  int sub;                                 // tokens of a subtile
  uint64_t wait_limit_ns;
};

// Header: what the CTA leaves in the workspace.
enum { kHasTail, kHasHead, kHeadEnds, kTailT0, kTailH, kTailTokens };

template <int D, bool FP8>
struct Cfg {
  static constexpr int kHalves = D / 64;                   // 128-byte columns of a row
  static constexpr int kSub = kTile * 128;                 // one half of a slot: 16 KB
  static constexpr int kSlot = kHalves * kSub;             // K or V of a tile, 16-bit
  static constexpr int kRaw = FP8 ? kTile * D : 0;         // its codes
  static constexpr int kRaws = FP8 ? 2 : 0;
  // Q of both subtiles, the ring, the codes: 224 KB at head_dim 128, 160 KB at 64
  static constexpr int kSlots = FP8 ? (D == 128 ? 4 : 6) : (D == 128 ? 5 : 8);
  // Three warpgroups of 168 registers a thread (65536 / 384), re-divided: 216 for a row's
  // 128 scores and their weights, 72 for the rest; 2 x 216 + 72 = 3 x 168.  With a fourth,
  // of converting warps: 128 at first, then 2 x 184 + 2 x 72 = 4 x 128.
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kSoftmaxRegs = FP8 ? 184 : 216, kOtherRegs = 72;
  static constexpr int kConvWarps = FP8 ? 5 : 1;
  static constexpr int kQ = 2 * kSlot;
  static constexpr int kBig = kQ + kSlots * kSlot + kRaws * kRaw;
};

struct Desc {                              // a piece, or the end (h < 0)
  int h, b, t0, n, L, i0, tokens;          // t0: q's first token; i0, tokens: of the sequence
  int k_lo, k_hi, g0;                      // tiles, and the number of the first in the CTA's stream
  int whole, part;                         // the whole item, or which part of the workspace
};

struct Meta {
  unsigned valid;                          // bit j: page j of the tile is seen and has a valid id
  float ks[kPages], vs[kPages], v_big;     // E4M3 pools: the scales, V's largest
};

enum : int {                               // mbarriers
  kFull = 0,
  kEmpty = kFull + 8,
  kRawFull = kEmpty + 8,
  kRawEmpty = kRawFull + 2,
  kQFull = kRawEmpty + 2,                  // by subtile, as those below
  kQEmpty = kQFull + 2,
  kQConv = kQEmpty + 2,
  kSFull = kQConv + 2,
  kPFull = kSFull + 2,
  kPHalf = kPFull + 2,                     // the second half of P
  kPVHalf = kPHalf + 2,                    // the product of a first half is done
  kODone = kPVHalf + 2,
  kVote = kODone + 2,
  kDFull = kVote + 2,
  kDEmpty = kDFull + kDescs,
  kFin = kDEmpty + kDescs,
  kBars = kFin + 2
};

struct Small {                             // shared memory behind the operands
  uint64_t bar[kBars];
  Desc desc[kDescs];
  Meta meta[kMetas];
  int tmem, dead, raw_end;
  int passed[2];                           // tiles that a subtile's products are issued for
  int skip[2];                             // the subtile's threads made this product themselves
  int flag[2][4];                          // by warp: a value of V is not finite
  int64_t lo, hi;                          // the CTA's share
  int b, h, j, off;                        // where it begins
};

struct Setup {                             // in the operands' place, before the copies start
  int n[kMaxSeqs], L[kMaxSeqs];
  int64_t before[kMaxSeqs + 1];            // units of the sequences before
};

__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* dead,
                                             uint64_t limit, unsigned* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
    if (global_ns() - t0 > limit) {
      *dead = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

// A value that all lanes hold, known to be one: what is computed from it, and loops that it
// bounds, need no vector registers (a product's descriptors are uniform registers, and
// bringing each there costs more than issuing the product).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0u;
}

// A box of a tensor map into shared memory (K and V of a prompt are read by many CTAs:
// no eviction hint).
__device__ __forceinline__ void box_g2s(uint32_t dst, const void* tmap, int x0, int x1, int x2,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x0), "r"(x1), "r"(x2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void page_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[tmem] . B[smem]: A's 16-bit pairs along K in the columns from tmem_a on.
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t db,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(db), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
constexpr uint32_t kBMajorN = 1u << 16;    // B MN-major (V: tokens along K, its rows along N)

// The pages `valid` of a tile (page j's id in lane j) into its slot, page j at rows 16j ..:
// one lane issues them all from uniform registers.
template <int HALVES, int SUB>
__device__ __forceinline__ void copy_pages(const void* tmap, int Hkv, int h, int id, unsigned valid,
                                           uint32_t slot, uint32_t full) {
  int page[kPages];
#pragma unroll
  for (int j = 0; j < kPages; ++j) page[j] = __shfl_sync(0xffffffffu, id, j) * Hkv + h;
  if (elect_one()) {
    mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(valid)) * (HALVES * 2048u));
#pragma unroll
    for (int j = 0; j < kPages; ++j)
      if ((valid >> j) & 1u)
#pragma unroll
        for (int x = 0; x < HALVES; ++x) box_g2s(slot + x * SUB + j * 2048, tmap, 64 * x, 0, page[j], full);
  }
  __syncwarp();
}
// The same for pages of codes, dense, page j at byte 16 D j.
template <int D>
__device__ __forceinline__ void copy_codes(const uint8_t* pool, int Hkv, int h, int id, unsigned valid,
                                           uint32_t to, uint32_t full) {
  int64_t page[kPages];
#pragma unroll
  for (int j = 0; j < kPages; ++j)
    page[j] = static_cast<int64_t>(__shfl_sync(0xffffffffu, id, j)) * Hkv + h;
  if (elect_one()) {
    mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(valid)) * (16u * D));
#pragma unroll
    for (int j = 0; j < kPages; ++j)
      if ((valid >> j) & 1u) page_g2s(to + j * 16 * D, pool + page[j] * (16 * D), 16 * D, full);
  }
  __syncwarp();
}

// Units of item j (its tiles; 1 when it sees none, for its zeros) of a sequence with n
// query tokens and L cached ones; *lo: the first tile.
__device__ __forceinline__ int item_units(int n, int L, int j, int sub, int window, int* lo) {
  const int i0 = j * 2 * sub, i1 = min(n, i0 + 2 * sub) - 1;
  const int last = L - n + i1, first = L - n + i0;
  *lo = 0;
  if (last < 0) return 1;
  if (window > 0) *lo = max(0, first - window + 1) / kTile;
  return last / kTile + 1 - *lo;
}
// The first page that a query of a piece's item sees: those before it are behind every
// window, and neither their ids nor their contents are looked at.
__device__ __forceinline__ int first_page(const Desc& d, int window) {
  return window > 0 ? max(0, d.L - d.n + d.i0 - window + 1) / 16 : 0;
}
// The tiles that subtile w of a piece sees, within the piece's.
__device__ __forceinline__ int2 sub_tiles(const Desc& d, int w, int sub, int window) {
  const int cnt = min(max(d.tokens - w * sub, 0), sub);
  const int first = d.L - d.n + d.i0 + w * sub, last = first + cnt - 1;
  if (cnt == 0 || last < 0) return make_int2(0, 0);
  const int lo = window > 0 ? max(0, first - window + 1) / kTile : 0;
  const int a = max(lo, d.k_lo), e = min(last / kTile + 1, d.k_hi);
  return a < e ? make_int2(a, e) : make_int2(0, 0);
}

// A warpgroup's registers a thread from here on (all its warps).
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float2 x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
  return unpair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
  return unpair(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
  return unpair(r);
}

template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
prefill_kernel(const __grid_constant__ Args ka) {
  using C = Cfg<D, FP8>;
  constexpr bool kMmaBf16 = BF16 && !FP8;  // the products' operand type
  // weights of f16 products are kept 2^6 larger, so that small ones stay in its normal
  // range (at an edge 2^(6 + kSlack) times a page scale up to twice the reference: below 2^16)
  constexpr float kLift = kMmaBf16 ? 0.f : 6.f;
  const PrefillArgs& a = ka.a;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  const uint32_t q_at = base, ring = base + C::kQ, raw = ring + C::kSlots * C::kSlot;
  Small& sm = *reinterpret_cast<Small*>(smem + C::kBig);
  const uint32_t bars = smem_u32(sm.bar);
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  volatile int* dead = &sm.dead;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uniform(tid >> 5);
  const int G = a.group, sub = ka.sub, cta = blockIdx.x;
  auto wait = [&](int b, int n) {          // the n-th completion (from 0) of barrier b
    return bounded_wait(bar(b), n & 1, dead, ka.wait_limit_ns, a.status);
  };
  auto wait_warp = [&](int b, int n) { return __all_sync(0xffffffffu, wait(b, n)); };

  griddep_wait();
  // ---- 1. the items' lengths, and this CTA's share of them
  {
    Setup& su = *reinterpret_cast<Setup*>(smem);
    for (int b = tid; b < a.B; b += C::kThreads) {
      const int s0 = a.starts[b], s1 = a.starts[b + 1], L = a.context_lens[b];
      const bool good = s0 >= 0 && s1 >= s0 && s1 <= a.T, fits = L >= 0 && L <= a.max_context_len;
      if (cta == 0 && (!good || (!fits && s1 > s0))) atomicOr(a.status, kStatusBadLen);
      su.n[b] = good ? s1 - s0 : 0;
      su.L[b] = fits ? L : 0;
    }
    if (tid == 0) {
      sm.dead = 0;
      sm.raw_end = INT_MAX;
      sm.passed[0] = sm.passed[1] = 0;
      su.before[0] = 0;
      for (int i = 0; i < kBars; ++i) {
        int n = 1;
        if (FP8 && i >= kFull && i < kFull + 8) n = C::kConvWarps;
        if (i >= kEmpty && i < kEmpty + 8) n = 2;
        if (i == kRawEmpty || i == kRawEmpty + 1) n = C::kConvWarps;
        if (i >= kQConv && i < kQConv + 2) n = 4;
        if (i >= kSFull && i < kSFull + 2) n = 2;
        if (i >= kPFull && i < kPHalf + 2) n = 4;
        if (i >= kVote && i < kVote + 2) n = 4;
        if (i >= kDEmpty && i < kDEmpty + kDescs) n = FP8 ? 2 + 8 : 3 + 8;
        mbar_init(bar(i), n);
      }
      mbar_init_fence();
    }
    __syncthreads();
    for (int b = warp; b < a.B; b += C::kThreads / 32) {
      const int n = su.n[b], L = su.L[b], items = (n + 2 * sub - 1) / (2 * sub);
      int64_t u = 0;
      int lo;
      for (int j = lane; j < items; j += 32)
        u += item_units(n, L, j, sub, a.window, &lo) + kItemCost;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
      if (lane == 0) su.before[b + 1] = u * a.Hkv;
    }
    __syncthreads();
    if (warp == 0) {                       // their prefix sums
      int64_t run = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        int64_t v = b0 + lane < a.B ? su.before[b0 + lane + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += t;
        }
        if (b0 + lane < a.B) su.before[b0 + lane + 1] = run + v;
        run += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
    const int64_t U = su.before[a.B];
    const int64_t NW = min(static_cast<int64_t>(gridDim.x), U);
    if (warp < 2) {                        // warp 0: where the share begins, warp 1: where it ends
      const int64_t k = min(static_cast<int64_t>(cta) + warp, NW);
      int64_t x = NW > 0 ? k * U / NW : 0;
      int b = 0, h = 0, j = 0, off = 0;
      if (x < U) {
        int l = 0, r = a.B;                // before[l] <= x < before[r]
        while (r - l > 1) {
          const int m = (l + r) >> 1;
          if (su.before[m] <= x) l = m;
          else r = m;
        }
        b = l;
        const int64_t per_head = (su.before[b + 1] - su.before[b]) / a.Hkv;
        int64_t rest = x - su.before[b];
        h = static_cast<int>(rest / per_head);
        rest -= h * per_head;
        const int n = su.n[b], L = su.L[b], items = (n + 2 * sub - 1) / (2 * sub);
        int units = 0;
        for (int j0 = 0; j0 < items; j0 += 32) {
          int lo;
          const int u = j0 + lane < items ? item_units(n, L, j0 + lane, sub, a.window, &lo) + kItemCost : 0;
          int64_t inc = u;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
          }
          const unsigned m = __ballot_sync(0xffffffffu, inc > rest);
          if (m != 0u) {
            const int at = __ffs(m) - 1;
            units = __shfl_sync(0xffffffffu, u, at);
            off = static_cast<int>(rest - (__shfl_sync(0xffffffffu, inc, at) - units));
            j = j0 + at;
            break;
          }
          rest -= __shfl_sync(0xffffffffu, inc, 31);
        }
        // a cut near an item's border moves there
        const int tile = off - kItemCost, left = units - off;
        if (tile < kSnap || left <= kSnap) {
          if (tile <= left) {
            x -= off;
            off = 0;
          } else {
            x += left;
            off = 0;
            const int all = (n + 2 * sub - 1) / (2 * sub);
            if (++j == all) {
              j = 0;
              if (++h == a.Hkv) {
                h = 0;
                do ++b;
                while (b < a.B && su.n[b] == 0);
              }
            }
          }
        } else {
          off = tile;
        }
      }
      if (lane == 0) {
        if (warp == 0) {
          sm.lo = static_cast<int64_t>(cta) < NW ? x : U;
          sm.b = b;
          sm.h = h;
          sm.j = j;
          sm.off = off;
        } else {
          sm.hi = x;
        }
      }
    }
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&sm.tmem), 512);
  fence_proxy_async_smem();                // the setup's place is the copies' now
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(sm.tmem));
  const uint32_t tmem_o = tmem + 2 * kTile;
  auto slot_at = [&](int i) { return ring + (i % C::kSlots) * C::kSlot; };   // i: K 2g, V 2g + 1

  if (warp >= 8) {
    regs_down<C::kOtherRegs>();
    if (warp == kCopyWarp) {
      // ================================================================ copies
      const int64_t hi = sm.hi;
      int b = sm.b, h = sm.h, j = sm.j, off = sm.off;
      int64_t pos = sm.lo - (off > 0 ? off + kItemCost : 0);   // the item's first unit
      int d = 0, g = 0, q_fills[2] = {0, 0}, raws = 0;
      int n = 0, L = 0, t0 = 0, loaded = -1;
      int head[6] = {0, 0, 0, 0, 0, 0};
      bool ok = true;
      // K (kv 0) or V (1) of tile g of kv head hh, whose page ids are the first lanes' `id`
      auto copy_tile = [&](int kv, int id, unsigned valid, int hh) {
        if constexpr (FP8) {
          if (raws >= C::kRaws && !wait_warp(kRawEmpty + raws % 2, raws / 2 - 1)) return false;
          const uint32_t full = bar(kRawFull + raws % 2), to = raw + (raws % 2) * C::kRaw;
          ++raws;
          copy_codes<D>(static_cast<const uint8_t*>(kv ? a.v_cache : a.k_cache), a.Hkv, hh, id, valid, to, full);
        } else {
          const int i = 2 * g + kv;
          if (i >= C::kSlots && !wait_warp(kEmpty + i % C::kSlots, i / C::kSlots - 1)) return false;
          if (g != a.drop_tile)
            copy_pages<C::kHalves, C::kSub>(&ka.tm_k, a.Hkv, hh, id, valid, slot_at(i),
                                            bar(kFull + i % C::kSlots));
        }
        return true;
      };
      // a piece's query rows
      auto copy_queries = [&](const Desc& x) {
        for (int w = 0; w < 2; ++w) {
          const int2 r = sub_tiles(x, w, sub, a.window);
          if (r.x == r.y) continue;
          if (q_fills[w] > 0 && !wait_warp(kQEmpty + w, q_fills[w] - 1)) return false;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(kQFull + w), static_cast<uint32_t>(C::kHalves * 128 * sub * G));
#pragma unroll
            for (int y = 0; y < C::kHalves; ++y)
              box_g2s(q_at + w * C::kSlot + y * C::kSub, &ka.tm_q, 64 * y, x.h * G, x.t0 + w * sub,
                      bar(kQFull + w));
          }
          ++q_fills[w];
          __syncwarp();
        }
        return true;
      };
      while (ok && pos < hi) {
        if (b != loaded) {                   // (bad starts and lengths were reported above)
          const int s0 = a.starts[b], s1 = a.starts[b + 1];
          n = s0 >= 0 && s1 >= s0 && s1 <= a.T ? s1 - s0 : 0;
          L = a.context_lens[b];
          L = L >= 0 && L <= a.max_context_len ? L : 0;
          t0 = s0;
          loaded = b;
        }
        const int items = (n + 2 * sub - 1) / (2 * sub);
        if (items == 0) {
          ++b;
          continue;
        }
        int k0;
        const int u = item_units(n, L, j, sub, a.window, &k0);
        const int64_t room = hi - pos - kItemCost;   // tiles of it before the share's end
        const int take = (room < u ? static_cast<int>(room) : u) - off;
        Desc x;
        x.h = h;
        x.b = b;
        x.n = n;
        x.L = L;
        x.i0 = j * 2 * sub;
        x.tokens = min(n - x.i0, 2 * sub);
        x.t0 = t0 + x.i0;
        const bool sees = L - n + x.i0 + x.tokens - 1 >= 0;
        x.k_lo = sees ? k0 + off : 0;
        x.k_hi = sees ? k0 + off + take : 0;
        x.g0 = g;
        x.whole = take == u;
        x.part = off > 0 ? 0 : 1;
        if (!x.whole) {
          if (off > 0) {
            head[kHasHead] = 1;
            head[kHeadEnds] = off + take == u;
          } else {
            head[kHasTail] = 1;
            head[kTailT0] = x.t0;
            head[kTailH] = h;
            head[kTailTokens] = x.tokens;
          }
        }
        if (d >= kDescs && !wait_warp(kDEmpty + d % kDescs, d / kDescs - 1)) break;
        if (lane == 0) {
          sm.desc[d % kDescs] = x;
          mbar_arrive(bar(kDFull + d % kDescs));
        }
        ++d;
        __syncwarp();
        // ---- its tiles: four tiles' page ids at a time, the next four on their way, and of
        // E4M3 pools the next tile's scales
        const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.mbs;
        const int p_lo = first_page(x, a.window), last_page = (L + 15) / 16 - 1;
        auto ids_at = [&](int t) {
          const int p = t * kPages + lane;
          return p >= p_lo && p <= last_page && t + (lane >> 3) < x.k_hi ? table[p] : -1;
        };
        int ids = ids_at(x.k_lo), ids_next = ids_at(x.k_lo + 4), id = -1;
        float sk = 0.f, sv = 0.f;
        bool valid = false;
        auto fetch = [&](int t) {
          const int in4 = (t - x.k_lo) & 3;
          if (in4 == 0 && t > x.k_lo) {
            ids = ids_next;
            ids_next = ids_at(t + 4);
          }
          id = __shfl_sync(0xffffffffu, ids, in4 * 8 + (lane & 7));
          const int p = t * kPages + lane;
          const bool mine = t < x.k_hi && lane < kPages && p >= p_lo && p <= last_page;
          valid = mine && id >= 0 && id < a.num_blocks;
          if (mine && !valid) atomicOr(a.status, kStatusBadBlock);
          if constexpr (FP8) {
            const int64_t page = static_cast<int64_t>(valid ? id : 0) * a.Hkv + h;
            sk = valid ? a.k_scale[page] : 0.f;
            sv = valid ? a.v_scale[page] : 0.f;
          }
        };
        fetch(x.k_lo);
        for (int t = x.k_lo; ok && t < x.k_hi; ++t, ++g) {
          const int id_now = id;
          const unsigned m = __ballot_sync(0xffffffffu, valid);
          Meta& mt = sm.meta[g % kMetas];
          if (lane == 0) mt.valid = m;
          if constexpr (FP8) {
            float top = sv;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane < kPages) {
              mt.ks[lane] = sk;
              mt.vs[lane] = sv;
              mt.v_big = top;
            }
          }
          __syncwarp();
          fetch(t + 1);
          ok = copy_tile(0, id_now, m, h) && (t > x.k_lo || copy_queries(x)) &&
               (!FP8 || copy_tile(1, id_now, m, h));
        }
        // ---- the next item
        pos += u + kItemCost;
        off = 0;
        if (++j == items) {
          j = 0;
          if (++h == a.Hkv) {
            h = 0;
            ++b;
          }
        }
      }
      if (ok && (d < kDescs || wait_warp(kDEmpty + d % kDescs, d / kDescs - 1))) {
        if (lane == 0) {
          sm.desc[d % kDescs].h = -1;
          mbar_arrive(bar(kDFull + d % kDescs));
        }
      }
      if (FP8 && lane == 0) {                // the converting warps' end
        *reinterpret_cast<volatile int*>(&sm.raw_end) = raws;
        __threadfence_block();
      }
      if (lane == 0)
        for (int i = 0; i < 6; ++i) ka.ws_head[cta * kHeader + i] = head[i];
      // no copy outlives the CTA
      if (lane == 0) {
        const uint64_t since = global_ns();
        const uint64_t limit = ka.wait_limit_ns > kWaitLimitNs ? ka.wait_limit_ns : kWaitLimitNs;
        auto settle = [&](int bb, int fills) {
          while (fills > 0 && !mbar_try_wait(bar(bb), (fills - 1) & 1) && global_ns() - since < limit) {
          }
        };
        for (int w = 0; w < 2; ++w) settle(kQFull + w, q_fills[w]);
        if (FP8) {
          for (int r = 0; r < 2; ++r) settle(kRawFull + r, (raws - r + 1) / 2);
        } else {
          for (int i = (max(2 * g - C::kSlots, 0) + 1) / 2 * 2; i < 2 * g; i += 2)   // each place's last
            settle(kFull + i % C::kSlots, i / C::kSlots + 1);
        }
      }
      __syncwarp();
    } else if (warp < kConvWarp) {
      // ================================================================ products
      // One warp a subtile: Q.K of a tile, then, once its weights are there, P.V.
      constexpr uint32_t kIdQK = umma_idesc_f16<kMmaBf16>(kTile, kTile, false);
      constexpr uint32_t kIdPV = umma_idesc_f16<kMmaBf16>(kTile, D, false) | kBMajorN;
      const int w = warp - kMmaWarp;
      const uint32_t ts = tmem + w * kTile, to = tmem_o + w * D;
      const uint64_t dq = umma_desc_sw128(q_at + w * C::kSlot, 16, 1024);
      const uint64_t dk0 = umma_desc_sw128(ring, 16, 1024);
      const uint64_t dv0 = umma_desc_sw128(ring, C::kSub, 1024);
      int p_n = 0, q_n = 0;
      // the next K's and V's place in the ring (K 0, V 1, K 2, ..) and their fills' parity
      int ks = 0, kp = 0, vs = 1, vp = 0;
      auto step2 = [&](int& slot, int& parity) {
        slot += 2;
        if (slot >= C::kSlots) {
          slot -= C::kSlots;
          parity ^= 1;
        }
      };
      auto full = [&](int slot, int parity) { return wait_warp(kFull + slot, parity); };
      bool issued = false, ok = true;
      // The subtiles take turns, tile by tile: left alone they either run in step, and the tensor
      // cores wait while both softmaxes run, or one runs ahead until the ring has no place
      // for its keys.
      int g = 0;                             // the tile in the CTA's stream
      volatile int* mine = &sm.passed[w];
      volatile int* other = &sm.passed[w ^ 1];
      auto my_turn = [&]() {                 // tile g is the first subtile's first
        uint64_t t0 = 0;
        for (unsigned i = 1; *other < g + w; ++i) {
          if (i % 256 != 0) continue;
          if (*dead) return false;
          const uint64_t now = global_ns();
          if (t0 == 0) {
            t0 = now;
          } else if (now - t0 > ka.wait_limit_ns) {
            *dead = 1;
            atomicOr(a.status, kStatusTimeout);
            return false;
          }
        }
        return true;
      };
      auto passed = [&]() {
        ++g;
        __syncwarp();
        if (lane == 0) *mine = g;
      };
      auto scores = [&](bool last) {         // Q.K of the next tile, whose K has landed
        if (elect_one()) {
          mbar_arrive(bar(kSFull + w));      // (orders the tile's meta before the softmax's reads)
          const uint64_t dk = dk0 + static_cast<uint64_t>(ks * (C::kSlot >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t o = static_cast<uint64_t>(((k >> 2) * C::kSub + (k & 3) * 32) >> 4);
            umma_f16(ts, dq + o, dk + o, kIdQK, k > 0);
          }
          umma_commit(bar(kSFull + w));
          umma_commit(bar(kEmpty + ks));
          if (last) umma_commit(bar(kQEmpty + w));
        }
        __syncwarp();
        issued = true;
        step2(ks, kp);
      };
      auto pass = [&](int tiles) {           // tiles that the other subtile alone sees
        for (int i = 0; i < tiles && ok; ++i) {
          ok = full(ks, kp) && full(vs, vp);
          if (ok && lane == 0) {
            mbar_arrive(bar(kEmpty + ks));
            mbar_arrive(bar(kEmpty + vs));
          }
          step2(ks, kp);
          step2(vs, vp);
          passed();
        }
      };
      for (int d = 0; ok; ++d) {
        if (!wait_warp(kDFull + d % kDescs, d / kDescs)) break;
        const Desc& x = sm.desc[d % kDescs];
        if (uniform(x.h) < 0) break;
        int2 r = sub_tiles(x, w, sub, a.window);
        r.x = uniform(r.x);
        r.y = uniform(r.y);
        const int k_lo = uniform(x.k_lo), k_hi = uniform(x.k_hi);
        const bool some = r.x < r.y;
        const int behind = some ? k_hi - r.y : 0;
        pass(some ? r.x - k_lo : k_hi - k_lo);
        if (ok && some) {
          ok = full(ks, kp) && wait_warp((FP8 && BF16 ? kQConv : kQFull) + w, q_n++);
          if (ok) {
            tc_fence_after();
            scores(r.x + 1 == r.y);
          }
        }
        for (int t = r.x; ok && t < r.y; ++t, ++p_n) {
          const bool more = t + 1 < r.y;
          ok = full(vs, vp) && (!more || full(ks, kp)) && wait_warp(kPFull + w, p_n) &&
               __all_sync(0xffffffffu, my_turn());
          if (!ok) break;
          tc_fence_after();
          const bool skip = uniform(*reinterpret_cast<volatile int*>(&sm.skip[w])) != 0;
          const uint64_t dv = dv0 + static_cast<uint64_t>(vs * (C::kSlot >> 4));
          if (skip) {
            if (lane == 0) mbar_arrive(bar(kPVHalf + w));
          } else if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              umma_f16_ts(to, ts + 8 * k, dv + static_cast<uint64_t>(k * (2048 >> 4)), kIdPV,
                          t > r.x || k > 0);
            umma_commit(bar(kPVHalf + w));
          }
          __syncwarp();
          ok = wait_warp(kPHalf + w, p_n);   // the weights of the second half of the tile
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (!skip) {
#pragma unroll
              for (int k = kTile / 32; k < kTile / 16; ++k)
                umma_f16_ts(to, ts + 8 * k, dv + static_cast<uint64_t>(k * (2048 >> 4)), kIdPV, true);
            }
            umma_commit(bar(kEmpty + vs));
            if (!more) umma_commit(bar(kODone + w));
          }
          __syncwarp();
          step2(vs, vp);
          if (more) scores(t + 2 == r.y);
          passed();
        }
        pass(behind);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kDEmpty + d % kDescs));
      }
      // no product outlives the CTA
      if (issued) {
        if (elect_one()) umma_commit(bar(kFin + w));
        __syncwarp();
        const uint64_t since = global_ns();
        const uint64_t limit = ka.wait_limit_ns > kWaitLimitNs ? ka.wait_limit_ns : kWaitLimitNs;
        while (!mbar_try_wait(bar(kFin + w), 0) && global_ns() - since < limit) {
        }
      }
      __syncwarp();
    } else if (!FP8) {
      // ================================================================ V's copies
      int g = 0;
      bool ok = true;
      for (int d = 0; ok; ++d) {
        if (!wait_warp(kDFull + d % kDescs, d / kDescs)) break;
        const Desc& x = sm.desc[d % kDescs];
        const int h = uniform(x.h);
        if (h < 0) break;
        const int k_lo = uniform(x.k_lo), k_hi = uniform(x.k_hi);
        const int32_t* table = a.block_tables + static_cast<int64_t>(x.b) * a.mbs;
        const int p_lo = first_page(x, a.window), last_page = (x.L + 15) / 16 - 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kDEmpty + d % kDescs));
        auto ids_at = [&](int t) {
          const int p = t * kPages + lane;
          return p >= p_lo && p <= last_page && t + (lane >> 3) < k_hi ? table[p] : -1;
        };
        int ids = ids_at(k_lo), ids_next = ids_at(k_lo + 4);
        for (int t = k_lo; ok && t < k_hi; ++t, ++g) {
          const int in4 = (t - k_lo) & 3;
          if (in4 == 0 && t > k_lo) {
            ids = ids_next;
            ids_next = ids_at(t + 4);
          }
          const int id = __shfl_sync(0xffffffffu, ids, in4 * 8 + (lane & 7));
          const unsigned m = __ballot_sync(0xffffffffu, lane < kPages && id >= 0 && id < a.num_blocks);
          const int i = 2 * g + 1;
          ok = i < C::kSlots || wait_warp(kEmpty + i % C::kSlots, i / C::kSlots - 1);
          if (ok)
            copy_pages<C::kHalves, C::kSub>(&ka.tm_v, a.Hkv, h, id, m, slot_at(i), bar(kFull + i % C::kSlots));
        }
      }
      if (lane == 0) {                       // no copy outlives the CTA
        const uint64_t since = global_ns();
        const uint64_t limit = ka.wait_limit_ns > kWaitLimitNs ? ka.wait_limit_ns : kWaitLimitNs;
        if (!ok) --g;                        // (the last one was not made)
        for (int i = max(2 * g - C::kSlots, 0) | 1; i < 2 * g; i += 2) {
          while (!mbar_try_wait(bar(kFull + i % C::kSlots), (i / C::kSlots) & 1) && global_ns() - since < limit) {
          }
        }
      }
      __syncwarp();
    } else {
      // ================================================================ codes to f16
      const int ct = tid - kConvWarp * 32;
      for (int f = 0;; ++f) {                // the next fill, or the end
        bool got = mbar_try_wait(bar(kRawFull + f % 2), (f / 2) & 1), end = false;
        if (!got) {
          const uint64_t since = global_ns();
          while (!got && !end) {
            got = mbar_try_wait(bar(kRawFull + f % 2), (f / 2) & 1);
            if (!got) {
              end = f >= *reinterpret_cast<volatile int*>(&sm.raw_end) || *dead;
              if (!end && global_ns() - since > ka.wait_limit_ns) {
                *dead = 1;
                atomicOr(a.status, kStatusTimeout);
                end = true;
              }
            }
          }
        }
        if (!__all_sync(0xffffffffu, got)) break;
        if (f >= C::kSlots && !wait_warp(kEmpty + f % C::kSlots, f / C::kSlots - 1)) break;
        const uint32_t src = raw + (f % 2) * C::kRaw, dst = slot_at(f);
        constexpr int kChunks = D / 16;      // 16 codes each, of a row
        constexpr int kAll = kTile * kChunks, kEach = (kAll + C::kConvWarps * 32 - 1) / (C::kConvWarps * 32);
        // Into registers, all loads in flight at once; then their place is free for the next
        // copy.  (Released once they were written out, two places kept 32 KB in flight at
        // most half of the time: 1.39 ms instead of 1.07, single calls, for two prompts' next
        // 512 tokens over 100k cached ones.)
        uint4 all[kEach];
#pragma unroll
        for (int n = 0; n < kEach; ++n) all[n] = lds128(src + 16 * min(ct + n * C::kConvWarps * 32, kAll - 1));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kRawEmpty + f % 2));
#pragma unroll
        for (int n = 0; n < kEach; ++n) {
          const int i = ct + n * C::kConvWarps * 32;
          if (i >= kAll) break;
          const uint4 codes = all[n];
          const int row = i / kChunks, c = i % kChunks, half = c / 4, p = (c % 4) * 2;
          uint4 lo, hi;
          lo.x = e4m3x2_to_f16x2(codes.x & 0xffffu);
          lo.y = e4m3x2_to_f16x2(codes.x >> 16);
          lo.z = e4m3x2_to_f16x2(codes.y & 0xffffu);
          lo.w = e4m3x2_to_f16x2(codes.y >> 16);
          hi.x = e4m3x2_to_f16x2(codes.z & 0xffffu);
          hi.y = e4m3x2_to_f16x2(codes.z >> 16);
          hi.z = e4m3x2_to_f16x2(codes.w & 0xffffu);
          hi.w = e4m3x2_to_f16x2(codes.w >> 16);
          const uint32_t at = dst + half * C::kSub + row * 128;
          // (the other half's lanes store their two chunks in the other order: no bank twice)
          const int p0 = half ? p + 1 : p, p1 = half ? p : p + 1;
          sts128(at + ((p0 ^ (row & 7)) << 4), half ? hi : lo);
          sts128(at + ((p1 ^ (row & 7)) << 4), half ? lo : hi);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kFull + f % C::kSlots));
      }
    }
  } else {
    // ================================================================ softmax
    regs_up<C::kSoftmaxRegs>();
    const int w = warp >> 2, wq = warp & 3, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t ts = tmem + lanes + w * kTile, to = tmem_o + lanes + w * D;
    const int tok = r / G, hd = r - tok * G;
    int s_n = 0, o_n = 0, q_n = 0, votes = 0;   // completions seen
    bool ok = true;
    for (int d = 0; ok; ++d) {
      if (!wait_warp(kDFull + d % kDescs, d / kDescs)) break;
      const Desc x = sm.desc[d % kDescs];
      if (x.h < 0) break;
      const int2 tiles = sub_tiles(x, w, sub, a.window);
      const int cnt = min(max(x.tokens - w * sub, 0), sub);
      const int first = x.L - x.n + x.i0 + w * sub, last = first + cnt - 1;
      const int pos = first + tok;         // this row's
      // rows behind the subtile's hold whatever was there: they ask for nothing
      const bool row_live = r < cnt * G;
      float off = -INFINITY, l = 0.f, ref = FP8 ? 0.f : 1.f;
      [[maybe_unused]] float low_ref = 0.f;   // the lowest reference of the warp's rows
      float sl2 = ka.sl2;
      if (FP8 && BF16 && tiles.x < tiles.y) {
        // bf16 rows to f16, scaled by a power of two so that the row's largest element lies
        // in [2^14, 2^15)
        if (!wait_warp(kQFull + w, q_n)) break;
        const uint32_t row = q_at + w * C::kSlot + r * 128;
        float big = 0.f;
#pragma unroll 4
        for (int c = 0; c < 8 * C::kHalves; ++c) {
          const uint4 x4 = lds128(row + (c >> 3) * C::kSub + (((c ^ r) & 7) << 4));
          for (const uint32_t u : {x4.x, x4.y, x4.z, x4.w})
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(u << 16)), fabsf(__uint_as_float(u & 0xffff0000u))));
        }
        const int e = big > 0.f && big < INFINITY ? 14 - ilogbf(big) : 0;
        // 2^e in two factors: e reaches 147
        const float f0 = __uint_as_float(static_cast<uint32_t>(127 + e / 2) << 23);
        const float f1 = __uint_as_float(static_cast<uint32_t>(127 + e - e / 2) << 23);
#pragma unroll 4
        for (int c = 0; c < 8 * C::kHalves; ++c) {
          const uint32_t chunk = row + (c >> 3) * C::kSub + (((c ^ r) & 7) << 4);
          uint4 x4 = lds128(chunk);
          for (uint32_t* u : {&x4.x, &x4.y, &x4.z, &x4.w})
            *u = pack2<false>(__uint_as_float(*u << 16) * f0 * f1, __uint_as_float(*u & 0xffff0000u) * f0 * f1);
          sts128(chunk, x4);
        }
        sl2 = copysignf(fmaxf(fabsf(sl2) / f0 / f1, 1e-37f), sl2);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQConv + w));
        ++q_n;
      }
      // tiles that all rows see whole, while their pages are valid: [full_lo, full_hi)
      const int full_hi = (first + 1) / kTile;
      const int full_lo = a.window > 0 ? (max(last - a.window + 1, 0) + kTile - 1) / kTile : 0;
      // what a score of page c is multiplied with (log2 units)
      auto factor = [&](const Meta& mt, int c) {
        if constexpr (FP8) return copysignf(fmaxf(fabsf(sl2) * mt.ks[c], 1e-37f), sl2);
        else return sl2;
      };
      // weights of N scores from page `page` on at the standing offset, as 16-bit pairs; their sum
      auto weigh = [&](auto n, const Meta& mt, const float* s, float* out, int page, unsigned bits) {
        constexpr int N = decltype(n)::value;
        const float sub_off = (off == -INFINITY ? 0.f : off) - kLift;
        [[maybe_unused]] const float inv_ref = FP8 ? 1.f / ref : 1.f;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const float k = factor(mt, page + j / 16);
          float2 e = fma2(make_float2(s[j], s[j + 1]), make_float2(k, k), make_float2(-sub_off, -sub_off));
          e.x = fast_exp2(e.x);
          e.y = fast_exp2(e.y);
          if (N == 32) {                   // (the exact form: what is masked weighs nothing)
            e.x = (bits >> j) & 1u ? e.x : 0.f;
            e.y = (bits >> (j + 1)) & 1u ? e.y : 0.f;
          }
          sum[(j / 2) & 1] = add2(sum[(j / 2) & 1], e);
          if constexpr (FP8) {
            float u = mt.vs[page + j / 16] * inv_ref;
            if (N == 32 && ((bits >> (j & 16)) & 0xffffu) == 0u) u = 0.f;   // (0 weights, whatever the scale)
            e = mul2(e, make_float2(u, u));
          }
          out[j / 2] = __uint_as_float(pack2<kMmaBf16>(e.x, e.y));
        }
        const float2 both = add2(sum[0], sum[1]);
        return both.x + both.y;
      };
      auto announce = [&](int b) {         // this warp's part of P is written
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b + w));
      };
      for (int t = tiles.x; ok && t < tiles.y; ++t) {
        // ---- a run of whole tiles: a loop of its own, as short as it can be.  The weights at
        // the standing offset do unless they have grown out of the products' range, which
        // their sum shows (a NaN too); then the exact form below takes over, from that half on.
        // (A tile of which a row sees a number gives it its offset.  Its first one need not be the
        // subtile's: a window may begin behind that, its pages may be invalid.)
        int from = 0;
        bool more = t > tiles.x && !__any_sync(0xffffffffu, row_live && off == -INFINITY);
        while (more) {
          if (!wait_warp(kSFull + w, s_n)) {
            ok = false;
            break;
          }
          const Meta& mt = sm.meta[(x.g0 + t - x.k_lo) % kMetas];
          if (t < full_lo || t >= full_hi || mt.valid != 0xffu || (FP8 && mt.v_big > 2.f * low_ref)) break;
          tc_fence_after();
          float v[kTile], p[32];
          tmem_ld<32>(ts, *reinterpret_cast<float (*)[32]>(v));
          tmem_ld<32>(ts + 32, *reinterpret_cast<float (*)[32]>(v + 32));
          tmem_wait_ld();
          tmem_ld<32>(ts + 64, *reinterpret_cast<float (*)[32]>(v + 64));
          tmem_ld<32>(ts + 96, *reinterpret_cast<float (*)[32]>(v + 96));
          float sum = weigh(std::integral_constant<int, 64>(), mt, v, p, 0, 0u);
          if (__any_sync(0xffffffffu, row_live && !(sum <= kMaxSum))) {
            tmem_wait_ld();
            break;
          }
          l += sum;
          tmem_st<32>(ts, p);
          if (wq == 0 && lane == 0) sm.skip[w] = 0;
          announce(kPFull);                // the product of the first half may begin
          tmem_wait_ld();
          sum = weigh(std::integral_constant<int, 64>(), mt, v + 64, p, 4, 0u);
          if (__any_sync(0xffffffffu, row_live && !(sum <= kMaxSum))) {
            from = 1;
            break;
          }
          l += sum;
          tmem_st<32>(ts + 32, p);
          announce(kPHalf);
          ++s_n;
          more = ++t < tiles.y;
        }
        if (!ok || t == tiles.y) break;
        // ---- the exact form: the first tile, tiles that some row sees in part, and where the
        // offset or the reference of V's scales has to move
        if (!wait_warp(kSFull + w, s_n)) {
          ok = false;
          break;
        }
        ++s_n;
        tc_fence_after();
        const int g = x.g0 + t - x.k_lo, p0 = t * kTile;
        const Meta& mt = sm.meta[g % kMetas];
        const unsigned valid = mt.valid;
        const bool start = t == tiles.x, edge = t < full_lo || t >= full_hi || valid != 0xffu;
        // columns [jl, jh) of the tile are this row's, those of valid pages
        const int jh = pos + 1 - p0, jl = a.window > 0 ? max(max(pos, 0) - a.window + 1 - p0, 0) : 0;
        auto below = [](int j) { return j <= 0 ? 0u : j >= 32 ? ~0u : (1u << j) - 1u; };
        auto word = [&](int c) {           // of columns 32c .. 32c + 31
          const unsigned pages = ((valid >> (2 * c)) & 1u ? 0xffffu : 0u) |
                                 ((valid >> (2 * c + 1)) & 1u ? 0xffff0000u : 0u);
          return edge ? below(jh - 32 * c) & ~below(jl - 32 * c) & pages : ~0u;
        };
        float v_big = 0.f;                 // the largest scale of V's pages that this row sees
        if constexpr (FP8) {
          if (edge) {
#pragma unroll 1
            for (int c = 0; c < kPages; ++c)
              if ((word(c / 2) >> (c % 2 * 16)) & 0xffffu) v_big = fmaxf(v_big, mt.vs[c]);
          } else {
            v_big = mt.v_big;
          }
        }
        if (from == 1 && !wait_warp(kPVHalf + w, s_n - 1)) {   // (O changes below)
          ok = false;
          break;
        }
        tc_fence_after();
        {
          float m = -INFINITY;
#pragma unroll 1
          for (int c = 2 * from; c < 4; ++c) {
            float s[32];
            tmem_ld<32>(ts + 32 * c, s);
            tmem_wait_ld();
            const unsigned bits = word(c);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float y = s[j] * factor(mt, 2 * c + j / 16);
              m = fmaxf(m, (bits >> j) & 1u ? y : -INFINITY);
            }
          }
          // A new offset for the rows that move, and a reference of V's scales that does for
          // this tile's; O (when it holds something) and the sum are scaled down to them.
          const bool move = start || (row_live && m > off + kSlack);
          const bool refer = FP8 && (v_big > 2.f * ref || !(ref > 0.f));
          if (__any_sync(0xffffffffu, move || refer)) {
            float f = 1.f;
            if (move) {
              const float to_off = fmaxf(off, m);
              f = off == to_off ? 1.f : fast_exp2(off - to_off);
              off = to_off;
              l *= f;
            }
            if (refer) {                   // a power of two at or above the largest scale so far
              const float top = __uint_as_float((__float_as_uint(fmaxf(v_big, 1e-30f)) + 0x7fffffu) & 0x7f800000u);
              f *= ref > 0.f ? ref / top : 1.f;
              ref = top;
            }
            if constexpr (FP8)
              low_ref = __uint_as_float(__reduce_min_sync(0xffffffffu, row_live ? __float_as_uint(ref) : 0x7f800000u));
            if (!start) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                float o[16];
                tmem_ld<16>(to + 16 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_st<16>(to + 16 * c, o);
              }
            }
          }
#pragma unroll 1
          for (int c = 2 * from; c < 4; ++c) {
            float s[32], y[16];
            tmem_ld<32>(ts + 32 * c, s);
            tmem_wait_ld();
            l += weigh(std::integral_constant<int, 32>(), mt, s, y, 2 * c, word(c));
            tmem_st<16>(ts + 16 * c, y);   // (over scores that have been read)
          }
          tmem_wait_st();
        }
        if (edge) {
          // token r of the tile: no data, a row of zeros; else is every value finite?
          const int i = 2 * g + 1;
          if (!wait_warp(kFull + i % C::kSlots, i / C::kSlots)) {
            ok = false;
            break;
          }
          const bool data = p0 + r < x.L && ((valid >> (r >> 4)) & 1u);
          const uint32_t vrow = slot_at(i) + r * 128;
          bool odd = false;
#pragma unroll 4
          for (int c = 0; c < 8 * C::kHalves; ++c) {
            // (neighbouring rows begin at different chunks: no bank twice)
            const uint32_t at = vrow + (c >> 3) * C::kSub + (((c ^ r) & 7) << 4);
            const uint4 x4 = lds128(at);
            // a 16-bit value is not finite when its exponent's bits are all set: one more in
            // the lowest of them carries into the sign
            constexpr uint32_t kExp = kMmaBf16 ? 0x7f807f80u : 0x7c007c00u;
            constexpr uint32_t kOne = kMmaBf16 ? 0x00800080u : 0x04000400u;
            odd |= ((((x4.x & kExp) + kOne) | ((x4.y & kExp) + kOne) | ((x4.z & kExp) + kOne) |
                     ((x4.w & kExp) + kOne)) & 0x80008000u) != 0u;
            if (!data && (x4.x | x4.y | x4.z | x4.w) != 0u) sts128(at, make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
          const bool any = __any_sync(0xffffffffu, odd && data);
          if (lane == 0) {
            sm.flag[w][wq] = any;
            mbar_arrive(bar(kVote + w));
          }
          if (!wait_warp(kVote + w, votes++)) {
            ok = false;
            break;
          }
          const volatile int* fl = sm.flag[w];
          const bool self = fl[0] | fl[1] | fl[2] | fl[3];
          if (self) {
            // this tile's product by the rows' own threads, over the tokens that they see
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 8) {
              float o[8];
              if (start) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
              } else {
                tmem_ld<8>(to + c0, o);
              }
              const uint32_t col = slot_at(i) + (c0 / 64) * C::kSub;
#pragma unroll 1
              for (int j0 = 0; j0 < kTile; j0 += 8) {
                const unsigned seen = word(j0 / 32) >> (j0 & 31);
                float p[4];
                tmem_ld<4>(ts + j0 / 2, p);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const int at = j0 + j;
                  const uint32_t two = __float_as_uint(p[j / 2]);
                  const uint32_t one = j & 1 ? two >> 16 : two & 0xffffu;
                  const float pf = kMmaBf16 ? __uint_as_float(one << 16)
                                            : __half2float(__ushort_as_half(static_cast<unsigned short>(one)));
                  const uint4 v = lds128(col + at * 128 + ((((c0 % 64) / 8) ^ (at & 7)) << 4));
                  if (!((seen >> j) & 1u)) continue;
                  const uint32_t us[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    float2 f;
                    if constexpr (kMmaBf16)
                      f = make_float2(__uint_as_float(us[k] << 16), __uint_as_float(us[k] & 0xffff0000u));
                    else
                      f = __half22float2(*reinterpret_cast<const __half2*>(&us[k]));
                    o[2 * k] = fmaf(pf, f.x, o[2 * k]);
                    o[2 * k + 1] = fmaf(pf, f.y, o[2 * k + 1]);
                  }
                }
              }
              __syncwarp();
              tmem_st<8>(to + c0, o);
            }
            tmem_wait_st();
          }
          if (wq == 0 && lane == 0) sm.skip[w] = self;
        } else if (from == 0 && wq == 0 && lane == 0) {
          sm.skip[w] = 0;
        }
        if (from == 0) announce(kPFull);
        announce(kPHalf);
      }
      if (!ok) break;
      // ---- the piece's result
      const bool some = tiles.x < tiles.y;
      if (some) {
        if (!wait_warp(kODone + w, o_n)) break;
        ++o_n;
        tc_fence_after();
      }
      const bool any = some && l != 0.f;   // (a NaN is something)
      const float f = !any ? 0.f : x.whole ? ref / l : ref;
      uint16_t* out = static_cast<uint16_t*>(a.out) +
                      ((static_cast<int64_t>(x.t0) + w * sub + tok) * a.Hq + x.h * G + hd) * D;
      const int64_t at = (static_cast<int64_t>(cta) * 2 + x.part) * 256 + w * kTile + r;
      if (!x.whole) ka.ws_ml[at] = make_float2(off, l);
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        float o[16];
        if (some) {
          tmem_ld<16>(to + 16 * c, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = any ? o[j] * f : 0.f;
        if (x.whole) {
          if (row_live) {
#pragma unroll
            for (int j = 0; j < 16; j += 8)
              *reinterpret_cast<uint4*>(out + 16 * c + j) =
                  make_uint4(pack2<BF16>(o[j], o[j + 1]), pack2<BF16>(o[j + 2], o[j + 3]),
                             pack2<BF16>(o[j + 4], o[j + 5]), pack2<BF16>(o[j + 6], o[j + 7]));
          }
        } else {                           // four columns of all rows together
          float4* dst = reinterpret_cast<float4*>(ka.ws_acc) +
                        ((static_cast<int64_t>(cta) * 2 + x.part) * 2 + w) * (kTile * D / 4) + r;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dst[(4 * c + j) * kTile] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kDEmpty + d % kDescs));
    }
  }
  // ---- every role has left its loop, with nothing in flight
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a cut item: CTA w's item is the one that CTA w of the launch
// before left open, with a part in each of the next ones up to where it ends.
constexpr int kMergeRows = 32;             // rows a CTA
template <int D, bool BF16>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ Args ka, int grid) {
  const PrefillArgs& a = ka.a;
  const int w = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int* head = ka.ws_head + w * kHeader;
  griddep_wait();
  if (!head[kHasTail]) return;
  const int t0 = head[kTailT0], h = head[kTailH], tokens = head[kTailTokens];
  const int row = blockIdx.y * kMergeRows + lane, s = row / kTile, r = row % kTile;
  if (s * ka.sub >= tokens) return;        // (of the whole CTA: 32 rows are of one subtile)
  int parts = 2;                             // (w, 1), (w + 1, 0), ..
  while (w + parts < grid && !ka.ws_head[(w + parts - 1) * kHeader + kHeadEnds]) ++parts;
  auto at = [&](int p) { return p == 0 ? w * 2 + 1 : (w + p) * 2; };
  // a lane a row, a warp D / 32 groups of four columns
  float top = -INFINITY;
  for (int p = 0; p < parts; ++p) {
    const float2 ml = ka.ws_ml[at(p) * INT64_C(256) + row];
    if (ml.y != 0.f) top = fmaxf(top, ml.x);
  }
  constexpr int E = D / 32;
  float4 acc[E] = {};
  float l = 0.f;
  for (int p = 0; p < parts; ++p) {
    const float2 ml = ka.ws_ml[at(p) * INT64_C(256) + row];
    const float f = ml.y == 0.f ? 0.f : ml.x == top ? 1.f : fast_exp2(ml.x - top);
    l += ml.y * f;
    const float4* src = reinterpret_cast<const float4*>(ka.ws_acc) +
                        (at(p) * INT64_C(2) + s) * (kTile * D / 4) + warp * E * kTile + r;
    float4 v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = src[e * kTile];
#pragma unroll
    for (int e = 0; e < E; ++e) {          // (a part that saw nothing holds zeros)
      acc[e].x += v[e].x * f;
      acc[e].y += v[e].y * f;
      acc[e].z += v[e].z * f;
      acc[e].w += v[e].w * f;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __shared__ uint2 tile[kMergeRows][D / 4 + 1];
#pragma unroll
  for (int e = 0; e < E; ++e)
    tile[lane][warp * E + e] = make_uint2(pack2<BF16>(acc[e].x * inv, acc[e].y * inv),
                                          pack2<BF16>(acc[e].z * inv, acc[e].w * inv));
  __syncthreads();
  for (int i = threadIdx.x; i < kMergeRows * (D / 4); i += 256) {
    const int k = i / (D / 4), c = i % (D / 4), rk = blockIdx.y * kMergeRows % kTile + k, tk = rk / a.group;
    if (tk >= ka.sub || s * ka.sub + tk >= tokens) continue;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) +
                              ((static_cast<int64_t>(t0) + s * ka.sub + tk) * a.Hq + h * a.group + rk - tk * a.group) * D +
                              4 * c) = tile[k][c];
  }
}

// --------------------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// The map of a 3-D tensor of 16-bit elements (innermost first; the innermost dense) in
// boxes of 64 elements x box1 x box2 with the 128-byte swizzle.  Encoding is host work
// of a few hundred nanoseconds, made for each call: nothing is kept.
cudaError_t tensor_map(CUtensorMap* m, const void* p, const cuuint64_t (&dims)[3],
                       const cuuint64_t (&strides)[2], unsigned box1, unsigned box2) {
  const auto enc = encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint32_t box[3] = {64, box1, box2};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r =
      enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(p), dims, strides, box, elem,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Space {
  size_t ml, acc, total;
};
Space space(int grid, int D) {
  Space s{};
  s.ml = (static_cast<size_t>(grid) * kHeader * 4 + 255) / 256 * 256;
  s.acc = s.ml + static_cast<size_t>(grid) * 2 * 256 * 8;
  s.total = s.acc + static_cast<size_t>(grid) * 2 * 256 * D * 4;
  return s;
}

template <int D, bool BF16, bool FP8>
cudaError_t launch(const PrefillArgs& args, cudaStream_t s) {
  using C = Cfg<D, FP8>;
  Args k{};
  const int grid = device_sm_count();
  const size_t smem = 1024 + C::kBig + sizeof(Small);
  static_assert(1024 + C::kBig + sizeof(Small) <= 232448, "227 KB");
  static_assert(sizeof(Setup) <= C::kBig, "the setup fits in the operands' place");
  auto* kern = prefill_kernel<D, BF16, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  k.sub = kTile / args.group;
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(args.Hq),
                                static_cast<cuuint64_t>(args.T)};
    const cuuint64_t strides[2] = {2 * D, static_cast<cuuint64_t>(args.q_stride) * 2};
    e = tensor_map(&k.tm_q, args.q, dims, strides, static_cast<unsigned>(args.group),
                   static_cast<unsigned>(k.sub));
    if (e != cudaSuccess) return e;
  }
  if (!FP8) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), 16,
                                static_cast<cuuint64_t>(args.num_blocks) * args.Hkv};
    const cuuint64_t strides[2] = {2 * D, 32 * D};
    e = tensor_map(&k.tm_k, args.k_cache, dims, strides, 16, 1);
    if (e == cudaSuccess) e = tensor_map(&k.tm_v, args.v_cache, dims, strides, 16, 1);
    if (e != cudaSuccess) return e;
  }
  const Space sp = space(grid, D);
  uint8_t* ws = static_cast<uint8_t*>(args.workspace);
  k.ws_head = reinterpret_cast<int*>(ws);
  k.ws_ml = reinterpret_cast<float2*>(ws + sp.ml);
  k.ws_acc = reinterpret_cast<float*>(ws + sp.acc);
  // scale 0: every score counts alike, and a masked one still gets the weight 0
  const float sl2 = args.scale * 1.4426950408889634f;
  k.sl2 = fabsf(sl2) > 1e-30f ? sl2 : 1e-30f;
  k.wait_limit_ns = args.wait_limit_ns;
  // an item of up to 2 kSnap tiles is never cut: every place in it is that near a border
  const bool cuts = args.max_context_len > 2 * kSnap * kTile;
  for (int b0 = 0; b0 < args.B; b0 += kMaxSeqs) {
    k.a = args;
    k.a.B = args.B - b0 < kMaxSeqs ? args.B - b0 : kMaxSeqs;
    k.a.block_tables = args.block_tables + static_cast<int64_t>(b0) * args.mbs;
    k.a.context_lens = args.context_lens + b0;
    k.a.starts = args.starts + b0;
    e = launch_after(kern, dim3(static_cast<unsigned>(grid)), C::kThreads, smem, s, k);
    if (e != cudaSuccess) return e;
    if (!cuts) continue;
    e = launch_after(merge_kernel<D, BF16>, dim3(static_cast<unsigned>(grid), 256 / kMergeRows), 256, 0, s, k, grid);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D, bool BF16>
cudaError_t launch(const PrefillArgs& a, bool fp8, cudaStream_t s) {
  return fp8 ? launch<D, BF16, true>(a, s) : launch<D, BF16, false>(a, s);
}

}  // namespace

size_t prefill_workspace_bytes(int, int, int, int, int D) { return space(device_sm_count(), D).total; }

cudaError_t launch_prefill(const PrefillArgs& a, bool fp8, bool bf16, cudaStream_t s) {
  if (a.D == 64) return bf16 ? launch<64, true>(a, fp8, s) : launch<64, false>(a, fp8, s);
  return bf16 ? launch<128, true>(a, fp8, s) : launch<128, false>(a, fp8, s);
}

}  // namespace pa
