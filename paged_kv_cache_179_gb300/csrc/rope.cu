// rope.cu -- rotary positions with several axes, and the append in one launch.
//
// Pair i of a head turns by the angle pos[axis(i)] * f_i: x' = x cos - y sin,
// y' = y cos + x sin.  The angle is reduced in fixed point: f_i is held as a
// 64-bit fraction of a turn (made on the host to 2^-63 of a turn, whatever the
// number of whole turns), the 64-bit product with the position drops whole
// turns by itself, and the upper 32 bits, read as a signed number, are the angle
// in (-1/2, 1/2] turns to 2^-32.  sincospif takes it from there, so a position
// of a million costs what position 1 does and loses nothing, without 64-bit
// floating point.
//
// Bytes: every element of q, k and v read once and written once; six fp32
// operations a pair.  HBM-bound for prompts, launch-bound for decode steps.
// One CTA serves one or two tokens: its threads compute their cos and sin once into
// shared memory, then walk over the tokens' heads, 32 bytes at a time.  Measured on
// a GB300 with 28 + 4 + 4 heads of 128: 56.6 us for 16384 bf16 tokens (302 MB, 79 %
// of the measured copy bandwidth), 6.1 us for 512, 4.3 us for 4 (8 heads of 64).
// 16 tokens of the same heads take 4.2 us with 512 threads a CTA, 6.2 us with 128.
// Prompts: 128 threads and two tokens a CTA; 256 threads 57 to 61 us, one token 63 us, four
// tokens 57 us, eight 68 us; two and more rows in flight a thread 65 us.
#include "pa_e4m3.cuh"
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeFewThreads = 512;   // of a CTA, while the tokens do not fill the GPU
constexpr int kRopeTokens = 2;   // most a CTA serves

__device__ __forceinline__ float2 rope_sincos(uint64_t turns, int32_t pos, float amplitude) {
  const uint64_t turn = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const int32_t top = static_cast<int32_t>(turn >> 32);
  float s, c;
  // half turns; the 24-bit rounding of the conversion is 2^-25 of half a turn
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}

// ceil(2^32 / rows): i / rows = umulhi(i, magic) for i below 4096, or below rows
// (at most 65535).  0 for one row: a CTA then serves one token.
__host__ __device__ __forceinline__ uint32_t rope_magic(int rows) {
  return rows == 1 ? 0u : static_cast<uint32_t>((0xffffffffull + rows) / rows);
}

// The two 16-byte chunks that item i of a head's row works on.  Rotated chunks
// come as the pair whose elements turn together (apart by rotary_dim / 2) or,
// for adjacent pairs, as two neighbours; both then use pairs 8i .. 8i + 7.
// b is -1 when the row ends with an odd chunk.
__device__ __forceinline__ void rope_chunks(const RopeArgs& a, int i, int& ca, int& cb,
                                            bool& turned) {
  const int rot_items = a.pairs / 8;
  turned = i < rot_items;
  if (turned && !a.adjacent) {
    ca = i;
    cb = i + rot_items;
  } else {
    ca = 2 * i;
    cb = 2 * i + 1 < a.D / 8 ? 2 * i + 1 : -1;
  }
}

// x cos - y sin and y cos + x sin, with the roundings fixed (one product, one
// fused multiply-add), so that every kernel here rotates to the same bits.
__device__ __forceinline__ float turn_x(float x, float y, float2 cs) {
  return __fmaf_rn(x, cs.x, -__fmul_rn(y, cs.y));
}
__device__ __forceinline__ float turn_y(float x, float y, float2 cs) {
  return __fmaf_rn(y, cs.x, __fmul_rn(x, cs.y));
}

template <bool BF16>
__device__ __forceinline__ uint32_t turn_adjacent(uint32_t w, float2 cs) {
  const float2 v = bits2_to_float2<BF16>(w);
  return pack2<BF16>(turn_x(v.x, v.y, cs), turn_y(v.x, v.y, cs));
}
// Words of two chunks whose elements are each other's partners.
template <bool BF16>
__device__ __forceinline__ void turn_half(uint32_t& lo, uint32_t& hi, float2 cs0, float2 cs1) {
  const float2 x = bits2_to_float2<BF16>(lo), y = bits2_to_float2<BF16>(hi);
  lo = pack2<BF16>(turn_x(x.x, y.x, cs0), turn_x(x.y, y.y, cs1));
  hi = pack2<BF16>(turn_y(x.x, y.x, cs0), turn_y(x.y, y.y, cs1));
}

template <bool BF16>
__device__ __forceinline__ void turn_chunks(uint4& va, uint4& vb, const float2 (&cs)[8],
                                            bool adjacent) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&va);
  uint32_t* b = reinterpret_cast<uint32_t*>(&vb);
  if (adjacent) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = turn_adjacent<BF16>(a[j], cs[j]);
      b[j] = turn_adjacent<BF16>(b[j], cs[4 + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) turn_half<BF16>(a[j], b[j], cs[2 * j], cs[2 * j + 1]);
  }
}

// One CTA serves `toks` tokens from `first` on; threads (x, y): x the item of a
// head's row, y the row.  A token's rows 0 .. Hq-1 are q's, then Hkv of k, then (with
// an append) Hkv of v.  A thread's next row is on its way while it works on one, its
// first while cos and sin are computed.
template <bool BF16>
__device__ __forceinline__ void rope_tokens(const RopeArgs& a, const RopeTable& t, int64_t first,
                                            int toks, int rows, uint32_t rows_magic,
                                            float2* cs_smem, int64_t* slot_smem) {
  const int items = (a.D + 15) / 16;
  const int x = threadIdx.x % items, y = threadIdx.x / items, ny = blockDim.x / items;
  const int chunks = a.D / 8;
  int ca, cb;
  bool turned;
  rope_chunks(a, x, ca, cb, turned);
  const int total = y < ny ? toks * rows : 0;   // threads behind the last whole row of items: none
  uint4 va, vb, next_a, next_b;
  auto load = [&](int i) {
    if (i >= total) return;
    const int tok = static_cast<int>(__umulhi(static_cast<uint32_t>(i), rows_magic)), r = i - tok * rows;
    const uint16_t* src;
    if (r < a.Hq) src = static_cast<const uint16_t*>(a.q) + (first + tok) * a.q_stride + r * a.D;
    else if (r < a.Hq + a.Hkv)
      src = static_cast<const uint16_t*>(a.k) + (first + tok) * a.k_stride + (r - a.Hq) * a.D;
    else
      src = static_cast<const uint16_t*>(a.v) + (first + tok) * a.v_stride + (r - a.Hq - a.Hkv) * a.D;
    next_a = __ldcs(reinterpret_cast<const uint4*>(src) + ca);
    next_b = cb >= 0 ? __ldcs(reinterpret_cast<const uint4*>(src) + cb) : make_uint4(0, 0, 0, 0);
  };
  load(y);
  for (int i = threadIdx.x; i < toks * a.pairs; i += blockDim.x) {
    const int tok = i / a.pairs, p = i - tok * a.pairs;
    const int32_t pos = __ldg(a.positions + static_cast<int64_t>(t.axis[p]) * a.T + first + tok);
    cs_smem[tok * kMaxRopePairs + p] = rope_sincos(t.turns[p], pos, a.amplitude);
  }
  if (a.slots != nullptr && static_cast<int>(threadIdx.x) < toks) {
    int64_t slot = __ldg(a.slots + first + threadIdx.x);
    if (slot >= a.num_blocks * a.block_size) {
      atomicOr(a.status, kStatusBadSlot);
      slot = -1;
    }
    // the slot's row of its block's first head, in rows; -1: nothing is appended
    slot_smem[threadIdx.x] =
        slot < 0 ? -1 : slot / a.block_size * a.Hkv * a.block_size + slot % a.block_size;
  }
  __syncthreads();
  for (int i = y; i < total; i += ny) {
    va = next_a, vb = next_b;
    load(i + ny);
    const int tok = static_cast<int>(__umulhi(static_cast<uint32_t>(i), rows_magic)), r = i - tok * rows;
    uint4* dst;
    if (r < a.Hq) {
      dst = static_cast<uint4*>(a.q_out) + ((first + tok) * a.Hq + r) * chunks;
    } else {
      const bool is_v = r >= a.Hq + a.Hkv;
      const int h = r - a.Hq - (is_v ? a.Hkv : 0);
      if (a.slots != nullptr) {
        if (slot_smem[tok] < 0) continue;
        dst = static_cast<uint4*>(is_v ? a.v_cache : a.k_cache) +
              (slot_smem[tok] + h * a.block_size) * chunks;
      } else {
        dst = static_cast<uint4*>(a.k_out) + ((first + tok) * a.Hkv + h) * chunks;
      }
    }
    if (turned && r < a.Hq + a.Hkv) {
      float2 cs[8];
      const float4* from = reinterpret_cast<const float4*>(cs_smem + tok * kMaxRopePairs + 8 * x);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float4 v = from[n];
        cs[2 * n] = make_float2(v.x, v.y);
        cs[2 * n + 1] = make_float2(v.z, v.w);
      }
      turn_chunks<BF16>(va, vb, cs, a.adjacent != 0);
    }
    dst[ca] = va;
    if (cb >= 0) dst[cb] = vb;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kRopeFewThreads)
rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable t, int rows,
            uint32_t rows_magic, int toks) {
  __shared__ __align__(16) float2 cs[kRopeTokens * kMaxRopePairs];
  __shared__ int64_t slots[kRopeTokens];
  const int64_t first = static_cast<int64_t>(blockIdx.x) * toks;
  rope_tokens<BF16>(a, t, first, static_cast<int>(min(static_cast<int64_t>(toks), a.T - first)), rows,
                    rows_magic, cs, slots);
}

// The E4M3 append: CTAs 0 .. T-1 rotate q; in the others one warp takes one
// (token, kv head, K|V) row, rotates K's and encodes it as append_fp8_kernel
// does (the rotated row is rounded to the activations' type first).
template <int D, bool BF16>
__global__ void __launch_bounds__(kRopeThreads)
rope_append_fp8_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable t,
                       int q_ctas) {
  __shared__ __align__(16) float2 cs[kMaxRopePairs];
  if (static_cast<int>(blockIdx.x) < q_ctas) {
    RopeArgs q = a;
    q.Hkv = 0;
    q.slots = nullptr;
    rope_tokens<BF16>(q, t, blockIdx.x, 1, a.Hq, rope_magic(a.Hq), cs, nullptr);
    return;
  }
  constexpr int P = RowF16<D>::PER_LANE;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x - q_ctas) * (kRopeThreads / 32) +
                    (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.T) * a.Hkv * 2) return;
  const int kv = static_cast<int>(w & 1);
  const int64_t th = w >> 1;
  const int64_t tok = th / a.Hkv, h = th - tok * a.Hkv;
  const int64_t s = __ldg(a.slots + tok);
  if (s < 0) return;
  if (s >= a.num_blocks * a.block_size) {
    if (lane == 0 && kv == 0 && h == 0) atomicOr(a.status, kStatusBadSlot);
    return;
  }
  const int64_t blk = s / a.block_size, row = s - blk * a.block_size;
  const uint16_t* src = kv ? static_cast<const uint16_t*>(a.v) + tok * a.v_stride + h * D
                           : static_cast<const uint16_t*>(a.k) + tok * a.k_stride + h * D;
  RowF16<D> x = load_row<D, BF16>(src, lane);
  if (!kv) {
    const int e0 = lane * P;   // the lane's first element
    if (a.adjacent) {
#pragma unroll
      for (int j = 0; j < P; j += 2) {
        const int i = (e0 + j) / 2;
        if (i < a.pairs) {
          const float2 c = rope_sincos(t.turns[i],
              __ldg(a.positions + static_cast<int64_t>(t.axis[i]) * a.T + tok), a.amplitude);
          const float u = x.x[j], v = x.x[j + 1];
          x.x[j] = turn_x(u, v, c);
          x.x[j + 1] = turn_y(u, v, c);
        }
      }
    } else {
      // pairs is a multiple of 8, so a lane's elements all lie in the first
      // half, in the second, or behind; the partners are `pairs / P` lanes away
      const bool lo = e0 < a.pairs, hi = !lo && e0 < 2 * a.pairs;
      const int from = lo ? lane + a.pairs / P : hi ? lane - a.pairs / P : lane;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float other = __shfl_sync(0xffffffffu, x.x[j], from);
        if (lo || hi) {
          const int i = e0 + j - (hi ? a.pairs : 0);
          const float2 c = rope_sincos(t.turns[i],
              __ldg(a.positions + static_cast<int64_t>(t.axis[i]) * a.T + tok), a.amplitude);
          x.x[j] = lo ? turn_x(x.x[j], other, c) : turn_y(other, x.x[j], c);
        }
      }
    }
    // rounded to the activations' type, as a separate rotation would store it
#pragma unroll
    for (int j = 0; j < P; j += 2) {
      const float2 r = bits2_to_float2<BF16>(pack2<BF16>(x.x[j], x.x[j + 1]));
      x.x[j] = r.x;
      x.x[j + 1] = r.y;
    }
  }
  float* scales = kv ? a.v_scale : a.k_scale;
  const int64_t tile = blk * a.Hkv + h;
  uint8_t* page = static_cast<uint8_t*>(kv ? a.v_cache : a.k_cache) + tile * a.block_size * D;
  const float amax = e4m3_row_amax<D>(x);
  float scale;
  if (row == 0) {
    scale = e4m3_page_scale(amax);
    if (lane == 0) scales[tile] = scale;
  } else {
    scale = scales[tile];
    if (e4m3_saturates(amax, scale)) {   // re-scale the page's earlier rows first
      const float s_new = e4m3_page_scale(amax);
      e4m3_rescale_rows<D, true>(page, page, nullptr, static_cast<int>(row), scale, s_new, lane);
      scale = s_new;
      if (lane == 0) scales[tile] = scale;
    }
  }
  store_row_codes<D>(page + row * D, lane, e4m3_row_codes<D>(x, scale));
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, const RopeTable& t, bool bf16, cudaStream_t s) {
  const int rows = a.Hq + a.Hkv * (a.v != nullptr ? 2 : 1);
  if (rows == 0) return cudaSuccess;
  // several tokens a CTA once that still leaves the GPU full; up to 4096 rows
  int toks = 1;
  while (rows > 1 && toks < kRopeTokens && 2 * toks * rows <= 4096 && a.T / (2 * toks) >= 4 * device_sm_count()) toks *= 2;
  const int items = (a.D + 15) / 16;
  // rows a CTA takes at once; few tokens are done sooner by more threads each
  const int most = (a.T <= 2 * device_sm_count() ? kRopeFewThreads : kRopeThreads) / items;
  const int passes = (toks * rows + most - 1) / most;
  const int threads = (toks * rows + passes - 1) / passes * items;
  auto* kernel = bf16 ? rope_kernel<true> : rope_kernel<false>;
  const int ctas = a.T / toks + (a.T % toks != 0);   // T + toks - 1 may pass 32 bits
  kernel<<<static_cast<unsigned>(ctas), threads, 0, s>>>(a, t, rows, rope_magic(rows), toks);
  return cudaGetLastError();
}

cudaError_t launch_rope_append_fp8(const RopeArgs& a, const RopeTable& t, bool bf16,
                                   cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(a.T) * a.Hkv * 2;
  const int q_ctas = a.Hq > 0 ? a.T : 0;
  const int64_t grid = q_ctas + (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  auto* kernel = a.D == 128 ? (bf16 ? rope_append_fp8_kernel<128, true>
                                    : rope_append_fp8_kernel<128, false>)
                            : (bf16 ? rope_append_fp8_kernel<64, true>
                                    : rope_append_fp8_kernel<64, false>);
  kernel<<<static_cast<unsigned>(grid), kRopeThreads, 0, s>>>(a, t, q_ctas);
  return cudaGetLastError();
}

}  // namespace pa
