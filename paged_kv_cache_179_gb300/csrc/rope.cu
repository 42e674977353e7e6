// rope.cu -- rotary positions with several axes, and the append in one launch.
//
// Pair i of a head turns by the angle pos[axis(i)] * f_i: x' = x cos - y sin,
// y' = y cos + x sin.  The angle is reduced in fixed point: f_i is held as a
// 64-bit fraction of a turn, the 64-bit product with the position drops whole
// turns by itself, and the upper 32 bits, read as a signed number, are the angle
// in (-1/2, 1/2] turns to 2^-32.  sincospif takes it from there, so a position
// of a million costs what position 1 does and loses nothing, without 64-bit
// floating point.
//
// Bytes: every element of q, k and v read once and written once; six fp32
// operations a pair.  HBM-bound for prompts, launch-bound for decode steps.
// One CTA serves one token: its threads compute the token's cos and sin once
// into shared memory, and each thread then holds the eight pairs of one 16-byte
// chunk pair while it walks over the token's heads.
#include "pa_e4m3.cuh"
#include "pa_ptx.cuh"
#include "serving_launch.h"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 rope_sincos(uint64_t turns, int32_t pos, float amplitude) {
  const uint64_t turn = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const int32_t top = static_cast<int32_t>(turn >> 32);
  float s, c;
  // half turns; the 24-bit rounding of the conversion is 2^-25 of half a turn
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}

// cos and sin of the token's pairs into cs[0 .. pairs).
__device__ __forceinline__ void rope_angles(const RopeArgs& a, const RopeTable& t, int64_t tok,
                                            float2* cs, int tid, int threads) {
  for (int i = tid; i < a.pairs; i += threads) {
    const int32_t pos = __ldg(a.positions + static_cast<int64_t>(t.axis[i]) * a.T + tok);
    cs[i] = rope_sincos(t.turns[i], pos, a.amplitude);
  }
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

// One CTA per token; threads (x, y): x the item of a head's row, y the row.
// Rows 0 .. Hq-1 are q's, then Hkv of k, then (with an append) Hkv of v.
template <bool BF16>
__device__ __forceinline__ void rope_token(const RopeArgs& a, const RopeTable& t, int64_t tok,
                                           int rows, float2* cs_smem) {
  const int items = (a.D + 15) / 16;
  const int x = threadIdx.x % items, y = threadIdx.x / items, ny = blockDim.x / items;
  rope_angles(a, t, tok, cs_smem, threadIdx.x, blockDim.x);
  int64_t dst_tok = tok;   // of k and v
  bool append = false;
  if (a.slots != nullptr) {
    const int64_t slot = __ldg(a.slots + tok);
    append = slot >= 0;
    if (slot >= a.num_blocks * a.block_size) {
      append = false;
      if (threadIdx.x == 0) atomicOr(a.status, kStatusBadSlot);
    }
    dst_tok = slot;
  }
  __syncthreads();
  int ca, cb;
  bool turned;
  rope_chunks(a, x, ca, cb, turned);
  float2 cs[8];
  if (turned) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = cs_smem[8 * x + j];
  }
  const int chunks = a.D / 8;
  if (y >= ny) return;   // threads behind the last whole row of items
  for (int r = y; r < rows; r += ny) {
    const uint4* src;
    uint4* dst;
    bool rotate = turned;
    if (r < a.Hq) {
      src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + tok * a.q_stride) +
            r * chunks;
      dst = static_cast<uint4*>(a.q_out) + (tok * a.Hq + r) * chunks;
    } else {
      const bool is_v = r >= a.Hq + a.Hkv;
      const int h = r - a.Hq - (is_v ? a.Hkv : 0);
      src = reinterpret_cast<const uint4*>(is_v
                ? static_cast<const uint16_t*>(a.v) + tok * a.v_stride
                : static_cast<const uint16_t*>(a.k) + tok * a.k_stride) + h * chunks;
      if (a.slots != nullptr) {
        if (!append) continue;
        const int64_t blk = dst_tok / a.block_size, row = dst_tok - blk * a.block_size;
        dst = static_cast<uint4*>(is_v ? a.v_cache : a.k_cache) +
              ((blk * a.Hkv + h) * a.block_size + row) * chunks;
      } else {
        dst = static_cast<uint4*>(a.k_out) + (tok * a.Hkv + h) * chunks;
      }
      rotate = turned && !is_v;
    }
    uint4 va = src[ca], vb = make_uint4(0, 0, 0, 0);
    if (cb >= 0) vb = src[cb];
    if (rotate) turn_chunks<BF16>(va, vb, cs, a.adjacent != 0);
    dst[ca] = va;
    if (cb >= 0) dst[cb] = vb;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable t, int rows) {
  __shared__ float2 cs[kMaxRopePairs];
  rope_token<BF16>(a, t, blockIdx.x, rows, cs);
}

// The E4M3 append: CTAs 0 .. T-1 rotate q; in the others one warp takes one
// (token, kv head, K|V) row, rotates K's and encodes it as append_fp8_kernel
// does (the rotated row is rounded to the activations' type first).
template <int D, bool BF16>
__global__ void __launch_bounds__(kRopeThreads)
rope_append_fp8_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTable t,
                       int q_ctas) {
  __shared__ float2 cs[kMaxRopePairs];
  if (static_cast<int>(blockIdx.x) < q_ctas) {
    rope_token<BF16>(a, t, blockIdx.x, a.Hq, cs);
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
  const int items = (a.D + 15) / 16;
  const int most = kRopeThreads / items;   // rows a full CTA takes at once
  const int passes = (rows + most - 1) / most;
  const int threads = (rows + passes - 1) / passes * items;
  auto* kernel = bf16 ? rope_kernel<true> : rope_kernel<false>;
  kernel<<<static_cast<unsigned>(a.T), threads, 0, s>>>(a, t, rows);
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
