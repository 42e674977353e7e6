// prefill.cu -- attention of prompts over the paged cache: the plain form, which
// the checks hold faster ones to.  A CTA takes 64 query rows (token, head of the
// group) of one (sequence, kv head), eight a warp, and walks the pages they see:
// keys and values as fp32 in shared memory, a lane holding D / 32 elements of each
// row's query and result, an online softmax in fp32.
#include "pa_launch.h"
#include "pa_ptx.cuh"
#include "request_launch.h"

namespace pa {
namespace {

constexpr int kRows = 64, kWarps = 8, kPer = kRows / kWarps;

template <int D, bool BF16>
__device__ __forceinline__ float load16(const void* p, int64_t i) {
  const uint16_t w = static_cast<const uint16_t*>(p)[i];
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
  else return __half2float(*reinterpret_cast<const __half*>(&w));
}

template <int D, bool BF16, bool FP8>
__global__ void __launch_bounds__(kWarps * 32) prefill_kernel(const PrefillArgs a) {
  constexpr int E = D / 32;
  __shared__ float sk[16][D], sv[16][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
  // the tile: blockIdx.x counts 64-row tiles over all sequences
  int tile = blockIdx.x, b = 0, n = 0;
  for (; b < a.B; ++b) {
    const int s0 = a.starts[b], s1 = a.starts[b + 1];
    const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.T;
    if (!ok && tile == 0 && tid == 0 && h == 0) atomicOr(a.status, kStatusBadLen);
    n = ok ? s1 - s0 : 0;
    const int tiles = (n * a.group + kRows - 1) / kRows;
    if (tile < tiles) break;
    tile -= tiles;
  }
  if (b == a.B) return;
  int L = a.context_lens[b];
  if (L < 0 || L > a.max_context_len) {
    if (tid == 0) atomicOr(a.status, kStatusBadLen);
    L = 0;
  }
  const int t0 = a.starts[b];
  float q[kPer][E], o[kPer][E], m[kPer], l[kPer];
  int pos[kPer];
  int first = INT32_MAX, last = -1;
  for (int r = 0; r < kPer; ++r) {
    const int row = tile * kRows + warp * kPer + r, i = row / a.group, g = row % a.group;
    pos[r] = row < n * a.group ? L - n + i : -1;
    m[r] = -INFINITY;
    l[r] = 0.f;
    for (int e = 0; e < E; ++e) {
      o[r][e] = 0.f;
      q[r][e] = pos[r] >= 0 ? load16<D, BF16>(a.q, (t0 + i) * a.q_stride + (h * a.group + g) * D + lane * E + e) * a.scale : 0.f;
    }
  }
  {
    const int i0 = tile * kRows / a.group, i1 = min(n - 1, (tile * kRows + kRows - 1) / a.group);
    last = L - n + i1;
    first = a.window > 0 ? max(0, L - n + i0 - a.window + 1) : 0;
  }
  for (int p = first / 16; p <= last / 16 && last >= 0; ++p) {
    const int id = a.block_tables[static_cast<int64_t>(b) * a.mbs + p];
    const bool ok = id >= 0 && id < a.num_blocks;
    if (!ok) {
      if (tid == 0) atomicOr(a.status, kStatusBadBlock);
      continue;
    }
    __syncthreads();
    const int64_t page = (static_cast<int64_t>(id) * a.Hkv + h) * 16 * D;
    const float ks = FP8 ? a.k_scale[static_cast<int64_t>(id) * a.Hkv + h] : 1.f;
    const float vs = FP8 ? a.v_scale[static_cast<int64_t>(id) * a.Hkv + h] : 1.f;
    for (int e = tid; e < 16 * D; e += kWarps * 32) {
      const bool in = p * 16 + e / D < L;
      float k, v;
      if constexpr (FP8) {
        const uint32_t two = static_cast<const uint8_t*>(a.k_cache)[page + e] |
                             static_cast<const uint8_t*>(a.v_cache)[page + e] << 8;
        const uint32_t w = e4m3x2_to_f16x2(two);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        k = f.x * ks;
        v = f.y * vs;
      } else {
        k = load16<D, BF16>(a.k_cache, page + e);
        v = load16<D, BF16>(a.v_cache, page + e);
      }
      sk[e / D][e % D] = in ? k : 0.f;
      sv[e / D][e % D] = in ? v : 0.f;
    }
    __syncthreads();
    for (int r = 0; r < kPer; ++r) {
      for (int j = 0; j < 16; ++j) {
        const int at = p * 16 + j;
        if (at > pos[r] || (a.window > 0 && at <= pos[r] - a.window)) continue;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s = fmaf(q[r][e], sk[j][lane * E + e], s);
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float mn = fmaxf(m[r], s);
        if (mn == -INFINITY) continue;
        const float f = expf(m[r] - mn), x = expf(s - mn);
        m[r] = mn;
        l[r] = l[r] * f + x;
        for (int e = 0; e < E; ++e) o[r][e] = o[r][e] * f + x * sv[j][lane * E + e];
      }
    }
  }
  for (int r = 0; r < kPer; ++r) {
    const int row = tile * kRows + warp * kPer + r, i = row / a.group, g = row % a.group;
    if (row >= n * a.group) continue;
    uint16_t* out = static_cast<uint16_t*>(a.out) + ((static_cast<int64_t>(t0) + i) * a.Hq + h * a.group + g) * D;
    for (int e = 0; e < E; ++e)
      out[lane * E + e] = static_cast<uint16_t>(pack2<BF16>(l[r] > 0.f ? o[r][e] / l[r] : 0.f, 0.f));
  }
}

template <int D, bool BF16>
cudaError_t launch(const PrefillArgs& a, bool fp8, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.T) * a.group;
  const dim3 grid(static_cast<unsigned>(rows / kRows + a.B), static_cast<unsigned>(a.Hkv));
  if (fp8) prefill_kernel<D, BF16, true><<<grid, kWarps * 32, 0, s>>>(a);
  else prefill_kernel<D, BF16, false><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t prefill_workspace_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_prefill(const PrefillArgs& a, bool fp8, bool bf16, cudaStream_t s) {
  if (a.D == 64) return bf16 ? launch<64, true>(a, fp8, s) : launch<64, false>(a, fp8, s);
  return bf16 ? launch<128, true>(a, fp8, s) : launch<128, false>(a, fp8, s);
}

}  // namespace pa
