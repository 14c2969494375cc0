// Attention over a block-scaled e4m3 cache, one warp per (query row, query head): the lanes
// share head_dim, the warp walks the visible keys one after another with the running maximum
// and sum of the softmax in float32.
#include "common.cuh"
#include "kernels.h"

namespace fkv {
namespace {

// The float32 values of N e4m3 codes at p.
template <int N>
FKV_DEV void decode_codes(const uint8_t* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(reinterpret_cast<const uint16_t*>(p)[i]));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// One query row against keys [lo, hi) of sequence b.
template <int D>
FKV_DEV void attend_row(const BlockPrefillParams& p, int b, int h, long long row, int lo, int hi) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, g = h / (p.Hq / p.Hkv);
  float q[E], acc[E];
  const __nv_bfloat16* src = p.q + (row * p.Hq + h) * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(src[i]);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    int id = p.block_table[static_cast<size_t>(b) * p.max_blocks + (j >> 4)];
    if (id < 0 || id >= p.num_blocks) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
      id = 0;
    }
    const size_t at = (static_cast<size_t>(id) * p.Hkv + g) * 16 * D + (j & 15) * D + lane * E;
    const size_t sc = static_cast<size_t>(id) * p.Hkv + g;
    float k[E], v[E], x = 0.f;
    decode_codes(p.k_cache + at, k);
    decode_codes(p.v_cache + at, v);
#pragma unroll
    for (int i = 0; i < E; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x *= p.k_scale[sc] * p.sm_scale_log2;
    const float mn = fmaxf(m, x);
    const float alpha = m == -INFINITY ? 0.f : ex2(m - mn), w = ex2(x - mn);
    m = mn;
    l = fmaf(l, alpha, w);
    const float wv = w * p.v_scale[sc];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = fmaf(acc[i], alpha, wv * v[i]);
  }
  const float inv = hi > lo ? 1.f / l : 0.f;
  __nv_bfloat16* dst = p.out + (row * p.Hq + h) * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) dst[i] = __float2bfloat16(acc[i] * inv);
}

// Context length of sequence b, clamped to what the block table addresses.
FKV_DEV int clamped_context(const BlockPrefillParams& p, int b, bool report) {
  const int T = p.ctx[b];
  if (T >= 0 && T <= static_cast<long long>(p.max_blocks) * 16) return T;
  if (report) raise_fault(p.fault, FKV_FAULT_CONTEXT);
  return T < 0 ? 0 : p.max_blocks * 16;
}

// grid (query rows / 4, Hq, B), 4 warps.
template <int D>
__global__ void __launch_bounds__(128) block_prefill_kernel(const BlockPrefillParams p) {
  const int b = blockIdx.z, h = blockIdx.y, i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const bool first = blockIdx.x == 0 && h == 0 && threadIdx.x == 0;
  const int T = clamped_context(p, b, first);
  const int r0 = p.cu[b], L = p.cu[b + 1] - r0;
  if (L < 0 || L > p.max_q_len || (p.causal && L > T) || r0 < 0 || r0 + static_cast<long long>(L) > p.total_q) {
    if (first) raise_fault(p.fault, FKV_FAULT_QLEN);
    return;
  }
  if (i >= L) return;
  const int pos = T - L + i;
  attend_row<D>(p, b, h, r0 + static_cast<long long>(i), p.window > 0 ? max(0, pos - p.window + 1) : 0,
                p.causal ? pos + 1 : T);
}

}  // namespace

cudaError_t launch_block_prefill(const BlockPrefillParams& p, int D, cudaStream_t s) {
  const dim3 grid((p.max_q_len + 3) / 4, p.Hq, p.B);
  auto kern = D == 64 ? block_prefill_kernel<64> : D == 128 ? block_prefill_kernel<128> : block_prefill_kernel<256>;
  kern<<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fkv
