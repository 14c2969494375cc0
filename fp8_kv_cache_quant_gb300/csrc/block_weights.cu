// The attention weight that the cached keys of a block-scaled pool receive from a chunk of queries, summed over the
// queries and the heads of a KV head's group: w_j = sum over rows r of 2^(x_rj - lse_r), x_rj = q_r . k_j * ks *
// softmax_scale * log2(e), lse_r = log2 sum_j 2^(x_rj).
//
// One CTA per row finds lse_r; then a thread per key adds up its column, in row order.
#include "block_common.cuh"

namespace fkv {
namespace {

// Sequence b's rows and keys; rows 0: nothing to do.
struct WeightsSeq {
  int r0, rows, T;
};
FKV_DEV WeightsSeq weights_seq(const BlockWeightsParams& p, int b, bool report) {
  WeightsSeq s;
  s.r0 = p.cu[b];
  s.rows = p.cu[b + 1] - s.r0;
  s.T = p.ctx[b];
  const long long most = min(p.max_blocks * 16LL, static_cast<long long>(p.weights_len));
  if (s.T < 0 || s.T > most) {
    if (report) raise_fault(p.fault, FKV_FAULT_CONTEXT);
    s.T = s.T < 0 ? 0 : static_cast<int>(most);
  }
  if (s.rows < 0 || s.rows > p.max_q_len || s.rows > s.T || s.r0 < 0 || s.r0 + static_cast<long long>(s.rows) > p.total_q) {
    if (report) raise_fault(p.fault, FKV_FAULT_QLEN);
    s.rows = 0;
  }
  return s;
}

template <int D>
FKV_DEV float score(const BlockWeightsParams& p, const __nv_bfloat16* q, int b, int g, int j) {
  int id = p.block_table[static_cast<size_t>(b) * p.max_blocks + (j >> 4)];
  if (id < 0 || id >= p.num_blocks) {
    raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
    id = 0;
  }
  const size_t at = static_cast<size_t>(id) * p.Hkv + g;
  const uint32_t* k = reinterpret_cast<const uint32_t*>(p.k_cache + (at * 16 + (j & 15)) * D);
  const uint2* qv = reinterpret_cast<const uint2*>(q);
  float x = 0.f;
  for (int i = 0; i < D / 4; ++i) {
    const uint32_t w = k[i];
    const uint2 y = qv[i];
    uint32_t h01, h23;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"(static_cast<uint16_t>(w >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01)), c = __half22float2(*reinterpret_cast<const __half2*>(&h23));
    const float2 q0 = bf16x2_to_f2(y.x), q1 = bf16x2_to_f2(y.y);
    x = fmaf(a.x, q0.x, x);
    x = fmaf(a.y, q0.y, x);
    x = fmaf(c.x, q1.x, x);
    x = fmaf(c.y, q1.y, x);
  }
  return x * p.k_scale[at] * p.sm_scale_log2;
}

constexpr int kThreads = 256;

// grid (query rows and heads of a sequence, 1, sequences)
template <int D>
__global__ void __launch_bounds__(kThreads) stats_kernel(const BlockWeightsParams p) {
  __shared__ float m_s[kThreads / 32], l_s[kThreads / 32];
  griddep_wait();
  const int b = blockIdx.z;
  const WeightsSeq s = weights_seq(p, b, blockIdx.x == 0 && threadIdx.x == 0);
  const int t = blockIdx.x / p.Hq, h = blockIdx.x - t * p.Hq;
  if (t >= s.rows) return;
  const __nv_bfloat16* q = p.q + (static_cast<size_t>(s.r0 + t) * p.Hq + h) * D;
  const int last = s.T - s.rows + t;
  float m = -3e38f, l = 0.f;
  for (int j = threadIdx.x; j <= last; j += kThreads) {
    const float x = score<D>(p, q, b, h / (p.Hq / p.Hkv), j);
    const float mx = fmaxf(m, x);
    l = l * exp2f(m - mx) + exp2f(x - mx);
    m = mx;
  }
  for (int off = 16; off > 0; off >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, off), l2 = __shfl_xor_sync(0xffffffffu, l, off), mx = fmaxf(m, m2);
    l = l * exp2f(m - mx) + l2 * exp2f(m2 - mx);
    m = mx;
  }
  if ((threadIdx.x & 31) == 0) {
    m_s[threadIdx.x >> 5] = m;
    l_s[threadIdx.x >> 5] = l;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) {
      const float mx = fmaxf(m, m_s[i]);
      l = l * exp2f(m - mx) + l_s[i] * exp2f(m_s[i] - mx);
      m = mx;
    }
    p.lse[static_cast<size_t>(s.r0 + t) * p.Hq + h] = m + log2f(l);
  }
}

// grid (tiles of keys, KV heads, sequences)
template <int D>
__global__ void __launch_bounds__(kThreads) sums_kernel(const BlockWeightsParams p) {
  griddep_wait();
  const int b = blockIdx.z, g = blockIdx.y, j = blockIdx.x * kThreads + threadIdx.x;
  const WeightsSeq s = weights_seq(p, b, false);
  if (s.rows == 0 || j >= s.T) return;
  const int G = p.Hq / p.Hkv, old = s.T - s.rows;
  float* w = p.weights + (static_cast<size_t>(b) * p.Hkv + g) * p.weights_len + j;
  float sum = 0.f;
  for (int t = max(0, j - old); t < s.rows; ++t)
    for (int h = g * G; h < (g + 1) * G; ++h) {
      const size_t row = static_cast<size_t>(s.r0 + t) * p.Hq + h;
      sum += exp2f(score<D>(p, p.q + row * D, b, g, j) - p.lse[row]);
    }
  *w = j < old && p.decay != 0.f ? fmaf(p.decay, *w, sum) : sum;
}

template <int D>
cudaError_t launch_t(const BlockWeightsParams& p, cudaStream_t s) {
  const cudaError_t e = launch_dependent(stats_kernel<D>, dim3(p.max_q_len * p.Hq, 1, p.B), dim3(kThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  const long long keys = std::min(p.max_blocks * 16LL, static_cast<long long>(p.weights_len));
  return launch_dependent(sums_kernel<D>, dim3(static_cast<unsigned>((keys + kThreads - 1) / kThreads), p.Hkv, p.B), dim3(kThreads), 0, s, p);
}

}  // namespace

size_t block_weights_workspace(int B, int total_q, int max_q_len, int Hq, int Hkv, int D, long long keys) {
  return 4 * static_cast<size_t>(total_q) * Hq;
}

cudaError_t launch_block_weights(const BlockWeightsParams& p, int D, int num_sms, cudaStream_t s) {
  if (D == 64) return launch_t<64>(p, s);
  if (D == 128) return launch_t<128>(p, s);
  return launch_t<256>(p, s);
}

}  // namespace fkv
