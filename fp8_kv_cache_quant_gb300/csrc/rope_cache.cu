// The cache writes that apply the rotary position embedding on the way: kv_rope_cache
// (slot-mapped, pools with per-tensor or per-head scales, or bf16) and kv_block_cache
// (block-scaled e4m3 pools).
//
// A head's row is handled in units of 16 elements, two 16-byte chunks whose elements pair up
// under the rotation, so that a pair's two halves meet in one thread: with the half split,
// chunks u and u + rot_dim / 16 of the turned part; otherwise two neighbouring chunks.  In
// both styles unit u of the turned part takes table entries 8 u .. 8 u + 7.
// The products and the sum of a rotation are rounded one by one to float32 (no fused
// multiply-add), as an elementwise evaluation rounds them, so that the codes are reproducible.
#include "block_common.cuh"

namespace fkv {
namespace {

// The kernels are launched while the one before in the stream finishes; their CTAs wait here, before they
// touch global memory, and only then let the next such kernel's in, so that what that one finds
// running are CTAs of this kernel alone.  4,133 tokens of 64/8 heads at head_dim 64 18.5 -> 16.9 us per call.
FKV_DEV void after_previous() {
  griddep_wait();
  griddep_launch_dependents();
}

// The two chunks (indices of 8 elements) of unit u.
FKV_DEV void unit_chunks(int u, int rot, bool interleaved, int& a, int& b) {
  const int n = rot >> 4;  // turned units
  if (!interleaved && u < n) {
    a = u;
    b = u + n;
  } else {
    a = 2 * u;
    b = 2 * u + 1;
  }
}

FKV_DEV void unpack8(const uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = bf16x2_to_f2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

FKV_DEV uint4 pack8_bf16(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 values times inv, rounded to float32, as FP8 codes.
template <bool kE5>
FKV_DEV uint2 pack8_fp8(const float (&f)[8], float inv) {
  uint32_t o[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float y0 = __fmul_rn(f[4 * k], inv), y1 = __fmul_rn(f[4 * k + 1], inv);
    const float y2 = __fmul_rn(f[4 * k + 2], inv), y3 = __fmul_rn(f[4 * k + 3], inv);
    const uint32_t lo = kE5 ? f32x2_to_e5m2x2(y0, y1) : f32x2_to_e4m3x2(y0, y1);
    const uint32_t hi = kE5 ? f32x2_to_e5m2x2(y2, y3) : f32x2_to_e4m3x2(y2, y3);
    o[k] = lo | (hi << 16);
  }
  return make_uint2(o[0], o[1]);
}

FKV_DEV void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

FKV_DEV void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// Turn unit u (values a and b of its two chunks) by the table row at `cs`.
FKV_DEV void turn_unit(float (&a)[8], float (&b)[8], const float* cs, int rot, int u, bool interleaved) {
  float c[8], s[8];
  load8(cs + 8 * u, c);
  load8(cs + rot / 2 + 8 * u, s);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
      turn(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(a[i], b[i], c[i], s[i]);
  }
}

// ---------------------------------------------------------------- kv_rope_cache

constexpr int kRopeThreads = 256;

// Thread = one unit of one row (query heads, then K heads, then V heads), the same one of every
// token that it handles: the grid's active threads are a multiple (t_step) of a token's units, so
// that row and unit are found once and token t is followed by t + t_step.  HBM-bound: the next
// token's elements, slot and position are loaded before the current token is turned and stored, so
// that a thread has 32 bytes in flight all the time.  Three CTAs per SM (four spill registers, five more):
// 65,536 tokens of 32/8 heads at head_dim 128 take 255 us, 5.9 TB/s (280 and 321 us).
// kPool: 0 e4m3, 1 e5m2, 2 bf16.
template <int D, int kPool>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_cache_kernel(const RopeCacheParams p, int t_step) {
  after_previous();
  constexpr int U = D / 16;
  const int per_token = (p.Hq + 2 * p.H) * U;
  const long long gid = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  if (gid >= static_cast<long long>(per_token) * t_step) return;
  const int t0 = static_cast<int>(gid / per_token), rem = static_cast<int>(gid - static_cast<long long>(t0) * per_token);
  const int row = rem / U, u = rem % U;
  const bool is_q = row < p.Hq, is_v = row >= p.Hq + p.H;
  const int h = is_q ? row : (is_v ? row - p.Hq - p.H : row - p.Hq);
  const bool turned = !is_v && u < (p.rot >> 4);
  int ca, cb;
  unit_chunks(u, is_v ? 0 : p.rot, p.interleaved, ca, cb);
  const long long stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = (is_q ? p.q : is_v ? p.v : p.k) + h * D;
  uint8_t* pool = is_v ? p.vc : p.kc;
  const float inv = is_q || kPool == 2 ? 1.f : __frcp_rn((is_v ? p.vs : p.ks)[p.per_head ? h : 0]);
  uint4 xa, xb;
  long long slot, pos;
  auto fetch = [&](long long t) {
    const uint4* x = reinterpret_cast<const uint4*>(src + t * stride);
    xa = x[ca];
    xb = x[cb];
    slot = p.slots[t];
    pos = p.positions[t];
  };
  if (t0 < p.n_tokens) fetch(t0);
  for (long long t = t0; t < p.n_tokens; t += t_step) {
    float a[8], b[8];
    unpack8(xa, a);
    unpack8(xb, b);
    const long long s = slot, x = pos;
    if (t + t_step < p.n_tokens) fetch(t + t_step);
    if (s < 0) continue;
    if (s >= p.capacity || x < 0 || x >= p.max_pos) {
      if (rem == 0) raise_fault(p.fault, s >= p.capacity ? FKV_FAULT_SLOT : FKV_FAULT_POSITION);
      continue;
    }
    if (turned) turn_unit(a, b, p.cos_sin + x * p.rot, p.rot, u, p.interleaved);
    if (is_q) {
      uint4* dst = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + h * D);
      dst[ca] = pack8_bf16(a);
      dst[cb] = pack8_bf16(b);
    } else {
      // chunk index of the row's first 8 elements in the pool
      const long long at = ((((s >> 4) * p.H + h) << 4) + (s & 15)) * (D >> 3);
      if constexpr (kPool == 2) {
        reinterpret_cast<uint4*>(pool)[at + ca] = pack8_bf16(a);
        reinterpret_cast<uint4*>(pool)[at + cb] = pack8_bf16(b);
      } else {
        reinterpret_cast<uint2*>(pool)[at + ca] = pack8_fp8<kPool == 1>(a, inv);
        reinterpret_cast<uint2*>(pool)[at + cb] = pack8_fp8<kPool == 1>(b, inv);
      }
    }
  }
}

// ---------------------------------------------------------------- kv_block_cache

constexpr int kBlockThreads = 256;
// warps per (KV head, K or V) of a block, and how many of those a CTA takes
constexpr int block_warps(int D) { return D <= 128 ? 2 : 4; }
constexpr int block_tasks(int D) { return kBlockThreads / 32 / block_warps(D); }
constexpr int kQueryLoads = 4;
constexpr int kQueryItems = kQueryLoads * kBlockThreads;  // units of the query rows per CTA

// Four e4m3 codes times r, each product rounded to float32, as e4m3 codes.
FKV_DEV uint32_t rescale4(uint32_t w, float r) {
  uint32_t h01, h23;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"(static_cast<uint16_t>(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h23));
  return static_cast<uint32_t>(f32x2_to_e4m3x2(__fmul_rn(a.x, r), __fmul_rn(a.y, r))) |
         (static_cast<uint32_t>(f32x2_to_e4m3x2(__fmul_rn(b.x, r), __fmul_rn(b.y, r))) << 16);
}

// The smallest power of two s >= 2^-126 with amax <= 448 s, from amax's bits: 448 = 1.75 * 2^8.
FKV_DEV float pow2_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  const int k = e - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(k, -126) + 127) << 23);
}

// grid (pages of a sequence's new tokens, sequences, kv_parts + slices of the query rows).
// CTAs z < kv_parts: K and V of one block, two (head_dim 256: four) warps per (KV head, K or V), which
// share its 16 rows: the rows stay in registers between the maximum and the codes, so that each
// input byte is read once, and several warps keep them few enough for four CTAs per SM (at head_dim 64 and 128 with
// 44 bytes of spills; head_dim 256 has three).  The others turn
// query rows, four units per thread with all loads up front.  HBM-bound: 4 x 16,384 tokens of 32/8
// heads at head_dim 128 take 273 us, 5.5 TB/s (three CTAs per SM 289 us; six units per thread 323 us).
template <int D>
__global__ void __launch_bounds__(kBlockThreads, D <= 128 ? 4 : 3) block_cache_kernel(const BlockCacheParams p, int kv_parts) {
  constexpr int U = D / 16;       // units of a row
  constexpr int TP = 32 / U;      // rows that a warp handles at once
  constexpr int WT = block_warps(D);
  constexpr int R = 16 / WT / TP; // rounds
  __shared__ uint32_t amax_s[kBlockThreads / 32];
  after_previous();
  const int b = blockIdx.y;
  const int r0 = p.cu[b], L = p.cu[b + 1] - r0, T = p.ctx[b];
  const bool first = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0;
  if (L < 0 || L > p.max_q_len || r0 < 0 || r0 + static_cast<long long>(L) > p.n_tokens) {
    if (first) raise_fault(p.fault, FKV_FAULT_QLEN);
    return;
  }
  if (T < 0 || T > static_cast<long long>(p.max_blocks) * 16) {
    if (first) raise_fault(p.fault, FKV_FAULT_CONTEXT);
    return;
  }
  if (L > T) {
    if (first) raise_fault(p.fault, FKV_FAULT_QLEN);
    return;
  }
  if (p.cos_sin != nullptr && T > p.max_pos && L > 0) {
    if (first) raise_fault(p.fault, FKV_FAULT_POSITION);
    return;
  }
  const int page = ((T - L) >> 4) + blockIdx.x;
  if (L == 0 || page > (T - 1) >> 4) return;
  const int lo = max(T - L, page * 16), hi = min(T, page * 16 + 16);  // new positions in the page
  const long long row0 = static_cast<long long>(r0) - (T - L);        // row of position x: row0 + x

  if (static_cast<int>(blockIdx.z) >= kv_parts) {
    const int items = (hi - lo) * p.Hq * U;
    const int i0 = (blockIdx.z - kv_parts) * kQueryItems + threadIdx.x;
    if (i0 >= items) return;
    const int u = i0 % U;  // the same in every step: the CTA's threads are a multiple of U
    int ca, cb;
    unit_chunks(u, p.rot, p.interleaved, ca, cb);
    uint4 xa[kQueryLoads], xb[kQueryLoads];
    int pos[kQueryLoads], h[kQueryLoads];
#pragma unroll
    for (int j = 0; j < kQueryLoads; ++j) {
      const int i = i0 + j * kBlockThreads;
      const int th = i / U, tl = th / p.Hq;
      pos[j] = lo + tl;
      h[j] = th - tl * p.Hq;
      if (i < items) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (row0 + pos[j]) * p.q_stride + h[j] * D);
        xa[j] = src[ca];
        xb[j] = src[cb];
      }
    }
#pragma unroll
    for (int j = 0; j < kQueryLoads; ++j) {
      if (i0 + j * kBlockThreads >= items) break;
      float a[8], c[8];
      unpack8(xa[j], a);
      unpack8(xb[j], c);
      if (u < (p.rot >> 4)) turn_unit(a, c, p.cos_sin + static_cast<long long>(pos[j]) * p.rot, p.rot, u, p.interleaved);
      uint4* dst = reinterpret_cast<uint4*>(p.q_out + (row0 + pos[j]) * p.q_out_stride + h[j] * D);
      dst[ca] = pack8_bf16(a);
      dst[cb] = pack8_bf16(c);
    }
    return;
  }

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int task = blockIdx.z * block_tasks(D) + warp / WT, part = warp % WT;
  if (task >= 2 * p.H) return;  // all warps of the task
  const int g = task >> 1;
  const bool is_v = task & 1;
  const int u = lane % U, rot = is_v ? 0 : p.rot;
  const int slot0 = (16 / WT) * part + lane / U;  // this lane's row in round 0
  int ca, cb;
  unit_chunks(u, rot, p.interleaved, ca, cb);
  const __nv_bfloat16* src = is_v ? p.v : p.k;
  const long long stride = is_v ? p.v_stride : p.k_stride;
  uint4 xa[R], xb[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int pos = page * 16 + slot0 + r * TP;
    xa[r] = xb[r] = make_uint4(0u, 0u, 0u, 0u);
    if (pos >= lo && pos < hi) {
      const uint4* s = reinterpret_cast<const uint4*>(src + (row0 + pos) * stride + g * D);
      xa[r] = s[ca];
      xb[r] = s[cb];
    }
  }
  const int id = p.block_table[static_cast<size_t>(b) * p.max_blocks + page];
  if (id < 0 || id >= p.num_blocks) {
    if (threadIdx.x == 0) raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
    return;
  }
  float* scale = (is_v ? p.vs : p.ks) + static_cast<size_t>(id) * p.H + g;
  const int kept = lo - page * 16;  // slots that already hold tokens
  const float old = kept > 0 ? *scale : 0.f;
  float a[R][8], c[R][8];
  uint32_t amax = 0;  // bits of the largest finite magnitude (magnitudes order as their bits)
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int pos = page * 16 + slot0 + r * TP;
    unpack8(xa[r], a[r]);
    unpack8(xb[r], c[r]);
    if (u < (rot >> 4) && pos >= lo && pos < hi)
      turn_unit(a[r], c[r], p.cos_sin + static_cast<long long>(pos) * p.rot, p.rot, u, p.interleaved);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = __float_as_uint(a[r][i]) & 0x7FFFFFFFu, y = __float_as_uint(c[r][i]) & 0x7FFFFFFFu;
      if (x < 0x7F800000u) amax = max(amax, x);
      if (y < 0x7F800000u) amax = max(amax, y);
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (lane == 0) amax_s[warp] = amax;
  // the task's barrier; its warps have read the old scale before it is replaced below
  asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WT), "n"(32 * WT) : "memory");
#pragma unroll
  for (int w = 0; w < WT; ++w) amax = max(amax, amax_s[warp - part + w]);
  float s = pow2_scale(amax);
  uint8_t* block = (is_v ? p.vc : p.kc) + (static_cast<size_t>(id) * p.H + g) * 16 * D;
  if (kept > 0 && old >= 0.f && old <= 3.402823466e+38f) {  // (0 and subnormal numbers are below every s)
    if (old >= s) {
      s = old;
    } else {
      const float r = __fdiv_rn(old, s);
      for (int i = lane + 32 * part; i < kept * D / 16; i += 32 * WT) {
        uint4* q4 = reinterpret_cast<uint4*>(block) + i;
        uint4 w = *q4;
        w.x = rescale4(w.x, r);
        w.y = rescale4(w.y, r);
        w.z = rescale4(w.z, r);
        w.w = rescale4(w.w, r);
        *q4 = w;
      }
    }
  }
  if (lane == 0 && part == 0) *scale = s;
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int slot = slot0 + r * TP, pos = page * 16 + slot;
    if (pos >= lo && pos < hi) {
      uint2* dst = reinterpret_cast<uint2*>(block + slot * D);
      dst[ca] = pack8_fp8<false>(a[r], inv);
      dst[cb] = pack8_fp8<false>(c[r], inv);
    }
  }
}

template <int D>
cudaError_t launch_rope(const RopeCacheParams& p, int pool, int num_sms, cudaStream_t s) {
  const long long per_token = static_cast<long long>(p.Hq + 2 * p.H) * (D / 16);
  // as many tokens at once as three CTAs per SM hold
  const long long t_step = std::min<long long>(p.n_tokens, std::max<long long>(1, 3LL * num_sms * kRopeThreads / per_token));
  const unsigned blocks = static_cast<unsigned>((per_token * t_step + kRopeThreads - 1) / kRopeThreads);
  auto kern = pool == 2 ? rope_cache_kernel<D, 2> : pool == 1 ? rope_cache_kernel<D, 1> : rope_cache_kernel<D, 0>;
  return launch_dependent(kern, dim3(blocks), dim3(kRopeThreads), 0, s, p, static_cast<int>(t_step));
}

}  // namespace

cudaError_t launch_rope_cache(const RopeCacheParams& p, int pool, int num_sms, cudaStream_t s) {
  if (p.D == 64) return launch_rope<64>(p, pool, num_sms, s);
  if (p.D == 128) return launch_rope<128>(p, pool, num_sms, s);
  return launch_rope<256>(p, pool, num_sms, s);
}

cudaError_t launch_block_cache(const BlockCacheParams& p, int D, cudaStream_t s) {
  // pages that max_q_len tokens can touch, wherever the first of them lies in its block
  const unsigned pages = static_cast<unsigned>((static_cast<long long>(p.max_q_len) + 14) / 16 + 1);
  const long long items = static_cast<long long>(std::min(16, p.max_q_len)) * p.Hq * (D / 16);
  const int kv_parts = (2 * p.H + block_tasks(D) - 1) / block_tasks(D);
  const dim3 grid(pages, p.B, static_cast<unsigned>(kv_parts + (items + kQueryItems - 1) / kQueryItems));
  auto kern = D == 64 ? block_cache_kernel<64> : D == 128 ? block_cache_kernel<128> : block_cache_kernel<256>;
  return launch_dependent(kern, grid, dim3(kBlockThreads), 0, s, p, kv_parts);
}

}  // namespace fkv
