// The rotary cache writes and the block-scaled cache's append and attention: their parameters and launches, and
// what their kernels share.
#pragma once
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace fkv {

// ex2 whose results below 2^-126 are not flushed.
FKV_DEV float ex2_subnormal(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four float32 values -> four e4m3 codes in a word, a's first, in one statement: joined from two
// 16-bit results in C++, the halves are widened, shifted and merged instead.
FKV_DEV uint32_t f32x4_to_e4m3x4(float2 a, float2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// The smallest power of two s >= 2^-126 with amax <= 448 s, from amax's bits: 448 = 1.75 * 2^8.
FKV_DEV float pow2_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  const int k = e - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(k, -126) + 127) << 23);
}

// A query row enters the products scaled by 2^-k, its largest magnitude (float32 bits `amax`, finite) in (224, 448], as
// two e4m3 terms.
FKV_DEV int query_exponent(uint32_t amax) {
  return max(static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);  // 448 = 1.75 * 2^8
}

// Four scaled query elements as two terms: hi the nearest code, lo that of what hi leaves.  A bf16 element
// has 8 significant bits, 4 of them (the nearest, so that the rest has at most 4) in hi: exact down to 1/4, below that
// within 2^-10, half a step of e4m3's subnormals, which is less than 2^-17 of the row's largest element.
FKV_DEV void split4_query(float2 a, float2 b, uint32_t& hi, uint32_t& lo) {
  hi = f32x4_to_e4m3x4(a, b);
  uint32_t h01, h23;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"(static_cast<uint16_t>(hi & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"(static_cast<uint16_t>(hi >> 16)));
  const float2 ha = __half22float2(*reinterpret_cast<const __half2*>(&h01));
  const float2 hb = __half22float2(*reinterpret_cast<const __half2*>(&h23));
  lo = f32x4_to_e4m3x4(make_float2(a.x - ha.x, a.y - ha.y), make_float2(b.x - hb.x, b.y - hb.y));
}

// Four values of P as two e4m3 terms: `hi` the leading 3 fraction bits, `lo` the rest.  kPacked: two values per
// instruction, for values that lie in pairs; where they do not, the pairs cost moves (the decode at head_dim 64:
// 60 us against 56 for 8 x 8k-32k, 64/8 heads).
template <bool kPacked>
FKV_DEV void split4(float2 a, float2 b, uint32_t& hi, uint32_t& lo) {
  auto lead = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFF00000u); };
  const float2 ha = make_float2(lead(a.x), lead(a.y)), hb = make_float2(lead(b.x), lead(b.y));
  float2 la, lb;
  if constexpr (kPacked) {
    const float2 neg = make_float2(-1.f, -1.f);
    la = __ffma2_rn(ha, neg, a);
    lb = __ffma2_rn(hb, neg, b);
  } else {
    la = make_float2(a.x - ha.x, a.y - ha.y);
    lb = make_float2(b.x - hb.x, b.y - hb.y);
  }
  hi = f32x4_to_e4m3x4(ha, hb);
  lo = f32x4_to_e4m3x4(la, lb);
}

// 2^n of a whole number -126 <= n <= 127.
FKV_DEV float pow2i(float n) { return __uint_as_float(static_cast<uint32_t>(static_cast<int>(n) + 127) << 23); }

// V scales in the exponent.  P_j = 2^(x_j + L_j - R) carries its block's scale vs = 2^L; the softmax's sum takes
// it out again, l = sum P_j 2^(o - L_j).  A scale 2^100 and more below the largest of its tile, zero among them,
// counts as zero: its keys enter l as if it were 2^-100 of the largest, so that their P stays a normal
// float32 number, and are left out of the product (their factor is given as -2^(o - L)).  The whole number o keeps
// l within float32: its factors are at most 2^80 for L >= o - 80, its largest term is above 2^-120 for L <= o + 118.
// It begins at 0, which serves scales from 2^-80 to 2^118, and follows smaller ones down and larger ones up (of
// scales 2^198 and more apart in one sequence the small ones count as zero as well).
struct ScaleRange {
  float o = 0.f, top = -INFINITY, low = INFINITY;  // the offset, the largest and the smallest L so far
};
struct BlockScale {
  float lv, iv;  // L and 2^(o - L), the latter negative where the scale counts as zero
  // Not as a rule: o changed, a scale counts as zero, or the scales so far lie so far apart that 2^-|r - R_t| may
  // underflow though the keys' weights are alike: the sums are joined by rare_factors.
  bool rare;
  float change;  // new o - old o
};

// A tile's scales, a block per lane (`in`: the lane has one that a query sees).  Every lane of the warp takes part.
FKV_DEV BlockScale block_scales(ScaleRange& range, float vs, bool in) {
  const bool some = in && vs > 0.f;
  const float L = some ? lg2(vs) : 0.f;
  float least, most;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(most) : "f"(some ? L : -INFINITY));
  const float bottom = most > -INFINITY ? most - 100.f : -100.f;
  bool zero = in && !(some && L > bottom);
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(least) : "f"(zero ? bottom : some ? L : INFINITY));
  range.top = fmaxf(range.top, most);
  range.low = fminf(range.low, least);
  const float o = fmaxf(fmaxf(fminf(range.o, floorf(least) + 80.f), ceilf(range.top) - 118.f), -120.f);
  zero = zero || (some && L < o - 80.f);
  BlockScale r;
  r.rare = __any_sync(0xffffffffu, zero) || o != range.o || range.top - range.low > 100.f;
  r.change = o - range.o;
  range.o = o;
  r.lv = zero ? fmaxf(bottom, o - 80.f) : L;
  r.iv = in ? ex2_subnormal(o - r.lv) : 1.f;
  if (zero) r.iv = -r.iv;
  return r;
}

// A row's state (r, l) joined by a rare tile's (R, lt), and the factors of acc and O_t.  Where o went down by n, l goes
// with it; where it went up, r does instead, and l, whose keys may be worth 2^-198 of the new ones, stays
// what it is (acc loses what is worth nothing beside them).  2^-|r - R| enters l in three equal factors: scales at the
// two ends of float32 make it 2^-254 and less where the keys' weights are alike.
struct RareFactors {
  float l, lt;          // l and lt are to be multiplied by these three times
  float alpha, beta;    // of acc and O_t
};
FKV_DEV RareFactors rare_factors(float& r, float& l, float R, float change) {
  const float up = r + fmaxf(change, 0.f), next = fmaxf(up, R);
  l *= ex2(fminf(change, 0.f));
  RareFactors f;
  f.l = ex2(0.33333334f * (up - next));
  f.lt = ex2(0.33333334f * (R - next));
  f.alpha = ex2(r - next);
  f.beta = ex2(R - next);
  r = next;
  return f;
}

// The axes of a head's pairs, two bits each, and the positions' strides; count 0: one position per token, or
// (kv_block_cache) the token's place.
struct PairAxes {
  int count;
  long long stride;                           // between the axes' positions
  uint32_t axis[8];                           // pair i: bits 2 i % 32 of word i / 16
};

struct RopeCacheParams {
  const __nv_bfloat16 *q, *k, *v;             // token rows at the strides (in elements)
  long long q_stride, k_stride, v_stride;
  __nv_bfloat16* q_out;
  long long q_out_stride;
  const float* cos_sin;                       // [max_pos][rot]
  int max_pos, rot;
  int interleaved;
  PairAxes axes;
  const int64_t* positions;                   // [n_tokens], of axis a at a * axes.stride
  const int64_t* slots;                       // [n_tokens]
  int n_tokens, Hq, H, D;                     // Hq 0: no queries
  uint8_t *kc, *vc;
  long long capacity;                         // slots of the pool
  const float *ks, *vs;
  int per_head;
  int32_t* fault;
};

// pool: 0 e4m3, 1 e5m2, 2 bf16
cudaError_t launch_rope_cache(const RopeCacheParams& p, int pool, int num_sms, cudaStream_t s);

struct BlockCacheParams {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  __nv_bfloat16* q_out;
  long long q_out_stride;
  const float* cos_sin;                       // null: no rotation (rot 0)
  int max_pos, rot;
  int interleaved;
  PairAxes axes;
  const int64_t* positions;                   // null: the tokens' places
  const int32_t* cu;                          // [B + 1]
  const int32_t* ctx;                         // [B]
  const int32_t* block_table;                 // [B][max_blocks]
  int n_tokens, B, max_q_len, Hq, H, num_blocks, max_blocks;
  uint8_t *kc, *vc;
  float *ks, *vs;                             // [num_blocks][H]
  int32_t* fault;
};

cudaError_t launch_block_cache(const BlockCacheParams& p, int D, cudaStream_t s);

struct EvictParams {
  uint8_t *kc, *vc;
  float *ks, *vs;                             // [num_blocks][H]
  int B, H, num_blocks, max_blocks, new_max_blocks;
  const int32_t* block_table;                 // [B][max_blocks]
  const int32_t* ctx;                         // [B]
  const float* weights;                       // [B][H][weights_len]
  int weights_len, new_weights_len;
  int budget, sink, recent;
  const int32_t* new_table;                   // [B][new_max_blocks]
  int32_t* new_lens;                          // [B]
  int32_t* kept;                              // [B][H][budget]
  float* new_weights;                         // [B][H][new_weights_len] or null
  int32_t* fault;
};

cudaError_t launch_block_evict(const EvictParams& p, int D, int num_sms, cudaStream_t s);

struct BlockWeightsParams {
  const __nv_bfloat16* q;                     // [total_q][Hq][D]
  const uint8_t* k_cache;
  const float* k_scale;                       // [num_blocks][Hkv]
  const int32_t* block_table;                 // [B][max_blocks]
  const int32_t* ctx;                         // [B]
  const int32_t* cu;                          // [B + 1]
  int B, Hq, Hkv, num_blocks, max_blocks, max_q_len, total_q;
  float sm_scale_log2;                        // softmax_scale * log2(e)
  float decay;
  float* weights;                             // [B][Hkv][weights_len]
  int weights_len;
  int32_t* fault;
  uint64_t stage_wait_ns;                     // bound of the copies' wait for a free stage (the others': kPipeWaitNs)
  // the workspace's parts (block_weights.cu), set by the launch
  int slots;                                  // CTAs of a launch, at most
  int32_t* done;                              // [2][slots] pieces finished of the unit that CTA k begins, in either pass
  float2* pieces;                             // [2 slots (+ units)][rows] maxima and sums
  float* sums;                                // [2 slots][256]
  float* rows;                                // [tiles][64]{c, c, -lse, -lse}
  uint8_t* q_tiles;                           // [tiles] of both terms
  int2* units;                                // [B][Hkv]{first CTA, pieces}
  float* scores;                              // [B][Hkv][16 max_blocks][rows]
};

size_t block_weights_workspace(int B, int total_q, int max_q_len, int Hq, int Hkv, int D, long long keys, int num_sms);
cudaError_t launch_block_weights(BlockWeightsParams p, int D, void* workspace, int num_sms, cudaStream_t s);

struct BlockPrefillParams {
  const __nv_bfloat16* q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;             // [num_blocks][Hkv]
  const int32_t* block_table;                 // [B][max_blocks]
  const int32_t* ctx;                         // [B]
  const int32_t* cu;                          // [B + 1]
  int B, Hq, Hkv, num_blocks, max_blocks, max_q_len, total_q;
  float sm_scale_log2;                        // softmax_scale * log2(e)
  int causal, window;
  __nv_bfloat16* out;
  int32_t* fault;
  uint64_t stage_wait_ns;                     // bound of the copies' wait for a free stage (the others': kPipeWaitNs)
  int head_parts, part_heads, part_tokens;    // set by the launch: a group in parts of part_heads heads, a CTA's tokens;
  int even_waves;                             // clusters are there to even out the last wave
};

cudaError_t launch_block_prefill(BlockPrefillParams p, int D, int num_sms, cudaStream_t s);

struct BlockDecodeParams {
  const __nv_bfloat16* q;                     // [B][Hq][D]
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;             // [num_blocks][Hkv >> halves]
  const int32_t* block_table;                 // [B][max_blocks]
  const int32_t* ctx;                         // [B]
  int B, Hq, Hkv, num_blocks, max_blocks;     // Hkv: units of a sequence, Hq / Hkv query heads each
  int halves;                                 // 1: units 2 g and 2 g + 1 share KV head g
  float sm_scale_log2;                        // softmax_scale * log2(e)
  int window;
  int32_t* done;                              // [N] pieces finished of the unit that CTA k begins, zero between calls
  float* lse_part;                            // [N + B * Hkv][G], base 2
  float* o_part;                              // [N + B * Hkv][G][D]
  __nv_bfloat16* out;                         // [B][Hq][D]
  int32_t* fault;
  uint64_t stage_wait_ns;                     // bound of the copies' wait for a free stage (the others': kPipeWaitNs)
  // what sequences share (block_shared.cu)
  const int4* shared;                         // [B]{shared keys, first piece's CTA, pieces per item, place in the group}
  int2* units;                                // [B * Hkv]{first CTA, pieces}
};

// CTAs of the block-scaled decode that an SM holds, pool blocks of its tiles, and its launch on N CTAs.
int block_decode_ctas_per_sm(int D);
int block_decode_tile_blocks(int D);
cudaError_t launch_block_decode(const BlockDecodeParams& p, int D, int N, cudaStream_t s);

}  // namespace fkv
