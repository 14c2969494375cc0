// Parameters and launches of the rotary cache writes and of the block-scaled cache's append and attention,
// and what their kernels share.  (Apart from kernels.h and common.cuh, so that the recorded profiles of the other
// kernels stay those of their source.)
#pragma once
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace fkv {

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

struct RopeCacheParams {
  const __nv_bfloat16 *q, *k, *v;             // token rows at the strides (in elements)
  long long q_stride, k_stride, v_stride;
  __nv_bfloat16* q_out;
  long long q_out_stride;
  const float* cos_sin;                       // [max_pos][rot]
  int max_pos, rot;
  int interleaved;
  const int64_t* positions;                   // [n_tokens]
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
  const int32_t* cu;                          // [B + 1]
  const int32_t* ctx;                         // [B]
  const int32_t* block_table;                 // [B][max_blocks]
  int n_tokens, B, max_q_len, Hq, H, num_blocks, max_blocks;
  uint8_t *kc, *vc;
  float *ks, *vs;                             // [num_blocks][H]
  int32_t* fault;
};

cudaError_t launch_block_cache(const BlockCacheParams& p, int D, cudaStream_t s);

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
  int head_parts, part_heads;                 // set by the launch: a group in parts of part_heads heads
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
  int32_t* done;                              // [B * Hkv] pieces finished, zero between calls
  float* lse_part;                            // [N + B * Hkv][G], base 2
  float* o_part;                              // [N + B * Hkv][G][D]
  __nv_bfloat16* out;                         // [B][Hq][D]
  int32_t* fault;
};

// CTAs of the block-scaled decode that an SM holds, pool blocks of its tiles, and its launch on N CTAs.
int block_decode_ctas_per_sm(int D);
int block_decode_tile_blocks(int D);
cudaError_t launch_block_decode(const BlockDecodeParams& p, int D, int N, cudaStream_t s);

}  // namespace fkv
