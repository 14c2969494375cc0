// Internal launcher interfaces between the C ABI (abi.cu) and the kernel files.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "../../include/fp8kv.h"

namespace fkv {

// Pool blocks per decode split, at most (the CUDA-core decode and the tensor-core decode at
// head_dim 128 and 256 stage a split's block ids in shared memory).
constexpr int kMaxSplitBlocks = 256;

struct DecodeParams {
  const __nv_bfloat16* q;      // [B][Hq][D]
  const uint8_t* k_cache;      // pool bytes
  const uint8_t* v_cache;
  const int32_t* block_table;  // [B][max_blocks]
  const int32_t* context_lens; // [B]
  const float* q_scale;
  const float* k_scale;
  const float* v_scale;
  int per_head;
  int B, Hq, Hkv, num_blocks, max_blocks;
  float sm_scale_log2;  // softmax_scale * log2(e)
  int window;
  int bps;              // blocks per split
  int max_splits;
  float* o_part;        // [B][Hq][max_splits][D]
  float* lse_part;      // [B][Hq][max_splits], base 2
  int32_t* done;        // [B][Hkv] splits finished (zeroed before the launch)
  __nv_bfloat16* out;   // [B][Hq][D]
  int32_t* fault;
  // the current token's K and V, bf16 [B][Hkv][D], quantised into the (e4m3) pools at
  // position T - 1 by the launch itself (fp8_decode_step); null: the pools are complete
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  // wall-clock bound of the tensor-core decode's pipeline waits (ns); the waits that let
  // issued copies and products drain before the CTA exits keep their own bound
  uint64_t pipe_wait_ns;
};

struct PrefillParams {
  const __nv_bfloat16* q;       // [total_q][Hq][D]
  const int32_t* cu_q;          // [B + 1]
  const int32_t* block_table;   // [B][max_blocks]
  const int32_t* context_lens;  // [B]
  const float* q_scale;
  const float* k_scale;
  const float* v_scale;
  int per_head;
  int B, Hq, Hkv, num_blocks, max_blocks, n_qtiles;
  float sm_scale_log2;
  int causal;
  int promote_every;            // 1: every tile; N >= 2: every N tiles; 0: never
  int window;                   // 0 = full, else the last `window` keys of each query
  __nv_bfloat16* out;           // [total_q][Hq][D]
  int32_t* fault;
};

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

cudaError_t launch_prefill(const PrefillParams& p, int D, bool bf16_layer, void* k_cache, void* v_cache,
                           cudaStream_t s);

// Launch `kern` with programmatic stream serialisation (the kernel must call griddep_wait
// before touching global memory that earlier kernels produce or consume).
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                             Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

cudaError_t launch_kv_quant_cache(const void* k, const void* v, const int64_t* slots, int n_tokens,
                                  const fkv_layer_cache& cache, const float* ks, const float* vs,
                                  int per_head, bool bf16_layer, int32_t* fault, cudaStream_t s,
                                  int num_sms, unsigned long long* clips);

// elt: the pool's element type, 1 e4m3, 2 bf16, 3 e5m2
cudaError_t launch_decode(const DecodeParams& p, int D, int elt, int G, cudaStream_t s);

// e4m3 layers (elt 1, head_dim 64 / 128 / 256) decode on the tensor cores (FP8 P, 128-key
// tiles); bf16 and e5m2 layers on the CUDA cores (P exact).
bool decode_uses_tensor_cores(int D, int elt);
cudaError_t launch_decode_tc(const DecodeParams& p, int D, int G, cudaStream_t s);

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

// Supplies the decode's workspace of `need` bytes when the caller passes none: sets *ws
// (256-byte aligned) and *bytes, with its first `counter_bytes` (the split counters) zero
// by the time work enqueued afterwards on `stream` runs, or returns the status the entry
// point then returns.
using ScratchProvider = fkv_status (*)(size_t need, size_t counter_bytes, cudaStream_t stream, void** ws,
                                       size_t* bytes);

// The whole of fp8_decode_attn (k_new = v_new = NULL) and fp8_decode_step: argument
// checks, the split-K plan, then the launch.  With scratch non-null the workspace comes
// from it, after every check (fp8_decode_attn_noalloc).
fkv_status decode_entry(const void* k_new, const void* v_new, const void* q, int32_t batch, int32_t num_q_heads,
                        fkv_layer_cache cache, const int32_t* block_table, int32_t max_blocks,
                        const int32_t* context_lens, const float* q_scale, const float* k_scale,
                        const float* v_scale, fkv_scale_gran gran, float softmax_scale, int32_t window,
                        int32_t layer, const uint8_t* skip_layer_mask, int32_t num_layers, void* out,
                        void* workspace, size_t workspace_bytes, ScratchProvider scratch, int32_t num_splits,
                        int32_t* fault, fkv_stream_t stream);

}  // namespace fkv
