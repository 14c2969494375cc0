// The C ABI of libfp8kv.so: argument validation, launch planning and dispatch.
// Nothing here allocates memory or keeps state between calls.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "block_common.cuh"
#include "block_shared.cuh"

namespace {

using fkv::DecodeParams;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether arrays of that many 4-byte elements have one in common.
bool overlap(const void* a, uint64_t an, const void* b, uint64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * bn && y < x + 4 * an;
}

int current_num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();  // no device: plan for a full GB300
    n = 152;
  }
  return n;
}

bool layer_is_bf16(int32_t layer, const uint8_t* mask, int32_t num_layers, fkv_status* st) {
  if (mask == nullptr) return false;
  if (layer < 0 || layer >= num_layers) {
    *st = FKV_INVALID_ARG;
    return false;
  }
  return mask[layer] != 0;
}

bool supported_head_dim(int32_t d) { return d == 64 || d == 128 || d == 256; }

bool valid_format(const fkv_layer_cache& c) { return c.kv_format == FKV_KV_E4M3 || c.kv_format == FKV_KV_E5M2; }

// Element type of a layer's pools for the decode kernels: 1 e4m3, 2 bf16, 3 e5m2.
int layer_elt(bool bf16, const fkv_layer_cache& c) { return bf16 ? 2 : (c.kv_format == FKV_KV_E5M2 ? 3 : 1); }

bool supported_group(int32_t G, int32_t D) {
  if (!(G == 1 || G == 2 || G == 4 || G == 8 || G == 16)) return false;
  return G * D <= 2048;
}

// Pool blocks per tile of the tensor-core decode (its P-rounding granularity): 128 keys,
// 256 at head_dim 64.  The split plan keeps whole tiles for every layer kind.
int decode_tile_blocks(int32_t D) { return D == 64 ? 16 : 8; }

struct DecodePlan {
  int bps = 0;
  int max_splits = 0;
  size_t o_bytes = 0, lse_bytes = 0, cnt_bytes = 0;
};

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Split-K plan.  Blocks per split (bps) are multiples of the tensor-core decode's tile (8
// blocks of 16 keys; 16 at head_dim 64) up to kMaxSplitBlocks (256), with at most 1024
// splits per sequence.
// Equal estimates go to the longer splits (fewer CTAs, fewer prologues and merges).  A requested
// num_splits sets bps = ceil(blocks / num_splits), rounded up.  Otherwise bps minimises
// the estimated time waves * bps, where a wave is one CTA on every resident slot
// (3 per SM) and the grid has B * Hkv * ceil(blocks / bps) CTAs: the longest split
// sets a wave's time, and a partly filled last wave costs as much as a full one.
bool plan_decode(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_blocks, int32_t window,
                 int32_t num_splits, DecodePlan* plan) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || max_blocks <= 0 || window < 0 || num_splits < 0) return false;
  long long nblk_max = max_blocks;
  if (window > 0) nblk_max = std::min<long long>(max_blocks, (window + 15) / 16 + 1);
  const long long tpb = decode_tile_blocks(D);
  long long bps;
  if (num_splits > 0) {
    bps = (nblk_max + num_splits - 1) / num_splits;
  } else {
    const long long units = static_cast<long long>(std::max(B, 1)) * Hkv;
    const long long slots = static_cast<long long>(current_num_sms()) * 3;
    long long best = -1, best_cost = 0;
    for (long long c = tpb; c <= fkv::kMaxSplitBlocks; c += tpb) {
      const long long ctas = units * ((nblk_max + c - 1) / c);
      const long long cost = (ctas + slots - 1) / slots * std::min(c, nblk_max);
      if (best < 0 || cost < best_cost || (cost == best_cost && c > best)) {
        best = c;
        best_cost = cost;
      }
    }
    bps = best;
  }
  bps = std::min<long long>(bps, fkv::kMaxSplitBlocks);
  bps = std::max<long long>(bps, (nblk_max + 1023) / 1024);
  bps = std::max<long long>(bps, 1);
  bps = (bps + tpb - 1) / tpb * tpb;
  if (bps > fkv::kMaxSplitBlocks) return false;  // context too long for 1024 splits of 256 blocks
  plan->bps = static_cast<int>(bps);
  plan->max_splits = static_cast<int>((nblk_max + bps - 1) / bps);
  const size_t rows = static_cast<size_t>(B) * Hq * plan->max_splits;
  plan->o_bytes = align256(rows * D * sizeof(float));
  plan->lse_bytes = align256(rows * sizeof(float));
  plan->cnt_bytes = align256(static_cast<size_t>(std::max(B, 1)) * Hkv * sizeof(int32_t));
  return true;
}

fkv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FKV_OK : FKV_CUDA_ERROR; }

// Bound of the pipeline waits of the tensor-core decode, and of the copies' waits of the block-scaled attention,
// set by fkv_set_decode_wait_limit_ns; 0 = the default (kPipeWaitNs).
std::atomic<unsigned long long> g_decode_wait_ns{0};
constexpr unsigned long long kDefaultPipeWaitNs = 200000000ull;  // 200 ms, as kPipeWaitNs in tc.cuh

unsigned long long pipe_wait_ns() {
  const unsigned long long ns = g_decode_wait_ns.load(std::memory_order_relaxed);
  return ns != 0 ? ns : kDefaultPipeWaitNs;
}

fkv_status cache_write(const void* k, const void* v, const int64_t* slot_mapping, int32_t n_tokens,
                       fkv_layer_cache cache, const float* k_scale, const float* v_scale, fkv_scale_gran gran,
                       int32_t layer, const uint8_t* skip_layer_mask, int32_t num_layers, int32_t* fault,
                       fkv_stream_t stream, unsigned long long* clips) {
  if (n_tokens < 0) return FKV_INVALID_ARG;
  if (cache.block_size != 16) return cache.block_size > 0 ? FKV_UNSUPPORTED : FKV_INVALID_ARG;
  if (cache.num_blocks <= 0 || cache.num_kv_heads <= 0 || !valid_format(cache)) return FKV_INVALID_ARG;
  if (!supported_head_dim(cache.head_dim)) return FKV_UNSUPPORTED;
  if (gran != FKV_SCALE_PER_TENSOR && gran != FKV_SCALE_PER_HEAD) return FKV_INVALID_ARG;
  fkv_status st = FKV_OK;
  const bool bf16 = layer_is_bf16(layer, skip_layer_mask, num_layers, &st);
  if (st != FKV_OK) return st;
  if (n_tokens == 0) return FKV_OK;
  if (!k || !v || !slot_mapping || !cache.k_cache || !cache.v_cache) return FKV_INVALID_ARG;
  if (!bf16 && (!k_scale || !v_scale)) return FKV_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache.k_cache, 16) || !aligned(cache.v_cache, 16) ||
      !aligned(slot_mapping, 8) || !aligned(clips, 8))
    return FKV_INVALID_ARG;
  return from_cuda(fkv::launch_kv_quant_cache(k, v, slot_mapping, n_tokens, cache, k_scale, v_scale,
                                              gran == FKV_SCALE_PER_HEAD, bf16, fault,
                                              reinterpret_cast<cudaStream_t>(stream), current_num_sms(), clips));
}

// ---- the rotary cache writes and the block-scaled cache

// A rotation of heads of head_dim elements.
fkv_status check_rope(const fkv_rope& r, int32_t head_dim) {
  if (!r.cos_sin || !aligned(r.cos_sin, 16) || r.max_positions <= 0 || r.rot_dim <= 0) return FKV_INVALID_ARG;
  if (r.rot_dim > head_dim) return FKV_INVALID_ARG;
  return r.rot_dim % 16 == 0 ? FKV_OK : FKV_UNSUPPORTED;
}

// Rows of `row` consecutive bf16 elements at `stride` elements.
bool valid_rows(const void* p, int64_t stride, int64_t row) {
  return p != nullptr && aligned(p, 16) && stride >= row && stride % 8 == 0;
}

fkv_status check_block_cache(const fkv_block_cache& c) {
  if (c.block_size != 16) return c.block_size > 0 ? FKV_UNSUPPORTED : FKV_INVALID_ARG;
  if (c.num_blocks <= 0 || c.num_kv_heads <= 0) return FKV_INVALID_ARG;
  return supported_head_dim(c.head_dim) ? FKV_OK : FKV_UNSUPPORTED;
}

bool valid_block_pools(const fkv_block_cache& c) {
  return c.k_cache && c.v_cache && c.k_scale && c.v_scale && aligned(c.k_cache, 16) && aligned(c.v_cache, 16) &&
         aligned(c.k_scale, 4) && aligned(c.v_scale, 4);
}

// Columns of a block table whose positions (and a tile more) the kernels count in 32 bits.
constexpr int32_t kMaxTableBlocks = (1 << 27) - 64;

// Rows (tokens times heads of a group) of an attention weights call that the kernels count in 32 bits, and their tiles' grid.
constexpr long long kMaxWeightRows = 1LL << 30;

// The block-scaled decode: CTAs resident at once, of which a unit (sequence, KV head) is given at
// most 160 (the merge of its pieces grows with them: 0.05 us each, a tile of its own 1.5 us), and the
// workspace: piece counters, the pieces' log-sum-exps and outputs.
struct BlockDecodePlan {
  long long ctas = 0;
  int halves = 0;  // 1: a group of 16 heads is two units of 8
  size_t cnt_bytes = 0, lse_bytes = 0, o_bytes = 0;
};

// Piece counters, one per CTA: a unit of several pieces counts at the CTA of its first, which can be that of
// one such unit only.  Their number is the same for every call, so that the scratch of one never lies
// where another counts.
constexpr long long kBlockDecodeCounters = 16384;

BlockDecodePlan plan_block_decode(int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
  BlockDecodePlan plan;
  plan.halves = Hq / Hkv == 16 ? 1 : 0;
  const int G = (Hq / Hkv) >> plan.halves;
  const long long units = static_cast<long long>(B) * Hkv << plan.halves;
  plan.ctas = std::min({static_cast<long long>(current_num_sms()) * fkv::block_decode_ctas_per_sm(D), 160 * units, kBlockDecodeCounters});
  const size_t rows = static_cast<size_t>(plan.ctas + units) * G;
  plan.cnt_bytes = kBlockDecodeCounters * sizeof(int32_t);
  plan.lse_bytes = align256(rows * sizeof(float));
  plan.o_bytes = rows * D * sizeof(float);
  return plan;
}

// The axes of the pairs in the kernels' form; false if there are none such.
bool pair_axes(const fkv_axes& a, int32_t rot_dim, fkv::PairAxes* out) {
  if (a.num_axes < 1 || a.num_axes > 4 || a.axis_stride < 0) return false;
  out->count = a.num_axes;
  out->stride = a.axis_stride;
  for (int32_t i = 0; a.pair_axis && i < rot_dim / 2; ++i) {
    if (a.pair_axis[i] >= a.num_axes) return false;
    out->axis[i / 16] |= static_cast<uint32_t>(a.pair_axis[i]) << (2 * (i % 16));
  }
  return true;
}

fkv_status rope_cache_entry(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride, const fkv_axes& axes,
                         const int64_t* slot_mapping, int32_t n_tokens, fkv_rope rope, fkv_layer_cache cache,
                         const float* k_scale, const float* v_scale, fkv_scale_gran gran, int32_t layer,
                         const uint8_t* skip_layer_mask, int32_t num_layers, int32_t* fault, fkv_stream_t stream) {
  if (n_tokens < 0 || num_q_heads < 0) return FKV_INVALID_ARG;
  if (cache.block_size != 16) return cache.block_size > 0 ? FKV_UNSUPPORTED : FKV_INVALID_ARG;
  if (cache.num_blocks <= 0 || cache.num_kv_heads <= 0 || !valid_format(cache)) return FKV_INVALID_ARG;
  if (!supported_head_dim(cache.head_dim)) return FKV_UNSUPPORTED;
  if (num_q_heads > 8192 || cache.num_kv_heads > 8192) return FKV_UNSUPPORTED;
  if (gran != FKV_SCALE_PER_TENSOR && gran != FKV_SCALE_PER_HEAD) return FKV_INVALID_ARG;
  fkv_status st = FKV_OK;
  const bool bf16 = layer_is_bf16(layer, skip_layer_mask, num_layers, &st);
  if (st != FKV_OK) return st;
  st = check_rope(rope, cache.head_dim);
  if (st != FKV_OK) return st;
  fkv::RopeCacheParams p;
  std::memset(&p, 0, sizeof(p));
  if (!pair_axes(axes, rope.rot_dim, &p.axes)) return FKV_INVALID_ARG;
  if (n_tokens == 0) return FKV_OK;
  if ((q != nullptr) != (num_q_heads > 0) || (q_out != nullptr) != (num_q_heads > 0)) return FKV_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * cache.head_dim;
  const int64_t kv_row = static_cast<int64_t>(cache.num_kv_heads) * cache.head_dim;
  if (!valid_rows(k, k_stride, kv_row) || !valid_rows(v, v_stride, kv_row)) return FKV_INVALID_ARG;
  if (q && (!valid_rows(q, q_stride, q_row) || !valid_rows(q_out, q_out_stride, q_row))) return FKV_INVALID_ARG;
  if (q && q == q_out && q_stride != q_out_stride) return FKV_INVALID_ARG;
  if (!axes.positions || !slot_mapping || !aligned(axes.positions, 8) || !aligned(slot_mapping, 8)) return FKV_INVALID_ARG;
  if (!cache.k_cache || !cache.v_cache || !aligned(cache.k_cache, 16) || !aligned(cache.v_cache, 16))
    return FKV_INVALID_ARG;
  if (!bf16 && (!k_scale || !v_scale)) return FKV_INVALID_ARG;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_out_stride = q_out_stride;
  p.cos_sin = rope.cos_sin;
  p.max_pos = rope.max_positions;
  p.rot = rope.rot_dim;
  p.interleaved = rope.interleaved != 0;
  p.positions = axes.positions;
  p.slots = slot_mapping;
  p.n_tokens = n_tokens;
  p.Hq = num_q_heads;
  p.H = cache.num_kv_heads;
  p.D = cache.head_dim;
  p.kc = static_cast<uint8_t*>(cache.k_cache);
  p.vc = static_cast<uint8_t*>(cache.v_cache);
  p.capacity = static_cast<long long>(cache.num_blocks) * 16;
  p.ks = k_scale;
  p.vs = v_scale;
  p.per_head = gran == FKV_SCALE_PER_HEAD;
  p.fault = fault;
  const int pool = bf16 ? 2 : cache.kv_format == FKV_KV_E5M2 ? 1 : 0;
  return from_cuda(fkv::launch_rope_cache(p, pool, current_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

fkv_status block_cache_entry(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride, int32_t n_tokens,
                          const fkv_axes* axes, const int32_t* cu_seqlens, int32_t batch, int32_t max_q_len, fkv_rope rope,
                          fkv_block_cache cache, const int32_t* block_table, int32_t max_blocks,
                          const int32_t* context_lens, int32_t* fault, fkv_stream_t stream) {
  if (n_tokens < 0 || batch < 0 || max_q_len < 0 || max_blocks <= 0 || num_q_heads < 0) return FKV_INVALID_ARG;
  fkv_status st = check_block_cache(cache);
  if (st != FKV_OK) return st;
  if (batch > 65535 || num_q_heads > 8192 || cache.num_kv_heads > 8192 || max_blocks > kMaxTableBlocks) return FKV_UNSUPPORTED;
  const bool turned = rope.cos_sin != nullptr;
  if (turned) {
    st = check_rope(rope, cache.head_dim);
    if (st != FKV_OK) return st;
  } else if (num_q_heads > 0 || rope.rot_dim != 0) {
    return FKV_INVALID_ARG;
  }
  fkv::BlockCacheParams p;
  std::memset(&p, 0, sizeof(p));
  if (axes && (!turned || !pair_axes(*axes, rope.rot_dim, &p.axes))) return FKV_INVALID_ARG;
  if (n_tokens == 0 || batch == 0 || max_q_len == 0) return FKV_OK;
  if (axes && (!axes->positions || !aligned(axes->positions, 8))) return FKV_INVALID_ARG;
  if ((q != nullptr) != (num_q_heads > 0) || (q_out != nullptr) != (num_q_heads > 0)) return FKV_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * cache.head_dim;
  const int64_t kv_row = static_cast<int64_t>(cache.num_kv_heads) * cache.head_dim;
  if (!valid_rows(k, k_stride, kv_row) || !valid_rows(v, v_stride, kv_row)) return FKV_INVALID_ARG;
  if (q && (!valid_rows(q, q_stride, q_row) || !valid_rows(q_out, q_out_stride, q_row))) return FKV_INVALID_ARG;
  if (q && q == q_out && q_stride != q_out_stride) return FKV_INVALID_ARG;
  if (!valid_block_pools(cache)) return FKV_INVALID_ARG;
  if (!cu_seqlens || !block_table || !context_lens || !aligned(cu_seqlens, 4) || !aligned(block_table, 4) ||
      !aligned(context_lens, 4))
    return FKV_INVALID_ARG;
  p.positions = axes ? axes->positions : nullptr;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q_out_stride = q_out_stride;
  p.cos_sin = rope.cos_sin;
  p.max_pos = rope.max_positions;
  p.rot = turned ? rope.rot_dim : 0;
  p.interleaved = rope.interleaved != 0;
  p.cu = cu_seqlens;
  p.ctx = context_lens;
  p.block_table = block_table;
  p.n_tokens = n_tokens;
  p.B = batch;
  p.max_q_len = std::min(max_q_len, n_tokens);  // (longer ones have rows beyond n_tokens)
  p.Hq = num_q_heads;
  p.H = cache.num_kv_heads;
  p.num_blocks = cache.num_blocks;
  p.max_blocks = max_blocks;
  p.kc = static_cast<uint8_t*>(cache.k_cache);
  p.vc = static_cast<uint8_t*>(cache.v_cache);
  p.ks = cache.k_scale;
  p.vs = cache.v_scale;
  p.fault = fault;
  return from_cuda(fkv::launch_block_cache(p, cache.head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

float base2_scale(float softmax_scale, int32_t head_dim) {
  const float tau = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
  return tau * 1.4426950408889634f;
}

// fp8_block_decode_attn, and with num_groups > 0 fp8_block_shared_decode_attn, whose plan and pieces lie behind the decode's own
// workspace.
fkv_status block_decode_entry(const void* q, int32_t batch, int32_t num_q_heads, fkv_block_cache cache, const int32_t* block_table,
                              int32_t max_blocks, const int32_t* context_lens, const int32_t* group_starts,
                              const int32_t* shared_lens, int32_t num_groups, float softmax_scale, int32_t window, void* out,
                              void* workspace, size_t workspace_bytes, int32_t* fault, fkv_stream_t stream) {
  if (batch < 0 || num_q_heads <= 0 || max_blocks <= 0 || window < 0) return FKV_INVALID_ARG;
  const fkv_status st = check_block_cache(cache);
  if (st != FKV_OK) return st;
  if (num_q_heads % cache.num_kv_heads != 0) return FKV_INVALID_ARG;
  const int G = num_q_heads / cache.num_kv_heads;
  if (!supported_group(G, cache.head_dim)) return FKV_UNSUPPORTED;
  if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale)) return FKV_INVALID_ARG;
  if (batch > 65535 || num_q_heads > 65535 || max_blocks > kMaxTableBlocks) return FKV_UNSUPPORTED;
  if (batch == 0) return FKV_OK;
  if (!q || !out || !block_table || !context_lens || !valid_block_pools(cache)) return FKV_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(context_lens, 4))
    return FKV_INVALID_ARG;
  const BlockDecodePlan plan = plan_block_decode(batch, num_q_heads, cache.num_kv_heads, cache.head_dim);
  const size_t own_bytes = align256(plan.cnt_bytes + plan.lse_bytes + plan.o_bytes);
  const size_t need = num_groups == 0 ? plan.cnt_bytes + plan.lse_bytes + plan.o_bytes
                                      : own_bytes + fkv::block_shared_workspace(batch, num_q_heads, cache.num_kv_heads, cache.head_dim,
                                                                                num_groups, current_num_sms());
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return FKV_INVALID_ARG;
  fkv::BlockDecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(cache.k_cache);
  p.v_cache = static_cast<const uint8_t*>(cache.v_cache);
  p.k_scale = cache.k_scale;
  p.v_scale = cache.v_scale;
  p.block_table = block_table;
  p.ctx = context_lens;
  p.B = batch;
  p.Hq = num_q_heads;
  p.Hkv = cache.num_kv_heads << plan.halves;
  p.halves = plan.halves;
  p.num_blocks = cache.num_blocks;
  p.max_blocks = max_blocks;
  p.sm_scale_log2 = base2_scale(softmax_scale, cache.head_dim);
  p.window = window;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  p.done = reinterpret_cast<int32_t*>(at);
  p.lse_part = reinterpret_cast<float*>(at + plan.cnt_bytes);
  p.o_part = reinterpret_cast<float*>(at + plan.cnt_bytes + plan.lse_bytes);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.fault = fault;
  p.stage_wait_ns = pipe_wait_ns();
  // no more CTAs than there can be places (a unit's tiles and the blank one that leads them)
  const long long blocks = window > 0 ? std::min<long long>(max_blocks, (window + 15LL) / 16 + 1) : max_blocks;
  const int tpb = fkv::block_decode_tile_blocks(cache.head_dim);
  const long long tiles = static_cast<long long>(batch) * p.Hkv * ((blocks + tpb - 1) / tpb + 1);
  if (tiles > INT32_MAX) return FKV_UNSUPPORTED;  // the kernel counts them in 32 bits
  const int ctas = static_cast<int>(std::min(plan.ctas, tiles));
  if (num_groups > 0)
    return from_cuda(fkv::launch_block_shared(p, cache.head_dim, ctas, group_starts, shared_lens, num_groups, at + own_bytes,
                                              current_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
  return from_cuda(fkv::launch_block_decode(p, cache.head_dim, ctas, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

namespace fkv {

// fp8_decode_attn, and with k_new / v_new given fp8_decode_step (the current token written
// into the pools by the same launch).  With `scratch` non-null the workspace arguments are
// ignored: after every argument check and the split-K plan, scratch(need, ...) supplies the
// workspace (fp8_decode_attn_noalloc), so both entry points return the same status for
// the same arguments.
fkv_status decode_entry(const void* k_new, const void* v_new, const void* q, int32_t batch, int32_t num_q_heads,
                        fkv_layer_cache cache, const int32_t* block_table, int32_t max_blocks,
                        const int32_t* context_lens, const float* q_scale, const float* k_scale,
                        const float* v_scale, fkv_scale_gran gran, float softmax_scale, int32_t window,
                        int32_t layer, const uint8_t* skip_layer_mask, int32_t num_layers, void* out,
                        void* workspace, size_t workspace_bytes, ScratchProvider scratch, int32_t num_splits,
                        int32_t* fault, fkv_stream_t stream) {
  const bool step = k_new != nullptr || v_new != nullptr;
  if (batch < 0 || num_q_heads <= 0 || max_blocks <= 0 || window < 0 || num_splits < 0)
    return FKV_INVALID_ARG;
  if (cache.block_size != 16) return cache.block_size > 0 ? FKV_UNSUPPORTED : FKV_INVALID_ARG;
  if (cache.num_blocks <= 0 || cache.num_kv_heads <= 0 || !valid_format(cache)) return FKV_INVALID_ARG;
  if (num_q_heads % cache.num_kv_heads != 0) return FKV_INVALID_ARG;
  if (!supported_head_dim(cache.head_dim)) return FKV_UNSUPPORTED;
  const int G = num_q_heads / cache.num_kv_heads;
  if (!supported_group(G, cache.head_dim)) return FKV_UNSUPPORTED;
  if (gran != FKV_SCALE_PER_TENSOR && gran != FKV_SCALE_PER_HEAD) return FKV_INVALID_ARG;
  if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale)) return FKV_INVALID_ARG;
  if (batch > 65535 || cache.num_kv_heads > 65535) return FKV_UNSUPPORTED;
  fkv_status st = FKV_OK;
  const bool bf16 = layer_is_bf16(layer, skip_layer_mask, num_layers, &st);
  if (st != FKV_OK) return st;
  const int elt = layer_elt(bf16, cache);
  if (batch == 0) return FKV_OK;
  if (step && (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16))) return FKV_INVALID_ARG;
  if (!q || !out || !block_table || !context_lens || !cache.k_cache || !cache.v_cache || (!workspace && !scratch))
    return FKV_INVALID_ARG;
  if (!bf16 && (!q_scale || !k_scale || !v_scale)) return FKV_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache.k_cache, 16) || !aligned(cache.v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(context_lens, 4))
    return FKV_INVALID_ARG;
  DecodePlan plan;
  if (!plan_decode(batch, num_q_heads, cache.num_kv_heads, cache.head_dim, max_blocks, window, num_splits, &plan))
    return FKV_UNSUPPORTED;
  const size_t need = plan.o_bytes + plan.lse_bytes + plan.cnt_bytes;
  if (scratch) {
    const fkv_status sst = scratch(need, plan.cnt_bytes, reinterpret_cast<cudaStream_t>(stream), &workspace,
                                   &workspace_bytes);
    if (sst != FKV_OK) return sst;
  }
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return FKV_INVALID_ARG;

  DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(cache.k_cache);
  p.v_cache = static_cast<const uint8_t*>(cache.v_cache);
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.q_scale = q_scale;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.per_head = gran == FKV_SCALE_PER_HEAD;
  p.B = batch;
  p.Hq = num_q_heads;
  p.Hkv = cache.num_kv_heads;
  p.num_blocks = cache.num_blocks;
  p.max_blocks = max_blocks;
  const float tau = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(cache.head_dim));
  p.sm_scale_log2 = tau * 1.4426950408889634f;
  p.window = window;
  p.bps = plan.bps;
  p.max_splits = plan.max_splits;
  // workspace: the split-completion counters first (zero between calls), then the
  // splits' log-sum-exps and normalised outputs (written before they are read)
  p.done = static_cast<int32_t*>(workspace);
  p.lse_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.cnt_bytes);
  p.o_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.cnt_bytes + plan.lse_bytes);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.fault = fault;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.pipe_wait_ns = pipe_wait_ns();
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (fkv::decode_uses_tensor_cores(cache.head_dim, elt)) return from_cuda(fkv::launch_decode_tc(p, cache.head_dim, G, s));
  return from_cuda(fkv::launch_decode(p, cache.head_dim, elt, G, s));
}

}  // namespace fkv

using fkv::decode_entry;

extern "C" {

const char* fkv_status_string(fkv_status status) {
  switch (status) {
    case FKV_OK: return "ok";
    case FKV_INVALID_ARG: return "invalid argument";
    case FKV_UNSUPPORTED: return "unsupported";
    case FKV_CUDA_ERROR: return "cuda error";
  }
  return "unknown status";
}

int32_t fkv_version(void) { return 107; }

void fkv_set_decode_wait_limit_ns(unsigned long long ns) { g_decode_wait_ns.store(ns, std::memory_order_relaxed); }


fkv_status kv_quant_cache(const void* k, const void* v, const int64_t* slot_mapping, int32_t n_tokens,
                          fkv_layer_cache cache, const float* k_scale, const float* v_scale,
                          fkv_scale_gran gran, int32_t layer, const uint8_t* skip_layer_mask,
                          int32_t num_layers, int32_t* fault, fkv_stream_t stream) {
  return cache_write(k, v, slot_mapping, n_tokens, cache, k_scale, v_scale, gran, layer, skip_layer_mask, num_layers,
                     fault, stream, nullptr);
}

fkv_status kv_quant_cache_clips(const void* k, const void* v, const int64_t* slot_mapping, int32_t n_tokens,
                                fkv_layer_cache cache, const float* k_scale, const float* v_scale,
                                fkv_scale_gran gran, int32_t layer, const uint8_t* skip_layer_mask,
                                int32_t num_layers, unsigned long long* clip_counts, int32_t* fault,
                                fkv_stream_t stream) {
  if (clip_counts == nullptr) return FKV_INVALID_ARG;
  return cache_write(k, v, slot_mapping, n_tokens, cache, k_scale, v_scale, gran, layer, skip_layer_mask, num_layers,
                     fault, stream, clip_counts);
}

size_t fp8_decode_attn_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t head_dim, int32_t max_blocks, int32_t window,
                                      int32_t num_splits) {
  DecodePlan plan;
  if (!supported_head_dim(head_dim)) return 0;
  if (!plan_decode(batch, num_q_heads, num_kv_heads, head_dim, max_blocks, window, num_splits, &plan)) return 0;
  return plan.o_bytes + plan.lse_bytes + plan.cnt_bytes;
}

int32_t fp8_decode_attn_split_blocks(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t max_blocks, int32_t window,
                                     int32_t num_splits) {
  DecodePlan plan;
  if (!plan_decode(batch, num_q_heads, num_kv_heads, head_dim, max_blocks, window, num_splits, &plan)) return 0;
  return plan.bps;
}

int32_t fkv_decode_block_n(int32_t head_dim, int32_t layer_kind) {
  const int elt = layer_kind == 0 ? 1 : layer_kind == 1 ? 2 : layer_kind == 2 ? 3 : 0;
  return elt != 0 && fkv::decode_uses_tensor_cores(head_dim, elt) ? 16 * decode_tile_blocks(head_dim) : 0;
}

int32_t fp8_decode_attn_num_splits(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t max_blocks, int32_t window,
                                   int32_t num_splits) {
  DecodePlan plan;
  if (!plan_decode(batch, num_q_heads, num_kv_heads, head_dim, max_blocks, window, num_splits, &plan)) return 0;
  return plan.max_splits;
}

fkv_status fp8_decode_attn(const void* q, int32_t batch, int32_t num_q_heads, fkv_layer_cache cache,
                           const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                           const float* q_scale, const float* k_scale, const float* v_scale,
                           fkv_scale_gran gran, float softmax_scale, int32_t window, int32_t layer,
                           const uint8_t* skip_layer_mask, int32_t num_layers, void* out, void* workspace,
                           size_t workspace_bytes, int32_t num_splits, int32_t* fault,
                           fkv_stream_t stream) {
  return decode_entry(nullptr, nullptr, q, batch, num_q_heads, cache, block_table, max_blocks, context_lens, q_scale,
                      k_scale, v_scale, gran, softmax_scale, window, layer, skip_layer_mask, num_layers, out, workspace,
                      workspace_bytes, nullptr, num_splits, fault, stream);
}

fkv_status fp8_decode_step(const void* k_new, const void* v_new, const void* q, int32_t batch,
                           int32_t num_q_heads, fkv_layer_cache cache, const int32_t* block_table,
                           int32_t max_blocks, const int32_t* context_lens, const float* q_scale,
                           const float* k_scale, const float* v_scale, fkv_scale_gran gran,
                           float softmax_scale, int32_t window, int32_t layer, const uint8_t* skip_layer_mask,
                           int32_t num_layers, void* out, void* workspace, size_t workspace_bytes,
                           int32_t num_splits, int32_t* fault, fkv_stream_t stream) {
  if (!k_new || !v_new) return FKV_INVALID_ARG;
  return decode_entry(k_new, v_new, q, batch, num_q_heads, cache, block_table, max_blocks, context_lens, q_scale,
                      k_scale, v_scale, gran, softmax_scale, window, layer, skip_layer_mask, num_layers, out, workspace,
                      workspace_bytes, nullptr, num_splits, fault, stream);
}

int32_t fkv_prefill_block_n(int32_t head_dim) { return supported_head_dim(head_dim) ? 128 : 0; }

fkv_status fp8_prefill_attn(const void* q, const int32_t* cu_seqlens_q, int32_t batch, int32_t num_q_heads,
                            int32_t max_q_len, fkv_layer_cache cache, const int32_t* block_table,
                            int32_t max_blocks, const int32_t* context_lens, const float* q_scale,
                            const float* k_scale, const float* v_scale, fkv_scale_gran gran,
                            float softmax_scale, int32_t causal, int32_t window, int32_t promote_every,
                            int32_t layer, const uint8_t* skip_layer_mask, int32_t num_layers, void* out,
                            int32_t* fault, fkv_stream_t stream) {
  if (batch < 0 || num_q_heads <= 0 || max_q_len < 0 || max_blocks <= 0) return FKV_INVALID_ARG;
  if (cache.block_size != 16) return cache.block_size > 0 ? FKV_UNSUPPORTED : FKV_INVALID_ARG;
  if (cache.num_blocks <= 0 || cache.num_kv_heads <= 0 || !valid_format(cache)) return FKV_INVALID_ARG;
  if (num_q_heads % cache.num_kv_heads != 0) return FKV_INVALID_ARG;
  if (!supported_head_dim(cache.head_dim)) return FKV_UNSUPPORTED;
  if (gran != FKV_SCALE_PER_TENSOR && gran != FKV_SCALE_PER_HEAD) return FKV_INVALID_ARG;
  if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale)) return FKV_INVALID_ARG;
  if (window < 0 || promote_every < 0) return FKV_INVALID_ARG;
  if (window > 0 && !causal) return FKV_UNSUPPORTED;                        // a window is causal
  fkv_status st = FKV_OK;
  const bool bf16 = layer_is_bf16(layer, skip_layer_mask, num_layers, &st);
  if (st != FKV_OK) return st;
  // bf16 layers at head_dim 256: TMEM holds one 128-column O_tile
  if (promote_every >= 2 && cache.head_dim > 128 && bf16) return FKV_UNSUPPORTED;
  if (!bf16 && cache.kv_format == FKV_KV_E5M2) return FKV_UNSUPPORTED;  // e5m2 layers: decode only
  if (batch > 65535 || num_q_heads > 65535) return FKV_UNSUPPORTED;
  if (batch == 0 || max_q_len == 0) return FKV_OK;
  if (!q || !cu_seqlens_q || !block_table || !context_lens || !cache.k_cache || !cache.v_cache || !out)
    return FKV_INVALID_ARG;
  if (!bf16 && (!q_scale || !k_scale || !v_scale)) return FKV_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache.k_cache, 16) || !aligned(cache.v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(cu_seqlens_q, 4))
    return FKV_INVALID_ARG;
  fkv::PrefillParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cu_q = cu_seqlens_q;
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.q_scale = q_scale;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.per_head = gran == FKV_SCALE_PER_HEAD;
  p.B = batch;
  p.Hq = num_q_heads;
  p.Hkv = cache.num_kv_heads;
  p.num_blocks = cache.num_blocks;
  p.max_blocks = max_blocks;
  p.n_qtiles = (max_q_len + 127) / 128;
  const float tau = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(cache.head_dim));
  p.sm_scale_log2 = tau * 1.4426950408889634f;
  p.causal = causal != 0;
  p.promote_every = promote_every;
  p.window = window;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.fault = fault;
  return from_cuda(fkv::launch_prefill(p, cache.head_dim, bf16, cache.k_cache, cache.v_cache,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

fkv_status kv_rope_cache(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int64_t* positions,
                         const int64_t* slot_mapping, int32_t n_tokens, fkv_rope rope, fkv_layer_cache cache,
                         const float* k_scale, const float* v_scale, fkv_scale_gran gran, int32_t layer,
                         const uint8_t* skip_layer_mask, int32_t num_layers, int32_t* fault, fkv_stream_t stream) {
  const fkv_axes one = {positions, 0, 1, nullptr};
  return rope_cache_entry(q, q_stride, q_out, q_out_stride, num_q_heads, k, k_stride, v, v_stride, one, slot_mapping, n_tokens,
                          rope, cache, k_scale, v_scale, gran, layer, skip_layer_mask, num_layers, fault, stream);
}

fkv_status kv_rope_cache_axes(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride, fkv_axes axes,
                              const int64_t* slot_mapping, int32_t n_tokens, fkv_rope rope, fkv_layer_cache cache,
                              const float* k_scale, const float* v_scale, fkv_scale_gran gran, int32_t layer,
                              const uint8_t* skip_layer_mask, int32_t num_layers, int32_t* fault, fkv_stream_t stream) {
  return rope_cache_entry(q, q_stride, q_out, q_out_stride, num_q_heads, k, k_stride, v, v_stride, axes, slot_mapping, n_tokens,
                          rope, cache, k_scale, v_scale, gran, layer, skip_layer_mask, num_layers, fault, stream);
}

fkv_status kv_block_cache(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride, int32_t n_tokens,
                          const int32_t* cu_seqlens, int32_t batch, int32_t max_q_len, fkv_rope rope,
                          fkv_block_cache cache, const int32_t* block_table, int32_t max_blocks,
                          const int32_t* context_lens, int32_t* fault, fkv_stream_t stream) {
  return block_cache_entry(q, q_stride, q_out, q_out_stride, num_q_heads, k, k_stride, v, v_stride, n_tokens, nullptr, cu_seqlens,
                           batch, max_q_len, rope, cache, block_table, max_blocks, context_lens, fault, stream);
}

fkv_status kv_block_cache_axes(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride, int32_t n_tokens,
                               fkv_axes axes, const int32_t* cu_seqlens, int32_t batch, int32_t max_q_len, fkv_rope rope,
                               fkv_block_cache cache, const int32_t* block_table, int32_t max_blocks,
                               const int32_t* context_lens, int32_t* fault, fkv_stream_t stream) {
  return block_cache_entry(q, q_stride, q_out, q_out_stride, num_q_heads, k, k_stride, v, v_stride, n_tokens, &axes, cu_seqlens,
                           batch, max_q_len, rope, cache, block_table, max_blocks, context_lens, fault, stream);
}

size_t fp8_block_decode_attn_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim) {
  if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0) return 0;
  if (!supported_head_dim(head_dim) || !supported_group(num_q_heads / num_kv_heads, head_dim)) return 0;
  const BlockDecodePlan plan = plan_block_decode(batch, num_q_heads, num_kv_heads, head_dim);
  return plan.cnt_bytes + plan.lse_bytes + plan.o_bytes;
}

fkv_status fp8_block_decode_attn(const void* q, int32_t batch, int32_t num_q_heads, fkv_block_cache cache,
                                 const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                                 float softmax_scale, int32_t window, void* out, void* workspace,
                                 size_t workspace_bytes, int32_t* fault, fkv_stream_t stream) {
  return block_decode_entry(q, batch, num_q_heads, cache, block_table, max_blocks, context_lens, nullptr, nullptr, 0, softmax_scale, window,
                            out, workspace, workspace_bytes, fault, stream);
}

fkv_status fp8_block_prefill_attn(const void* q, const int32_t* cu_seqlens_q, int32_t total_q, int32_t batch,
                                  int32_t num_q_heads, int32_t max_q_len, fkv_block_cache cache,
                                  const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                                  float softmax_scale, int32_t causal, int32_t window, void* out, int32_t* fault,
                                  fkv_stream_t stream) {
  if (total_q < 0 || batch < 0 || num_q_heads <= 0 || max_q_len < 0 || max_blocks <= 0) return FKV_INVALID_ARG;
  const fkv_status st = check_block_cache(cache);
  if (st != FKV_OK) return st;
  if (num_q_heads % cache.num_kv_heads != 0) return FKV_INVALID_ARG;
  if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale) || window < 0) return FKV_INVALID_ARG;
  if (window > 0 && !causal) return FKV_UNSUPPORTED;  // a window is causal
  if (batch > 65535 || num_q_heads > 65535 || max_blocks > kMaxTableBlocks) return FKV_UNSUPPORTED;
  if (total_q == 0 || batch == 0 || max_q_len == 0) return FKV_OK;
  if (!q || !cu_seqlens_q || !block_table || !context_lens || !out || !valid_block_pools(cache)) return FKV_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(context_lens, 4) ||
      !aligned(cu_seqlens_q, 4))
    return FKV_INVALID_ARG;
  fkv::BlockPrefillParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(cache.k_cache);
  p.v_cache = static_cast<const uint8_t*>(cache.v_cache);
  p.k_scale = cache.k_scale;
  p.v_scale = cache.v_scale;
  p.block_table = block_table;
  p.ctx = context_lens;
  p.cu = cu_seqlens_q;
  p.B = batch;
  p.Hq = num_q_heads;
  p.Hkv = cache.num_kv_heads;
  p.num_blocks = cache.num_blocks;
  p.max_blocks = max_blocks;
  p.max_q_len = std::min(max_q_len, total_q);  // (longer ones have rows beyond total_q)
  p.total_q = total_q;
  p.sm_scale_log2 = base2_scale(softmax_scale, cache.head_dim);
  p.causal = causal != 0;
  p.window = window;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.fault = fault;
  p.stage_wait_ns = pipe_wait_ns();
  return from_cuda(fkv::launch_block_prefill(p, cache.head_dim, current_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

size_t fp8_block_shared_decode_attn_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                                   int32_t head_dim, int32_t num_groups) {
  const size_t own = fp8_block_decode_attn_workspace_size(batch, num_q_heads, num_kv_heads, head_dim);
  if (num_groups <= 0 || own == 0) return num_groups < 0 ? 0 : own;
  return align256(own) + fkv::block_shared_workspace(batch, num_q_heads, num_kv_heads, head_dim, num_groups, current_num_sms());
}

fkv_status fp8_block_shared_decode_attn(const void* q, int32_t batch, int32_t num_q_heads, fkv_block_cache cache,
                                        const int32_t* block_table, int32_t max_blocks, const int32_t* context_lens,
                                        const int32_t* group_starts, const int32_t* shared_lens, int32_t num_groups,
                                        float softmax_scale, int32_t window, void* out, void* workspace,
                                        size_t workspace_bytes, int32_t* fault, fkv_stream_t stream) {
  if (num_groups < 0) return FKV_INVALID_ARG;
  if (num_groups > 0 && (!group_starts || !shared_lens || !aligned(group_starts, 4) || !aligned(shared_lens, 4)))
    return FKV_INVALID_ARG;
  return block_decode_entry(q, batch, num_q_heads, cache, block_table, max_blocks, context_lens, group_starts, shared_lens, num_groups,
                            softmax_scale, window, out, workspace, workspace_bytes, fault, stream);
}

size_t fp8_block_attn_weights_workspace_size(int32_t batch, int32_t total_q, int32_t max_q_len, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim, int32_t max_blocks) {
  if (batch <= 0 || total_q <= 0 || max_q_len <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks <= 0) return 0;
  if (num_q_heads % num_kv_heads != 0 || !supported_head_dim(head_dim) || max_blocks > kMaxTableBlocks) return 0;
  if (static_cast<long long>(total_q) * (num_q_heads / num_kv_heads) > kMaxWeightRows) return 0;
  return fkv::block_weights_workspace(batch, total_q, std::min(max_q_len, total_q), num_q_heads, num_kv_heads, head_dim,
                                      max_blocks * 16LL, current_num_sms());
}

fkv_status fp8_block_attn_weights(const void* q, const int32_t* cu_seqlens_q, int32_t total_q, int32_t batch,
                                  int32_t num_q_heads, int32_t max_q_len, fkv_block_cache cache, const int32_t* block_table,
                                  int32_t max_blocks, const int32_t* context_lens, float softmax_scale, float decay,
                                  float* weights, int32_t weights_len, void* workspace, size_t workspace_bytes,
                                  int32_t* fault, fkv_stream_t stream) {
  if (total_q < 0 || batch < 0 || num_q_heads <= 0 || max_q_len < 0 || max_blocks <= 0 || weights_len < 0) return FKV_INVALID_ARG;
  const fkv_status st = check_block_cache(cache);
  if (st != FKV_OK) return st;
  if (num_q_heads % cache.num_kv_heads != 0) return FKV_INVALID_ARG;
  if (!(softmax_scale >= 0.f) || std::isinf(softmax_scale) || !std::isfinite(decay)) return FKV_INVALID_ARG;
  if (batch > 65535 || num_q_heads > 65535 || max_blocks > kMaxTableBlocks) return FKV_UNSUPPORTED;
  if (static_cast<long long>(total_q) * (num_q_heads / cache.num_kv_heads) > kMaxWeightRows) return FKV_UNSUPPORTED;
  if (total_q == 0 || batch == 0 || max_q_len == 0) return FKV_OK;
  if (!q || !cu_seqlens_q || !block_table || !context_lens || (!weights && weights_len > 0) || !valid_block_pools(cache))
    return FKV_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(cu_seqlens_q, 4) || !aligned(weights, 4))
    return FKV_INVALID_ARG;
  const size_t need = fp8_block_attn_weights_workspace_size(batch, total_q, max_q_len, num_q_heads, cache.num_kv_heads,
                                                            cache.head_dim, max_blocks);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return FKV_INVALID_ARG;
  fkv::BlockWeightsParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(cache.k_cache);
  p.k_scale = cache.k_scale;
  p.block_table = block_table;
  p.ctx = context_lens;
  p.cu = cu_seqlens_q;
  p.B = batch;
  p.Hq = num_q_heads;
  p.Hkv = cache.num_kv_heads;
  p.num_blocks = cache.num_blocks;
  p.max_blocks = max_blocks;
  p.max_q_len = std::min(max_q_len, total_q);  // (longer ones have rows beyond total_q)
  p.total_q = total_q;
  p.sm_scale_log2 = base2_scale(softmax_scale, cache.head_dim);
  p.decay = decay;
  p.weights = weights;
  p.weights_len = weights_len;
  p.fault = fault;
  p.stage_wait_ns = pipe_wait_ns();
  return from_cuda(fkv::launch_block_weights(p, cache.head_dim, workspace, current_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

fkv_status kv_block_evict(fkv_block_cache cache, const int32_t* block_table, int32_t batch, int32_t max_blocks,
                          const int32_t* context_lens, const float* weights, int32_t weights_len, int32_t budget,
                          int32_t sink, int32_t recent, const int32_t* new_table, int32_t new_max_blocks, int32_t* new_lens,
                          int32_t* kept, float* new_weights, int32_t new_weights_len, int32_t* fault, fkv_stream_t stream) {
  if (batch < 0 || max_blocks <= 0 || weights_len < 0 || new_max_blocks < 0 || new_weights_len < 0) return FKV_INVALID_ARG;
  if (budget < 1 || sink < 0 || recent < 0 || recent > budget || sink > budget - recent) return FKV_INVALID_ARG;
  const fkv_status st = check_block_cache(cache);
  if (st != FKV_OK) return st;
  if (batch > 65535 || cache.num_kv_heads > 8192 || max_blocks > kMaxTableBlocks) return FKV_UNSUPPORTED;
  const long long most = std::min({static_cast<long long>(budget), max_blocks * 16LL, static_cast<long long>(weights_len)});
  if (most > new_max_blocks * 16LL || (new_weights && most > new_weights_len)) return FKV_INVALID_ARG;
  // the kernels' grids
  if (static_cast<long long>(batch) * cache.num_kv_heads * ((most + 15) / 16 + 8) > INT32_MAX) return FKV_UNSUPPORTED;
  if (batch == 0) return FKV_OK;
  if (!valid_block_pools(cache)) return FKV_INVALID_ARG;
  if (!block_table || !context_lens || (!weights && weights_len > 0) || (!new_table && new_max_blocks > 0) || !new_lens || !kept || !aligned(block_table, 4) ||
      !aligned(context_lens, 4) || !aligned(weights, 4) || !aligned(new_table, 4) || !aligned(new_lens, 4) ||
      !aligned(kept, 4) || !aligned(new_weights, 4))
    return FKV_INVALID_ARG;
  // a sequence's heads read its length, and their weights, in any order
  const uint64_t units = static_cast<uint64_t>(batch) * cache.num_kv_heads;
  if (overlap(new_lens, batch, context_lens, batch) ||
      (new_weights && overlap(new_weights, units * new_weights_len, weights, units * weights_len)))
    return FKV_INVALID_ARG;
  fkv::EvictParams p;
  std::memset(&p, 0, sizeof(p));
  p.kc = static_cast<uint8_t*>(cache.k_cache);
  p.vc = static_cast<uint8_t*>(cache.v_cache);
  p.ks = cache.k_scale;
  p.vs = cache.v_scale;
  p.B = batch;
  p.H = cache.num_kv_heads;
  p.num_blocks = cache.num_blocks;
  p.max_blocks = max_blocks;
  p.new_max_blocks = new_max_blocks;
  p.block_table = block_table;
  p.ctx = context_lens;
  p.weights = weights;
  p.weights_len = weights_len;
  p.new_weights_len = new_weights_len;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.new_table = new_table;
  p.new_lens = new_lens;
  p.kept = kept;
  p.new_weights = new_weights;
  p.fault = fault;
  return from_cuda(fkv::launch_block_evict(p, cache.head_dim, current_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
