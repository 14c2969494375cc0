// Decode attention over a block-scaled cache for sequences that share their first tokens: the shared keys and values are read
// and multiplied once for all members of a group.
//
//   plan_kernel    on the GPU, where lengths and groups are known: which groups share, into how many pieces their keys are cut,
//                  which CTA takes which;
//   prefix_kernel  a CTA per piece: up to 128 rows (member, head) of a KV head against a share of the shared keys, the
//                  tile of block_attend.cuh, whose result goes to the workspace as (o, lse);
//   block_decode_kernel<.., true>  what every sequence has of its own, and sequences that share nothing;
//   join_kernel    per (sequence, KV head) o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M) over both kinds of pieces.
#include "block_attend.cuh"
#include "block_decode_kernel.cuh"
#include "block_shared.cuh"

namespace fkv {
namespace {

// Sharing costs three more launches and the pieces' way through memory; the decode by itself reads 6 TB/s.
constexpr long long kLeastSaved = 1;

constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;
constexpr int kGroupsHeld = 512;  // groups whose numbers the plan keeps in shared memory

FKV_DEV int context_of(const SharedParams& p, int b) { return min(max(p.ctx[b], 0), static_cast<int>(min(p.max_blocks * 16LL, static_cast<long long>(INT32_MAX)))); }

FKV_DEV long long warp_sum(long long x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const SharedParams p) {
  __shared__ long long sum_s[kPlanWarps];
  __shared__ int items_s[kGroupsHeld], tiles_s[kGroupsHeld], most_s[kPlanWarps], cut_s[3], base_s;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto block_sum = [&](long long x) {
    x = warp_sum(x);
    __syncthreads();
    if (lane == 0) sum_s[warp] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) x += sum_s[w];
    return x;
  };
  bool bad = false;
  for (int i = tid; i < p.num_groups; i += kPlanThreads) {
    const int a = p.starts[i], e = p.starts[i + 1];
    bad = bad || a < 0 || e < a || e > p.B;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) raise_fault(p.fault, FKV_FAULT_QLEN);
  // the groups: members, shared keys (as many as the first member has), items (row tile, KV head), key tiles
  long long saved = 0, items = 0, steps = 0;
  int most = 0;
  for (int i = tid; i < p.num_groups; i += kPlanThreads) {
    SharedGroup g = {};
    int n_items = 0, tiles = 0;
    if (!bad) {
      g.first = p.starts[i];
      g.members = p.starts[i + 1] - g.first;
      g.keys = p.lens[i];
      if (g.keys < 0 || g.keys > p.max_blocks * 16LL) {
        raise_fault(p.fault, FKV_FAULT_CONTEXT);
        g.keys = 0;
      }
      g.keys = g.members >= 2 ? min(g.keys, context_of(p, g.first)) : 0;
      if (g.keys > 0) {
        g.lo = p.window > 0 ? max(0, g.keys - p.window) : 0;
        tiles = (g.keys + 127) / 128 - g.lo / 128;
        n_items = (g.members + p.tok - 1) / p.tok * p.Hkv;
        saved += static_cast<long long>(g.members - 1) * (g.keys - g.lo);
        items += n_items;
        steps += static_cast<long long>(n_items) * tiles;
        most = max(most, tiles);
      }
    }
    p.groups[i] = g;
    if (i < kGroupsHeld) {
      items_s[i] = n_items;
      tiles_s[i] = tiles;
    }
  }
  saved = block_sum(saved);
  items = block_sum(items);
  steps = block_sum(steps);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) most_s[warp] = most;
  __syncthreads();
  most = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) most = max(most, most_s[w]);
  const bool share = saved * p.Hkv * 2 * p.D >= kLeastSaved;
  // How many key tiles a piece has: the fewest whose pieces fit the SMs once (or twice, or three times: cut_s), by as many tries
  // as a warp has lanes; a wave costs about three tiles besides its own.  More items than that are not cut.
  if (share && warp < 3) {
    const long long room = static_cast<long long>(warp + 1) * p.num_sms;
    int c = 0;
    if (items <= room && p.num_groups <= kGroupsHeld) {
      const long long least = (steps + room - 1) / room;
      const int mine = static_cast<int>(least + least * lane / 12 + (least < 12 ? lane : 0));
      long long pieces = 0;
      for (int i = 0; i < p.num_groups; ++i) pieces += items_s[i] == 0 ? 0 : static_cast<long long>(items_s[i]) * ((tiles_s[i] + mine - 1) / mine);
      const unsigned fits = __ballot_sync(0xffffffffu, pieces <= room);
      if (fits != 0) c = __shfl_sync(0xffffffffu, mine, __ffs(fits) - 1);
    }
    if (lane == 0) cut_s[warp] = c;
  }
  if (tid == 0) base_s = 0;
  __syncthreads();
  int cut = max(most, 1);
  if (share) {
    long long best = items <= 3LL * p.num_sms ? (items + p.num_sms - 1) / p.num_sms * (most + 3LL) : 0;
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      const long long cost = (m + 1) * (cut_s[m] + 3LL);
      if (cut_s[m] > 0 && cost < best) {
        best = cost;
        cut = cut_s[m];
      }
    }
  }
  // the pieces' places, group after group
  for (int i0 = 0; i0 < p.num_groups; i0 += kPlanThreads) {
    const int i = i0 + tid;
    SharedGroup g = {};
    int pieces = 0;
    if (i < p.num_groups) {
      g = p.groups[i];
      if (!share) g.keys = 0;
      if (g.keys > 0) {
        const int tiles = (g.keys + 127) / 128 - g.lo / 128;
        g.shares = (tiles + cut - 1) / cut;
        pieces = (g.members + p.tok - 1) / p.tok * p.Hkv * g.shares;
      }
    }
    int upto = pieces;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) most_s[warp] = upto;
    __syncthreads();
    int before = base_s;
    for (int w = 0; w < warp; ++w) before += most_s[w];
    g.base = before + upto - pieces;
    if (i < p.num_groups) p.groups[i] = g;
    __syncthreads();
    if (tid == kPlanThreads - 1) base_s = before + upto;
    __syncthreads();
  }
  if (tid == 0) *p.pieces = base_s;
  // the sequences: in which group, if it shares (a member shorter than the shared part does not)
  for (int b = tid; b < p.B; b += kPlanThreads) {
    int lo = 0, hi = share && !bad ? p.num_groups : 0;  // groups before lo begin at or before b, those from hi on behind it
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.starts[mid] <= b) lo = mid + 1;
      else hi = mid;
    }
    int4 out = make_int4(0, 0, 0, 0);
    if (lo > 0) {
      const SharedGroup g = p.groups[lo - 1];
      if (b < g.first + g.members && g.keys > 0 && context_of(p, b) >= g.keys) out = make_int4(g.keys, g.base, g.shares, b - g.first);
    }
    p.info[b] = out;
  }
}

template <int D, bool WIN>
__global__ void __launch_bounds__(512, 1)
    prefix_kernel(const __grid_constant__ BlockPrefillParams p, const __grid_constant__ SharedParams sp, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv) {
  // (the tensor memory, all of an SM's, is allocated after this wait, as in the prefill)
  griddep_wait();
  const int k = blockIdx.x, lane = threadIdx.x & 31;
  if (k >= *sp.pieces) return;
  // the last group whose pieces begin at or before this one
  int i = 0;
  for (int i0 = 0; i0 < sp.num_groups; i0 += 32) {
    const unsigned m = __ballot_sync(0xffffffffu, i0 + lane < sp.num_groups && sp.groups[i0 + lane].base <= k);
    if (m == 0) break;
    i = i0 + 31 - __clz(m);
    if (m != 0xffffffffu) break;
  }
  const SharedGroup g = sp.groups[i];
  const int at = k - g.base, item = at / g.shares, tile = item / sp.Hkv;
  Piece piece;
  piece.g = item - tile * sp.Hkv;
  piece.table_row = g.first;
  piece.kv_lo = g.lo;
  piece.o = sp.piece_o + static_cast<size_t>(k) * (D / 4) * 128;
  piece.lse = sp.piece_lse + static_cast<size_t>(k) * 128;
  attend_tile<D, WIN, kPieces>(p, tmk, tmv, g.first, g.members, g.keys, tile, at - item * g.shares, g.shares, piece);
}

constexpr int kJoinThreads = 128;

// CTA per (sequence, unit of the decode): a thread takes four columns of a head at a time, heads next to one another (as they lie
// in the prefix's pieces).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const SharedParams p, int units, int G) {
  __shared__ float top_s[16], inv_s[16];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / units, u = blockIdx.x - b * units;
  const int4 info = p.info[b];
  if (info.x == 0) return;
  const int T = context_of(p, b);
  int2 own = make_int2(0, 0);
  if (T > info.x) own = p.units[blockIdx.x];
  const float* own_lse = p.lse_part + (static_cast<long long>(own.x) + blockIdx.x) * G;
  const float4* own_o = reinterpret_cast<const float4*>(p.o_part + (static_cast<long long>(own.x) + blockIdx.x) * G * D);
  // head h of the unit among the rows of the prefix's pieces: the first one's CTA, and the row
  const int group = p.Hq / p.Hkv, tile = info.w / p.tok, row0 = (info.w - tile * p.tok) * group;
  auto place = [&](int h, int& row) {
    const int head = u * G + h, g = head / group;
    row = row0 + head - g * group;
    return info.y + (tile * p.Hkv + g) * info.z;
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = info.z + own.y;
  for (int h = warp; h < G; h += kJoinThreads / 32) {
    int row;
    const int k0 = place(h, row);
    auto lse = [&](int i) { return i < info.z ? p.piece_lse[static_cast<size_t>(k0 + i) * 128 + row] : own_lse[static_cast<size_t>(i - info.z) * G + h]; };
    float top = -kHuge;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, lse(i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) sum += ex2(lse(i) - top);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) {
      top_s[h] = top;
      inv_s[h] = 1.f / sum;
    }
  }
  __syncthreads();
  for (int q = threadIdx.x; q < G * D / 4; q += kJoinThreads) {
    const int d4 = q / G, h = q - d4 * G;
    int row;
    const int k0 = place(h, row);
    const float top = top_s[h];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, float4 x) {
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    };
#pragma unroll 4
    for (int i = 0; i < info.z; ++i)
      add(ex2(p.piece_lse[static_cast<size_t>(k0 + i) * 128 + row] - top), p.piece_o[(static_cast<size_t>(k0 + i) * (D / 4) + d4) * 128 + row]);
#pragma unroll 4
    for (int i = 0; i < own.y; ++i) add(ex2(own_lse[static_cast<size_t>(i) * G + h] - top), own_o[(static_cast<size_t>(i) * G + h) * (D / 4) + d4]);
    const float inv = inv_s[h];
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out + (static_cast<size_t>(b) * p.Hq + u * G + h) * D + 4 * d4);
    dst[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    dst[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  }
}

// CTAs of the prefix kernel, at most: three for every SM, or one for every item (groups of two and more).
long long prefix_ctas(int B, int Hq, int Hkv, int num_groups, int num_sms) {
  const int tok = 128 / (Hq / Hkv);
  return std::max<long long>(3LL * num_sms, static_cast<long long>(Hkv) * (B / tok + std::min(num_groups, B / 2)));
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

size_t lay_out(SharedParams* p, uint8_t* base, int B, int Hq, int Hkv, int D, int num_groups, long long ctas) {
  size_t at = 0;
  auto part = [&](size_t bytes) {
    uint8_t* x = base ? base + at : nullptr;
    at += up256(bytes);
    return x;
  };
  uint8_t* groups = part(static_cast<size_t>(num_groups) * sizeof(SharedGroup));
  uint8_t* pieces = part(sizeof(int));
  uint8_t* info = part(static_cast<size_t>(B) * sizeof(int4));
  uint8_t* units = part(static_cast<size_t>(B) * Hkv * 2 * sizeof(int2));
  uint8_t* lse = part(static_cast<size_t>(ctas) * 128 * sizeof(float));
  uint8_t* o = part(static_cast<size_t>(ctas) * 128 * D * sizeof(float));
  if (p) {
    p->groups = reinterpret_cast<SharedGroup*>(groups);
    p->pieces = reinterpret_cast<int*>(pieces);
    p->info = reinterpret_cast<int4*>(info);
    p->units = reinterpret_cast<int2*>(units);
    p->piece_lse = reinterpret_cast<float*>(lse);
    p->piece_o = reinterpret_cast<float4*>(o);
  }
  return at;
}

template <int D, int G>
cudaError_t launch_own(const BlockDecodeParams& p, const CUtensorMap& tmk, const CUtensorMap& tmv, int N, cudaStream_t s) {
  auto kern = block_decode_kernel<D, G, true>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BlockDecodeCfg<D, G>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(N), dim3(kThreads), BlockDecodeCfg<D, G>::SMEM, s, p, tmk, tmv);
}

template <int D, bool WIN>
cudaError_t launch_prefix(const BlockPrefillParams& p, const SharedParams& sp, const CUtensorMap& tmk, const CUtensorMap& tmv, int ctas, cudaStream_t s) {
  using C = BlockPrefillCfg<D>;
  auto kern = prefix_kernel<D, WIN>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // the warpgroups' register budgets add up to the launch's 128 per thread (a kernel built with fewer would wait forever)
  cudaFuncAttributes a;
  e = cudaFuncGetAttributes(&a, kern);
  if (e != cudaSuccess) return e;
  if (a.numRegs != C::REG_LAUNCH) return cudaErrorInvalidKernelImage;
  return launch_dependent(kern, dim3(ctas), dim3(C::THREADS), C::SMEM, s, p, sp, tmk, tmv);
}

template <int D>
cudaError_t launch_d(const BlockDecodeParams& dp, const SharedParams& sp, int ctas, int prefix, cudaStream_t s) {
  CUtensorMap tmk, tmv;
  constexpr int RB = BlockPrefillCfg<D>::RB;
  static_assert(RB == BlockDecodeCfg<D, 1>::RB, "one map serves both kernels");
  if (!make_pool_map(&tmk, const_cast<uint8_t*>(dp.k_cache), D, sp.Hkv, dp.num_blocks, RB) ||
      !make_pool_map(&tmv, const_cast<uint8_t*>(dp.v_cache), D, sp.Hkv, dp.num_blocks, RB))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_dependent(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, sp);
  if (e != cudaSuccess) return e;
  BlockPrefillParams p = {};
  p.q = dp.q;
  p.k_cache = dp.k_cache;
  p.v_cache = dp.v_cache;
  p.k_scale = dp.k_scale;
  p.v_scale = dp.v_scale;
  p.block_table = dp.block_table;
  p.ctx = dp.ctx;
  p.B = dp.B;
  p.Hq = dp.Hq;
  p.Hkv = sp.Hkv;
  p.num_blocks = dp.num_blocks;
  p.max_blocks = dp.max_blocks;
  p.sm_scale_log2 = dp.sm_scale_log2;
  p.window = dp.window;
  p.fault = dp.fault;
  p.stage_wait_ns = dp.stage_wait_ns;
  p.head_parts = 1;
  p.part_heads = dp.Hq / sp.Hkv;
  p.part_tokens = sp.tok;
  e = dp.window > 0 ? launch_prefix<D, true>(p, sp, tmk, tmv, prefix, s) : launch_prefix<D, false>(p, sp, tmk, tmv, prefix, s);
  if (e != cudaSuccess) return e;
  const int G = dp.Hq / dp.Hkv;
  e = G == 1 ? launch_own<D, 1>(dp, tmk, tmv, ctas, s) : G == 2 ? launch_own<D, 2>(dp, tmk, tmv, ctas, s) :
      G == 4 ? launch_own<D, 4>(dp, tmk, tmv, ctas, s) : G == 8 ? launch_own<D, 8>(dp, tmk, tmv, ctas, s) : cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return launch_dependent(join_kernel<D>, dim3(dp.B * dp.Hkv), dim3(kJoinThreads), 0, s, sp, dp.Hkv, G);
}

}  // namespace

size_t block_shared_workspace(int B, int Hq, int Hkv, int D, int num_groups, int num_sms) {
  return lay_out(nullptr, nullptr, B, Hq, Hkv, D, num_groups, prefix_ctas(B, Hq, Hkv, num_groups, num_sms));
}

cudaError_t launch_block_shared(BlockDecodeParams dp, int D, int ctas, const int32_t* starts, const int32_t* lens, int num_groups, void* workspace,
                                int num_sms, cudaStream_t s) {
  SharedParams sp = {};
  sp.B = dp.B;
  sp.Hq = dp.Hq;
  sp.Hkv = dp.Hkv >> dp.halves;
  sp.D = D;
  sp.max_blocks = dp.max_blocks;
  sp.window = dp.window;
  sp.num_groups = num_groups;
  sp.num_sms = num_sms;
  sp.tok = 128 / (sp.Hq / sp.Hkv);
  sp.ctx = dp.ctx;
  sp.starts = starts;
  sp.lens = lens;
  sp.out = dp.out;
  sp.fault = dp.fault;
  sp.lse_part = dp.lse_part;
  sp.o_part = dp.o_part;
  const long long prefix = prefix_ctas(dp.B, sp.Hq, sp.Hkv, num_groups, num_sms);
  if (prefix > INT32_MAX) return cudaErrorInvalidValue;
  lay_out(&sp, static_cast<uint8_t*>(workspace), dp.B, sp.Hq, sp.Hkv, D, num_groups, prefix);
  dp.shared = sp.info;
  dp.units = sp.units;
  if (D == 64) return launch_d<64>(dp, sp, ctas, static_cast<int>(prefix), s);
  if (D == 128) return launch_d<128>(dp, sp, ctas, static_cast<int>(prefix), s);
  return launch_d<256>(dp, sp, ctas, static_cast<int>(prefix), s);
}

}  // namespace fkv
