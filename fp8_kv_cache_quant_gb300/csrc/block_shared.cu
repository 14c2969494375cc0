// Decode attention over a block-scaled cache for sequences that share their first tokens: the shared keys and values are read
// and multiplied once for all members of a group.
//
//   plan_kernel    on the GPU, where lengths and groups are known: which groups share, into how many pieces their keys are cut,
//                  which CTA takes which;
//   prefix_kernel  a CTA per piece: up to 128 rows (member, head) of a KV head against a share of the shared keys, the
//                  tile of block_attend.cuh, whose result goes to the workspace as (o, lse);
//   block_decode_kernel<.., true>  what every sequence has of its own, and sequences that share nothing;
//   join_kernel    per (sequence, KV head) o = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M) over both kinds of pieces.
//
// What bounds it.  32 sequences of 16 to 1,024 tokens behind 32,768 shared ones, 32/8 heads of 128: 54 us (271 read one by one), in a
// chain: plan 3, prefix 26 (14 key tiles a CTA at 1.4 us, the softmax's instructions, as in the prefill), their own tokens 18
// (its fixed 15 of ramp, last pieces and merge) and join 6.  The four kernels follow one another in the stream.
#include <atomic>

#include "block_attend.cuh"
#include "block_decode_kernel.cuh"
#include "block_shared.cuh"

namespace fkv {
namespace {

// Bytes of keys and values that sharing has to save: it costs more launches, the pieces' way through memory and, per key tile that a
// CTA takes in turn, 0.8 to 1.5 us, where the decode by itself reads 6 TB/s.  us shared and not, 32/8 heads of 128: 8 sequences behind
// 8,192 tokens (saved 117 MB, 4 tiles) 26.0 and 27.0, behind 4,096 (59 MB, 2) 23.3 and 18.2; 4 behind 32,768 (201 MB, 14) 37.7 and
// 42.2, behind 16,384 (101 MB, 7) 29.2 and 25.8; 64/8 heads of 64: 8 behind 16,384 (117 MB, 7) 28.9 and 37.5, 4 (50 MB) 28.7 and
// 24.8; 16/8 heads of 256: 4 behind 16,384 (201 MB, 7) 41.5 and 46.6, 8,192 (101 MB, 4) 33.5 and 28.7.
__host__ __device__ constexpr bool sharing_pays(long long tokens, int Hkv, int D, int tiles) {  // (tokens, times heads, may pass 64 bits)
  return static_cast<double>(tokens) * 2 * Hkv * D >= static_cast<double>((48LL + D / 4 << 20) + (static_cast<long long>(D < 128 ? D : 128) << 16) * tiles);
}

constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;
constexpr int kGroupsHeld = 512, kLensHeld = 1024;  // groups and sequences whose numbers the plan keeps in shared memory

FKV_DEV int context_of(const SharedParams& p, int b) { return min(max(p.ctx[b], 0), static_cast<int>(min(p.max_blocks * 16LL, static_cast<long long>(INT32_MAX)))); }

FKV_DEV long long warp_sum(long long x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

FKV_DEV int tiles_of(const SharedGroup& g) { return (g.keys + 127) / 128 - g.lo / 128; }
FKV_DEV int items_of(const SharedParams& p, const SharedGroup& g) { return (g.members + p.tok - 1) / p.tok * p.Hkv; }  // (row tile, KV head)

// One CTA; what bounds it are its round trips to L2 (all numbers of the first 256 groups and sequences in one of them).
// With a window the shared part is what the shortest sharing member sees of the shared keys, as it sees them: what lies before its window is
// before every member's, where the blocks may be gone, and a longer member's row may have lost blocks that it still names.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const SharedParams p) {
  __shared__ SharedGroup held_s[kGroupsHeld];
  __shared__ long long sum_s[3][kPlanWarps];
  __shared__ int lens_s[kLensHeld], most_s[kPlanWarps], cut_s[3], base_s;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool first_in = tid < p.num_groups;
  const int first_a = first_in ? p.starts[tid] : 0, first_e = first_in ? p.starts[tid + 1] : 0, first_n = first_in ? p.lens[tid] : 0;
  for (int b = tid; b < min(p.B, kLensHeld); b += kPlanThreads) lens_s[b] = context_of(p, b);
  __syncthreads();
  auto context = [&](int b) { return b < kLensHeld ? lens_s[b] : context_of(p, b); };
  auto group = [&](int i) { return i < kGroupsHeld ? held_s[i] : p.groups[i]; };
  // the group that b is in, or would be by the groups' starts alone: the last that begins at or before it (-1: none)
  auto group_of = [&](int b) {
    int lo = 0, hi = p.num_groups;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (group(mid).first <= b) lo = mid + 1;
      else hi = mid;
    }
    return lo - 1;
  };
  // the groups: members, shared keys (as many as the first member has); what they save, their items and steps (item, key tile)
  long long saved = 0, items = 0, steps = 0;
  int most = 0;
  bool bad = false;
  auto counted = [&](const SharedGroup& g) {
    if (g.keys <= 0) return;
    const int tiles = tiles_of(g), n = items_of(p, g);
    saved += static_cast<long long>(g.members - 1) * (g.keys - g.lo);
    items += n;
    steps += static_cast<long long>(n) * tiles;
    most = max(most, tiles);
  };
  for (int i = tid; i < p.num_groups; i += kPlanThreads) {
    SharedGroup g = {};
    const int e = i < kPlanThreads ? first_e : p.starts[i + 1];
    g.first = i < kPlanThreads ? first_a : p.starts[i];
    g.keys = i < kPlanThreads ? first_n : p.lens[i];
    if (g.first < 0 || e < g.first || e > p.B) {
      bad = true;
      g.first = g.keys = 0;
    } else {
      g.members = e - g.first;
      if (g.keys < 0 || g.keys > p.max_blocks * 16LL) {
        raise_fault(p.fault, FKV_FAULT_CONTEXT);
        g.keys = 0;
      }
      g.keys = g.members >= 2 ? min(g.keys, context(g.first)) : 0;
    }
    g.row = g.first;
    if (p.window == 0) counted(g);
    (i < kGroupsHeld ? held_s[i] : p.groups[i]) = g;
    if (p.window > 0) p.least[i] = ~0ull;
  }
  if (p.window > 0) {
    __syncthreads();
    for (int b = tid; b < p.B; b += kPlanThreads) {
      const int i = group_of(b), T = context(b);
      if (i < 0) continue;
      const SharedGroup g = group(i);
      if (b < g.first + g.members && g.keys > 0 && T >= g.keys) atomicMin(&p.least[i], static_cast<unsigned long long>(T) << 32 | static_cast<unsigned>(b));
    }
    __syncthreads();
    for (int i = tid; i < p.num_groups; i += kPlanThreads) {
      SharedGroup g = group(i);
      const unsigned long long least = __ldcg(&p.least[i]);
      const int T = static_cast<int>(least >> 32);  // (-1: no member shares)
      g.lo = max(0, T - p.window);
      g.row = static_cast<int>(least & 0xFFFFFFFFu);
      if (T < 0 || g.lo >= g.keys) g.keys = 0;
      counted(g);
      (i < kGroupsHeld ? held_s[i] : p.groups[i]) = g;
    }
  }
  saved = warp_sum(saved);
  items = warp_sum(items);
  steps = warp_sum(steps);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    sum_s[0][warp] = saved;
    sum_s[1][warp] = items;
    sum_s[2][warp] = steps;
    most_s[warp] = most;
  }
  if (tid == 0) base_s = 0;
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) raise_fault(p.fault, FKV_FAULT_QLEN);
  saved = items = steps = most = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    saved += sum_s[0][w];
    items += sum_s[1][w];
    steps += sum_s[2][w];
    most = max(most, most_s[w]);
  }
  bool share = !bad && sharing_pays(saved, p.Hkv, p.D, 1);
  // How many key tiles a piece has: the fewest whose pieces fit the SMs once (or, where the grid has room for it, twice, or three
  // times: cut_s), by as many tries as a warp has lanes; a wave costs about three tiles besides its own.  More items than that are
  // not cut.
  if (share && warp < 3) {
    const long long room = static_cast<long long>(warp + 1) * p.num_sms;
    int c = 0;
    if (items <= room && room <= p.most_pieces && p.num_groups <= kGroupsHeld) {
      const long long least = (steps + room - 1) / room;
      const int mine = static_cast<int>(least + least * lane / 12 + (least < 12 ? lane : 0));
      long long pieces = 0;
      for (int i = 0; i < p.num_groups; ++i)
        if (held_s[i].keys > 0) pieces += static_cast<long long>(items_of(p, held_s[i])) * ((tiles_of(held_s[i]) + mine - 1) / mine);
      const unsigned fits = __ballot_sync(0xffffffffu, pieces <= room);
      if (fits != 0) c = __shfl_sync(0xffffffffu, mine, __ffs(fits) - 1);
    }
    if (lane == 0) cut_s[warp] = c;
  }
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
    share = sharing_pays(saved, p.Hkv, p.D, cut);
  }
  // the pieces' places, group after group
  for (int i0 = 0; i0 < p.num_groups; i0 += kPlanThreads) {
    const int i = i0 + tid;
    SharedGroup g = {};
    int pieces = 0;
    if (i < p.num_groups) {
      g = group(i);
      if (!share) g.keys = 0;
      if (g.keys > 0) {
        g.shares = (tiles_of(g) + cut - 1) / cut;
        pieces = items_of(p, g) * g.shares;
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
    if (i < p.num_groups) {
      p.groups[i] = g;
      if (i < kGroupsHeld) held_s[i] = g;
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) base_s = before + upto;
    __syncthreads();
  }
  if (tid == 0) *p.pieces = base_s;
  // the sequences: in which group, if it shares (a member shorter than the shared part does not)
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const int T = context(b), i = share ? group_of(b) : -1;
    int4 out = make_int4(0, 0, 0, 0);
    if (i >= 0) {
      const SharedGroup g = group(i);
      if (b < g.first + g.members && g.keys > 0 && T >= g.keys) out = make_int4(g.keys, g.base, g.shares, b - g.first);
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
  piece.table_row = g.row;
  piece.kv_lo = g.lo;
  piece.o = sp.piece_o + static_cast<size_t>(k) * (D / 4) * 128;
  piece.lse = sp.piece_lse + static_cast<size_t>(k) * 128;
  attend_tile<D, WIN, kPieces>(p, tmk, tmv, g.first, g.members, g.keys, tile, at - item * g.shares, g.shares, piece);
}

constexpr int kJoinThreads = 512;

// CTA per (sequence, unit of the decode): a thread takes four columns of a head, heads next to one another (as they lie in the prefix's
// pieces), and every PARTS-th piece, eight of them on their way at a time; the threads' maxima, sums and columns are put together in
// shared memory.  What bounds it are its round trips to L2 (the sequence's numbers, its pieces, once or twice).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const SharedParams p, int units, int G) {
  constexpr int U = 8;
  __shared__ float top_s[kJoinThreads], sum_s[kJoinThreads];
  __shared__ float4 o_s[kJoinThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / units, u = blockIdx.x - b * units;
  const int4 info = p.info[b];
  if (info.x == 0) return;
  int2 own = p.units[blockIdx.x];
  if (context_of(p, b) <= info.x) own = make_int2(0, 0);  // (not written)
  const float* own_lse = p.lse_part + (static_cast<long long>(own.x) + blockIdx.x) * G;
  const float4* own_o = reinterpret_cast<const float4*>(p.o_part + (static_cast<long long>(own.x) + blockIdx.x) * G * D);
  const int quads = G * D / 4, parts = kJoinThreads / quads;  // (quads: a power of two from 16 to 512)
  const int part = threadIdx.x / quads, q = threadIdx.x - part * quads, d4 = q / G, h = q - d4 * G;
  // head h of the unit among the rows of the prefix's pieces: the first one's CTA, and the row
  const int group = p.Hq / p.Hkv, tile = info.w / p.tok, head = u * G + h, g = head / group;
  const int row = (info.w - tile * p.tok) * group + head - g * group, k0 = info.y + (tile * p.Hkv + g) * info.z;
  float top = -kHuge, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = part; i0 < info.z + own.y; i0 += U * parts) {
    float lse[U];
    float4 x[U];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int i = i0 + v * parts, j = i - info.z;
      lse[v] = -INFINITY;
      x[v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < 0) {
        lse[v] = p.piece_lse[static_cast<size_t>(k0 + i) * 128 + row];
        x[v] = p.piece_o[(static_cast<size_t>(k0 + i) * (D / 4) + d4) * 128 + row];
      } else if (j < own.y) {
        lse[v] = own_lse[static_cast<size_t>(j) * G + h];
        x[v] = own_o[(static_cast<size_t>(j) * G + h) * (D / 4) + d4];
      }
    }
    float m = top;
#pragma unroll
    for (int v = 0; v < U; ++v) m = fmaxf(m, lse[v]);
    const float a = ex2(top - m);  // (of -kHuge: 1 or 0)
    top = m;
    sum *= a;
    o.x *= a, o.y *= a, o.z *= a, o.w *= a;
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const float w = ex2(lse[v] - m);  // (a piece of NaN has lse +infinity: NaN)
      sum += w;
      o.x = fmaf(w, x[v].x, o.x);
      o.y = fmaf(w, x[v].y, o.y);
      o.z = fmaf(w, x[v].z, o.z);
      o.w = fmaf(w, x[v].w, o.w);
    }
  }
  top_s[threadIdx.x] = top;
  sum_s[threadIdx.x] = sum;
  o_s[threadIdx.x] = o;
  __syncthreads();
  if (part > 0) return;
  for (int i = 1; i < parts; ++i) top = fmaxf(top, top_s[i * quads + q]);
  sum = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < parts; ++i) {
    const int at = i * quads + q;
    const float w = ex2(top_s[at] - top);
    sum = fmaf(w, sum_s[at], sum);
    o.x = fmaf(w, o_s[at].x, o.x);
    o.y = fmaf(w, o_s[at].y, o.y);
    o.z = fmaf(w, o_s[at].z, o.z);
    o.w = fmaf(w, o_s[at].w, o.w);
  }
  const float inv = 1.f / sum;
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out + (static_cast<size_t>(b) * p.Hq + head) * D + 4 * d4);
  dst[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  dst[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
}

// CTAs of the prefix kernel.  Items (groups of two and more have them), at most; where an SM can have two each, the SMs, and otherwise
// three for every SM or one for every item.
long long prefix_ctas(int B, int Hq, int Hkv, int num_groups, int num_sms) {
  const int tok = 128 / (Hq / Hkv);
  const long long items = static_cast<long long>(Hkv) * (B / tok + std::min(num_groups, B / 2));
  return 2 * items <= num_sms ? num_sms : std::max<long long>(3LL * num_sms, items);
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
  uint8_t* least = part(static_cast<size_t>(num_groups) * sizeof(unsigned long long));
  uint8_t* pieces = part(sizeof(int));
  uint8_t* info = part(static_cast<size_t>(B) * sizeof(int4));
  uint8_t* units = part(static_cast<size_t>(B) * Hkv * 2 * sizeof(int2));
  uint8_t* lse = part(static_cast<size_t>(ctas) * 128 * sizeof(float));
  uint8_t* o = part(static_cast<size_t>(ctas) * 128 * D * sizeof(float));
  if (p) {
    p->groups = reinterpret_cast<SharedGroup*>(groups);
    p->least = reinterpret_cast<unsigned long long*>(least);
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
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != C::REG_LAUNCH) return cudaErrorInvalidKernelImage;
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
  // (keys that a group can save, whatever the groups are)
  const long long keys = std::min(dp.max_blocks * 16LL, dp.window > 0 ? static_cast<long long>(dp.window) : INT64_MAX);
  if (!sharing_pays((dp.B - 1) * keys, dp.Hkv >> dp.halves, D, 1)) return launch_block_decode(dp, D, ctas, s);
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
  sp.most_pieces = static_cast<int>(prefix);
  lay_out(&sp, static_cast<uint8_t*>(workspace), dp.B, sp.Hq, sp.Hkv, D, num_groups, prefix);
  dp.shared = sp.info;
  dp.units = sp.units;
  if (D == 64) return launch_d<64>(dp, sp, ctas, static_cast<int>(prefix), s);
  if (D == 128) return launch_d<128>(dp, sp, ctas, static_cast<int>(prefix), s);
  return launch_d<256>(dp, sp, ctas, static_cast<int>(prefix), s);
}

}  // namespace fkv
