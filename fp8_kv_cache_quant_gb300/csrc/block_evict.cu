// Eviction from a block-scaled cache by accumulated attention weight: per (sequence, KV head) the
// tokens that stay are found (evict_select_kernel), then copied to the sequence's new blocks with
// scales of their own (evict_gather_kernel).
//
// Selection.  Of T weights the n = min(T, budget) largest stay, equal ones by ascending index; the first
// `sink` and the last `recent` tokens count as larger than any weight.  Weights become 32-bit keys that order
// like the numbers (NaN below everything), and the n-th largest key is found digit by digit, from the top, 11, 11 and 10
// bits, with a histogram of the keys that share the digits found so far: three counts of T keys whatever the weights are.
// A last walk in index order numbers the kept ones.
// A unit (sequence, KV head) is a cluster of CTAs, each with a consecutive share of its keys in shared memory (so that
// the weights are read from HBM once), whose histograms meet through distributed shared memory.  Of every 32 keys two words
// say which are above the digits found so far, and which share them: the walks behind the first look at the latter alone.
//
// What bounds it: 32 keys and fewer a thread, so its chain of walks, barriers and round trips through distributed shared memory.  8 heads
// of 8 sequences of 16k-24k tokens (two CTAs a unit) 16 us, of one of 131,072 (eight) 20, kept to 4,096 and 32,768; reading the weights
// alone takes 1.
//
// Copy.  A warp per (new block, KV head): 16 kept tokens' K and V rows from anywhere, their largest finite
// magnitude, the block's new scale as an append of the same values to an empty block would choose it, the codes brought to it.
#include <atomic>
#include <type_traits>

#include "block_common.cuh"

namespace fkv {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMaxResident = 40960;  // keys of a CTA held in shared memory, at most (160 KB, and 10 KB of masks)

FKV_DEV uint32_t rank_in_cluster() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
FKV_DEV uint32_t ctas_of_cluster() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster: earlier writes of all are visible behind it.
FKV_DEV void arrive_cluster() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
FKV_DEV void wait_cluster() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
FKV_DEV void sync_cluster() {
  arrive_cluster();
  wait_cluster();
}
FKV_DEV void peer_add(int* p, uint32_t rank, int v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
FKV_DEV int2 peer_int2(const int* p, uint32_t rank) {
  uint32_t a;
  int2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// A key that orders like the weight, NaN below all; tokens that always stay take the top one, which no weight has.
constexpr uint32_t kSure = 0xFFFFFFFFu;
FKV_DEV uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // (-0 is 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectShared {
  int hist[3][kBins];    // this CTA's keys
  int total[3][kBins];   // the cluster's (of the second digit: of the pairs of bins that are this CTA's to sum)
  int warp_sum[32], warp_eq[32];
  int digit, left;       // of the last histogram: the digit, and what is to be taken of it
  int gt_eq[2];          // this CTA's keys above the threshold, and equal to it
  uint2 masks[kMaxResident / 32];  // of 32 keys each
};
constexpr int kMaxCluster = 8;
constexpr int kLoads = 8;  // weights that a thread has on their way

__global__ void __launch_bounds__(kSelectThreads, 1) evict_select_kernel(const EvictParams p, int resident_keys) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelectShared& sh = *reinterpret_cast<SelectShared*>(smem);
  uint32_t* held = reinterpret_cast<uint32_t*>(smem + sizeof(SelectShared));  // this CTA's keys
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(ctas_of_cluster()), rank = static_cast<int>(rank_in_cluster());
  for (int i = tid; i < 6 * kBins; i += kSelectThreads) (&sh.hist[0][0])[i] = 0;
  if (C > 1) arrive_cluster();  // (waited for before the first access to another CTA)
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x / C;
  const int b = unit / p.H, h = unit - b * p.H;
  const long long most = min(p.max_blocks * 16LL, static_cast<long long>(p.weights_len));
  int T = p.ctx[b];
  if (T < 0 || T > most) {
    if (h == 0 && rank == 0 && tid == 0) raise_fault(p.fault, FKV_FAULT_CONTEXT);
    T = T < 0 ? 0 : static_cast<int>(most);
  }
  const int n = min(T, p.budget);
  if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = n;
  int32_t* kept = p.kept + static_cast<size_t>(unit) * p.budget;
  const float* weights = p.weights + static_cast<size_t>(unit) * p.weights_len;
  float* moved = p.new_weights ? p.new_weights + static_cast<size_t>(unit) * p.new_weights_len : nullptr;
  const int all = C * kSelectThreads, me = rank * kSelectThreads + tid;
  // (budgets and contexts go up to 2^31 - 1 and 2^31 - 1024: a step of all threads behind them passes 32 bits)
  for (long long i = n + static_cast<long long>(me); i < p.budget; i += all) kept[i] = -1;
  if (T <= p.budget) {  // (the whole cluster)
    if (C > 1) wait_cluster();
    for (long long i = me; i < n; i += all) {
      kept[i] = static_cast<int>(i);
      if (moved) moved[i] = weights[i];
    }
    return;
  }
  // this CTA's keys [lo, hi)
  const int seg = ((T + C - 1) / C + 31) & ~31;
  const int lo = min(rank * seg, T), hi = min(lo + seg, T);
  const bool resident = seg <= resident_keys;
  auto key_of_token = [&](int i, float w) -> uint32_t { return i < p.sink || i >= T - p.recent ? kSure : key_of(w); };
  __syncthreads();
  for (int left0 = hi - lo - tid; left0 > 0; left0 -= kLoads * kSelectThreads) {  // (keys from this thread's next on)
    const int i0 = hi - left0;
    float w[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) w[j] = j * kSelectThreads < left0 ? weights[i0 + j * kSelectThreads] : 0.f;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      if (j * kSelectThreads >= left0) break;
      const int i = i0 + j * kSelectThreads;
      const uint32_t k = key_of_token(i, w[j]);
      if (resident) held[i - lo] = k;
      atomicAdd(&sh.hist[0][k >> 21], 1);
    }
  }
  // warp w walks the keys [wlo, whi), 32 at a time
  const int wseg = (((hi - lo + 31) / 32) + 31) & ~31;
  const int wlo = min(lo + warp * wseg, hi), whi = min(wlo + wseg, hi);
  // Of every 32 keys (i0 ...) those whose digits from bit `shift` up are above `found`, and those that have them, to act(i0, masks, the
  // lane's key where it is one of the latter).  Behind the first walk, words without any of the latter are passed over, `all` aside.
  auto walk = [&](auto first, auto all, int shift, uint32_t found, auto act) {
    if (!resident) {
      for (int i0 = wlo; i0 < whi; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < whi ? key_of_token(i, weights[i]) : 0u, d = k >> shift;
        act(i0, make_uint2(__ballot_sync(0xffffffffu, i < whi && d > found), __ballot_sync(0xffffffffu, i < whi && d == found)), k);
      }
      return;
    }
    const uint32_t* keys = held + (wlo - lo) + lane;
    uint2* masks = sh.masks + ((wlo - lo) >> 5);
    const int words = (whi - wlo + 31) >> 5, rest = whi - wlo - lane;  // keys of this lane at 0, 32, ... below rest
    if constexpr (decltype(first)::value) {
#pragma unroll 4
      for (int x = 0; x < words; ++x) {
        const bool in = 32 * x < rest;
        const uint32_t k = in ? keys[32 * x] : 0u, d = k >> shift;
        const uint2 m = make_uint2(__ballot_sync(0xffffffffu, in && d > found), __ballot_sync(0xffffffffu, in && d == found));
        if (lane == 0) masks[x] = m;
        act(wlo + 32 * x, m, k);
      }
    } else {
      for (int x0 = 0; x0 < words; x0 += 32) {  // a word per lane
        uint2 mine = x0 + lane < words ? masks[x0 + lane] : make_uint2(0u, 0u);
        for (unsigned some = __ballot_sync(0xffffffffu, mine.y != 0); some != 0; some &= some - 1) {
          const int at = __ffs(some) - 1, x = x0 + at;
          const uint32_t y = __shfl_sync(0xffffffffu, mine.y, at);
          const bool in = y >> lane & 1u;
          const uint32_t k = in ? keys[32 * x] : 0u, d = k >> shift;
          uint2 m = make_uint2(__ballot_sync(0xffffffffu, in && d > found), __ballot_sync(0xffffffffu, in && d == found));
          if (lane == at) mine = make_uint2(mine.x | m.x, m.y);
          if constexpr (!decltype(all)::value) act(wlo + 32 * x, m, k);
        }
        if constexpr (decltype(all)::value) act(x0, mine, 0u);
        if (x0 + lane < words) masks[x0 + lane] = mine;
      }
    }
    __syncwarp();
  };
  int left = n;        // keys to take among those that share the digits found so far
  uint32_t found = 0;  // these digits
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    if (pass > 0) {
      if (pass == 1)
        walk(std::true_type(), std::false_type(), 21, found, [&](int, uint2 m, uint32_t k) {
          if (m.y >> lane & 1u) atomicAdd(&sh.hist[1][k >> 10 & 2047u], 1);
        });
      else
        walk(std::false_type(), std::false_type(), 10, found, [&](int, uint2 m, uint32_t k) {
          if (m.y >> lane & 1u) atomicAdd(&sh.hist[2][k & 1023u], 1);
        });
    }
    __syncthreads();
    // thread t: the t-th pair of bins from the top.  Where few bins are taken (a key's exponent and first digits, and what is left in the
    // end) every CTA adds its own to all CTAs' totals; in between, where most are, pair x is summed in CTA x % C alone and read there
    // (131k keys of a unit, cycles added to all and to one: 3,900 and 5,000, 15,000 and 5,400, 3,600 and 6,100).
    const int hi_bin = kBins - 1 - 2 * tid;
    int c0 = sh.hist[pass][hi_bin], c1 = sh.hist[pass][hi_bin - 1];
    if (C > 1) {
      if (pass == 0) wait_cluster();
      const int owner = tid & (C - 1);
      for (int r = pass == 1 ? owner : 0; r <= (pass == 1 ? owner : C - 1); ++r) {
        if (c0 != 0) peer_add(&sh.total[pass][hi_bin], r, c0);
        if (c1 != 0) peer_add(&sh.total[pass][hi_bin - 1], r, c1);
      }
      sync_cluster();
      int2 x = *reinterpret_cast<const int2*>(&sh.total[pass][hi_bin - 1]);
      if (pass == 1) x = peer_int2(&sh.total[pass][hi_bin - 1], owner);
      c0 = x.y;
      c1 = x.x;
    }
    int upto = c0 + c1;  // inclusive sums over the threads
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    int before = upto - c0 - c1;
    {
      const int x = lane < warp ? sh.warp_sum[lane] : 0;
      before += __reduce_add_sync(0xffffffffu, x);
    }
    if (before < left && left <= before + c0) {
      sh.digit = hi_bin;
      sh.left = left - before;
    } else if (before + c0 < left && left <= before + c0 + c1) {
      sh.digit = hi_bin - 1;
      sh.left = left - before - c0;
    }
    __syncthreads();
    found = pass < 2 ? found << 11 | sh.digit : found << 10 | sh.digit;
    left = sh.left;
  }
  // of the keys equal to the threshold `found` the first `left` stay
  int gt = 0, eq = 0;
  walk(std::false_type(), std::true_type(), 0, found, [&](int, uint2 m, uint32_t) {  // (resident: a word per lane)
    gt += __popc(m.x);
    eq += __popc(m.y);
  });
  if (resident) {
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
  }
  if (lane == 0) {
    sh.warp_sum[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  // above and equal: in the warps before this one, in the CTA, and in the CTAs before it
  int gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0), eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_eq[lane] : 0);
  const int gt_cta = __reduce_add_sync(0xffffffffu, sh.warp_sum[lane]), eq_cta = __reduce_add_sync(0xffffffffu, sh.warp_eq[lane]);
  int gt_peers = 0, eq_peers = 0;
  if (C > 1) {
    if (tid == 0) {
      sh.gt_eq[0] = gt_cta;
      sh.gt_eq[1] = eq_cta;
    }
    sync_cluster();
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      if (r >= rank) break;
      const int2 x = peer_int2(sh.gt_eq, r);
      gt_peers += x.x;
      eq_peers += x.y;
    }
    arrive_cluster();  // (the last access to another CTA)
  }
  eq_before += eq_peers;
  const int base = gt_peers + min(eq_peers, left);  // this CTA's first place
  int at = gt_peers + gt_before + min(eq_before, left);
  if (resident && wseg >= 256) {
    // the tokens that stay into a list over the keys, a word per lane, and from there in order: 4,800 cycles for 16,384 keys of a CTA
    // (straight from the masks, stores of a few lanes each: 9,000; for 1,536 keys 1,500 against 3,700, most lanes without a word)
    int* list = reinterpret_cast<int*>(held);
    const int words = (whi - wlo + 31) >> 5;
    for (int x0 = 0; x0 < words; x0 += 32) {
      const uint2 m = x0 + lane < words ? sh.masks[((wlo - lo) >> 5) + x0 + lane] : make_uint2(0u, 0u);
      int eq_to = __popc(m.y);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, eq_to, off);
        if (lane >= off) eq_to += x;
      }
      uint32_t y = m.y;
      for (int over = min(eq_before + eq_to - left, __popc(y)); over > 0; --over) y &= ~(0x80000000u >> __clz(y));
      uint32_t keeps = m.x | y;
      int to = __popc(keeps);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, to, off);
        if (lane >= off) to += x;
      }
      const int sum = __shfl_sync(0xffffffffu, to, 31);
      to += at - base - __popc(keeps);
      for (; keeps != 0; keeps &= keeps - 1) list[to++] = wlo + 32 * (x0 + lane) + __ffs(keeps) - 1;
      at += sum;
      eq_before += __shfl_sync(0xffffffffu, eq_to, 31);
    }
    __syncthreads();
    const int count = gt_cta + min(eq_peers + eq_cta, left) - min(eq_peers, left);
#pragma unroll 4
    for (int j = tid; j < count; j += kSelectThreads) {
      const int i = list[j];
      kept[base + j] = i;
      if (moved) moved[base + j] = weights[i];
    }
  } else {
    const uint32_t below = (1u << lane) - 1u;
    auto put = [&](int i0, uint2 m) {
      uint32_t keeps = m.x | m.y;
      if (eq_before + __popc(m.y) > left)
        keeps = __ballot_sync(0xffffffffu, m.x >> lane & 1u || (m.y >> lane & 1u && eq_before + __popc(m.y & below) < left));
      if (keeps >> lane & 1u) {
        const int i = i0 + lane, to = at + __popc(keeps & below);
        kept[to] = i;
        if (moved) moved[to] = weights[i];
      }
      at += __popc(keeps);
      eq_before += __popc(m.y);
    };
    if (resident) {
#pragma unroll 4
      for (int i0 = wlo; i0 < whi; i0 += 32) put(i0, sh.masks[(i0 - lo) >> 5]);
    } else {
      walk(std::false_type(), std::false_type(), 0, found, [&](int i0, uint2 m, uint32_t) { put(i0, m); });
    }
  }
  if (C > 1) wait_cluster();  // no CTA leaves while another reads its shared memory
}

constexpr int kGatherThreads = 256;

// Four codes as float32 values times s (rounded to float32).
FKV_DEV void values4(uint32_t w, float s, float (&x)[4]) {
  uint32_t h01, h23;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"(static_cast<uint16_t>(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h23));
  x[0] = __fmul_rn(a.x, s);
  x[1] = __fmul_rn(a.y, s);
  x[2] = __fmul_rn(b.x, s);
  x[3] = __fmul_rn(b.y, s);
}

// Four codes times r in binary16, as codes.
FKV_DEV uint32_t scaled4(uint32_t w, __half2 r) {
  uint32_t out;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 a, b;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 a, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 b, hi;\n\t"
      "mul.rn.f16x2 a, a, %2;\n\t"
      "mul.rn.f16x2 b, b, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 lo, a;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hi, b;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(out)
      : "r"(w), "r"(*reinterpret_cast<const uint32_t*>(&r)));
  return out;
}

// The largest magnitude code of 16 (NaN, 0x7F, the largest of all).
FKV_DEV uint32_t top_code(uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, __vmaxu2(w[i] & 0x007F007Fu, w[i] >> 8 & 0x007F007Fu));
  return max(m & 0xFFFFu, m >> 16);
}

// Four values of the row's scale s as codes of the scale `to`, inv = 1 / to.
FKV_DEV uint32_t recode4(uint32_t w, float s, float inv) {
  float y[4];
  values4(w, s, y);
  return f32x4_to_e4m3x4(make_float2(__fmul_rn(y[0], inv), __fmul_rn(y[1], inv)), make_float2(__fmul_rn(y[2], inv), __fmul_rn(y[3], inv)));
}

// Warps go from item to item (new block, KV head): while the rows of one are on their way, the table entries of the next and the kept
// indices of the one behind it are read, so that an item costs one round trip to memory instead of four.
template <int D>
__global__ void __launch_bounds__(kGatherThreads, D <= 128 ? 4 : 2) evict_gather_kernel(const EvictParams p, int blocks) {
  constexpr int CPR = D / 16;          // 16-byte chunks of a row
  constexpr int N = 16 * CPR / 32;     // chunks per lane of K, and of V
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long items = static_cast<long long>(p.B) * p.H * blocks, step = static_cast<long long>(gridDim.x) * (kGatherThreads / 32);
  struct Item {
    int b, blk, h, n;     // n: rows of the block, 0: none
  };
  auto item_at = [&](long long x) -> Item {
    Item t = {0, 0, 0, 0};
    if (x >= items) return t;
    t.h = static_cast<int>(x % p.H);
    const long long rest = x / p.H;
    t.blk = static_cast<int>(rest % blocks);
    t.b = static_cast<int>(rest / blocks);
    t.n = min(16, p.new_lens[t.b] - 16 * t.blk);
    return t;
  };
  // lane r < 16: row r's old index, then its block (and the new block); -1: none
  auto index_of = [&](const Item& t) -> int { return lane < t.n ? p.kept[(static_cast<size_t>(t.b) * p.H + t.h) * p.budget + 16 * t.blk + lane] : -1; };
  auto block_of = [&](const Item& t, int i) -> int { return i >= 0 ? p.block_table[static_cast<size_t>(t.b) * p.max_blocks + (i >> 4)] : 0; };
  auto target_of = [&](const Item& t) -> int { return t.n > 0 ? p.new_table[static_cast<size_t>(t.b) * p.new_max_blocks + t.blk] : 0; };
  long long x = static_cast<long long>(blockIdx.x) * (kGatherThreads / 32) + (threadIdx.x >> 5);
  Item now = item_at(x), next = item_at(x + step);
  int i_now = index_of(now), i_next = index_of(next);
  int id = block_of(now, i_now), dst = target_of(now);
  for (; x < items; x += step) {
    const Item t = now;
    const int slot = i_now & 15, to = dst;
    if (lane < t.n && (id < 0 || id >= p.num_blocks)) {
      raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
      id = 0;
    }
    const size_t src_row = static_cast<size_t>(id) * p.H + t.h;
    float ks = 0.f, vs = 0.f;
    if (lane < t.n) {
      ks = p.ks[src_row];
      vs = p.vs[src_row];
    }
    uint4 k[N], v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = lane + 32 * j, row = c / CPR;
      const int b = __shfl_sync(0xffffffffu, id, row), s = __shfl_sync(0xffffffffu, slot, row);
      k[j] = v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (row < t.n) {
        const size_t at = ((static_cast<size_t>(b) * p.H + t.h) * 16 + s) * CPR + c % CPR;
        k[j] = reinterpret_cast<const uint4*>(p.kc)[at];
        v[j] = reinterpret_cast<const uint4*>(p.vc)[at];
      }
    }
    now = next;
    i_now = i_next;
    next = item_at(x + 2 * step);
    id = block_of(now, i_now);
    dst = target_of(now);
    i_next = index_of(next);
    if (t.n <= 0) continue;
    if (to < 0 || to >= p.num_blocks) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
      continue;
    }
    const size_t at = static_cast<size_t>(to) * p.H + t.h;
    auto store = [&](uint4 (&x4)[N], float scale_of_row, uint8_t* pool, float* scale) {
      // Magnitudes order as their codes, so a chunk's largest is found among the codes.  Where a row holds a NaN, or a scale is
      // no finite number that keeps its products finite, value by value: what is not finite does not count.
      float s[N];
      uint32_t amax = 0;  // bits of the largest finite magnitude
      bool odd = false;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s[j] = __shfl_sync(0xffffffffu, scale_of_row, (lane + 32 * j) / CPR);
        const uint32_t top = top_code(x4[j]);
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(top)));
        const uint32_t m = __float_as_uint(__fmul_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu))), s[j])) & 0x7FFFFFFFu;
        odd = odd || top == 0x7Fu || m >= 0x7F800000u;
        amax = max(amax, m);
      }
      if (__any_sync(0xffffffffu, odd)) {
        amax = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t w[4] = {x4[j].x, x4[j].y, x4[j].z, x4[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y[4];
            values4(w[i], s[j], y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t m = __float_as_uint(y[e]) & 0x7FFFFFFFu;
              if (m < 0x7F800000u) amax = max(amax, m);
            }
          }
        }
      }
      amax = __reduce_max_sync(0xffffffffu, amax);
      const float to_scale = pow2_scale(amax);
      const float inv = __frcp_rn(to_scale);
      if (lane == 0) scale[at] = to_scale;
      // Scales that are powers of two: a code times r = s / to_scale is exact in binary16 from r = 2^-24 (below which every code ends at
      // zero) to 2^15, save for what lies 2^-24 and below, where every code has long ended at zero.
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int c = lane + 32 * j;
        const uint32_t sb = __float_as_uint(s[j]);
        const float r = s[j] * inv;
        if (r != 1.f) {
          if ((sb & 0x807FFFFFu) == 0u && sb != 0u && r <= 32768.f) {
            const __half2 rh = __float2half2_rn(r);
            x4[j] = make_uint4(scaled4(x4[j].x, rh), scaled4(x4[j].y, rh), scaled4(x4[j].z, rh), scaled4(x4[j].w, rh));
          } else {
            x4[j] = make_uint4(recode4(x4[j].x, s[j], inv), recode4(x4[j].y, s[j], inv), recode4(x4[j].z, s[j], inv), recode4(x4[j].w, s[j], inv));
          }
        }
        if (c / CPR < t.n) reinterpret_cast<uint4*>(pool)[at * 16 * CPR + c] = x4[j];
      }
    };
    store(k, ks, p.kc, p.ks);
    store(v, vs, p.vc, p.vs);
  }
}

}  // namespace

cudaError_t launch_block_evict(const EvictParams& p, int D, int num_sms, cudaStream_t s) {
  const long long most = std::min(p.max_blocks * 16LL, static_cast<long long>(p.weights_len));
  const long long units = static_cast<long long>(p.B) * p.H;
  // clusters while SMs would idle and a CTA has more keys than its threads take at once
  int C = 1;
  while (C < kMaxCluster && 2 * C * units <= num_sms && most / C > 2 * kSelectThreads) C *= 2;
  const long long seg = ((most + C - 1) / C + 31) & ~31LL;
  const int resident = static_cast<int>(std::min<long long>(seg, kMaxResident));
  const size_t smem = sizeof(SelectShared) + 4 * static_cast<size_t>(resident);
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(SelectShared) + 4 * static_cast<size_t>(kMaxResident)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * C));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = C;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, resident);
  if (e != cudaSuccess) return e;
  const int blocks = static_cast<int>((std::min<long long>(most, p.budget) + 15) / 16);
  if (blocks == 0) return cudaSuccess;
  const long long items = units * blocks;
  auto kern = D == 64 ? evict_gather_kernel<64> : D == 128 ? evict_gather_kernel<128> : evict_gather_kernel<256>;
  static std::atomic<int> known[3];  // CTAs of each that an SM holds, asked once
  std::atomic<int>& k = known[D == 64 ? 0 : D == 128 ? 1 : 2];
  int per_sm = k.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kGatherThreads, 0);
    if (e != cudaSuccess) return e;
    k.store(per_sm, std::memory_order_relaxed);
  }
  const unsigned grid = static_cast<unsigned>(std::min<long long>((items + kGatherThreads / 32 - 1) / (kGatherThreads / 32),
                                                                  static_cast<long long>(per_sm) * num_sms));
  return launch_dependent(kern, dim3(grid), dim3(kGatherThreads), 0, s, p, blocks);
}

}  // namespace fkv
