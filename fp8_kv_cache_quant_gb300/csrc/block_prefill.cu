// Prefill (chunked) attention over a block-scaled e4m3 cache: which CTAs take which tiles of queries (block_attend.cuh).
#include <atomic>

#include "block_attend.cuh"

namespace fkv {
namespace {

// Whether a sequence's query tiles gain from sharing their key tiles in clusters of two where that evens out the last
// wave: a chunk over a context long enough for its CTAs to be alike (2,048 queries, 32/8 heads, head_dim 128, us shared and
// not: over 8,192 keys 334 and 307, over 12,288 467 and 463, over 16,384 600 and 622).
__host__ __device__ constexpr bool sharing_pays(long long keys, long long queries) { return keys >= 6 * queries && keys >= 8192; }

template <int D, bool WIN, bool SPLIT>
__global__ void __launch_bounds__(512, 1)
    block_prefill_kernel(const __grid_constant__ BlockPrefillParams p, const __grid_constant__ CUtensorMap tmk,
                         const __grid_constant__ CUtensorMap tmv) {
  const int b = blockIdx.z;
  // Launched with programmatic stream serialisation.  The tensor memory, all of an SM's, is allocated
  // after this wait: taken before, it could be what a CTA of the kernel before still needs to go on.
  griddep_wait();

  // ------------------------------------------------------------ sequence geometry
  const bool first_cta = blockIdx.x == gridDim.x - 1 && blockIdx.y == 0 && threadIdx.x == 0;
  const int r0 = p.cu[b];
  const int Lq = p.cu[b + 1] - r0;
  int T = p.ctx[b];
  if (T < 0 || T > static_cast<long long>(p.max_blocks) * 16) {
    if (first_cta) raise_fault(p.fault, FKV_FAULT_CONTEXT);
    T = T < 0 ? 0 : p.max_blocks * 16;
  }
  if (Lq < 0 || Lq > p.max_q_len || (p.causal && Lq > T) || r0 < 0 || r0 + static_cast<long long>(Lq) > p.total_q) {
    if (first_cta) raise_fault(p.fault, FKV_FAULT_QLEN);
    return;
  }
  // longest (latest) query tiles first
  const int at = static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x);
  if constexpr (!SPLIT) {
    if (at * p.part_tokens < Lq) attend_tile<D, WIN, kAlone>(p, tmk, tmv, r0, Lq, T, at, 0, 1);
  } else {
    // a cluster per query tile, or, where clusters are there for the last wave's sake, a CTA per query tile for the
    // sequences that do not gain from sharing
    const int size = static_cast<int>(cluster_size());
    if (D > 128 || !p.even_waves || sharing_pays(WIN ? min(static_cast<long long>(T), p.window + 256LL) : T, Lq)) {
      const int qt = at / size;
      if (qt * p.part_tokens < Lq) attend_tile<D, WIN, kClusters>(p, tmk, tmv, r0, Lq, T, qt, static_cast<int>(cluster_rank()), size);
    } else {
      const int qt = at - static_cast<int>(gridDim.x) + static_cast<int>(gridDim.x) / size;
      if (qt >= 0 && qt * p.part_tokens < Lq) attend_tile<D, WIN, kAlone>(p, tmk, tmv, r0, Lq, T, qt, 0, 1);
    }
  }
}

template <int D, bool WIN, bool SPLIT>
cudaError_t launch_t(const BlockPrefillParams& p, dim3 grid, int shares, cudaStream_t s) {
  using C = BlockPrefillCfg<D>;
  CUtensorMap tmk, tmv;
  if (!make_pool_map(&tmk, const_cast<uint8_t*>(p.k_cache), D, p.Hkv, p.num_blocks, C::RB) ||
      !make_pool_map(&tmv, const_cast<uint8_t*>(p.v_cache), D, p.Hkv, p.num_blocks, C::RB))
    return cudaErrorInvalidValue;
  auto kern = block_prefill_kernel<D, WIN, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // the warpgroups' register budgets add up to the launch's 128 per thread: a kernel built with
  // fewer would wait forever in setmaxnreg.inc, so it is never launched
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, kern);
    if (e != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != C::REG_LAUNCH) return cudaErrorInvalidKernelImage;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = shares;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, tmk, tmv);
}

// Clusters of that many CTAs that the current device holds at once: fewer than its SMs over the size, since
// a cluster stays within a group of SMs.  Asked once per device and size.
template <int D, bool WIN>
int clusters_at_once(int shares) {
  using C = BlockPrefillCfg<D>;
  constexpr int kDevices = 16;
  static std::atomic<int> known[kDevices][9];  // the number plus 1
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kDevices && (n = known[dev][shares].load(std::memory_order_relaxed)) != 0) return n - 1;
  auto kern = block_prefill_kernel<D, WIN, true>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(shares);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = shares;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
  if (dev < kDevices) known[dev][shares].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int D, bool WIN>
cudaError_t launch_w(BlockPrefillParams p, dim3 grid, long long ctas, int num_sms, cudaStream_t s) {
  // the table's width bounds the contexts from above; the kernel knows them, and shares no more than they are worth
  const long long keys = WIN ? std::min<long long>(p.max_blocks * 16LL, static_cast<long long>(p.window) + 256) : p.max_blocks * 16LL;
  // CTAs that would leave SMs idle share their key tiles, two at least each, in clusters as large as can
  // all be there at once
  int shares = static_cast<int>(std::max<long long>(1, std::min<long long>(std::min<long long>(8, num_sms / ctas), keys / 256)));
  while (shares > 1 && ctas > clusters_at_once<D, WIN>(shares)) --shares;
  // Clusters of two also even out the last wave of a chunk over a long context, where that saves more than
  // sharing costs: over 32,768 keys (32/8 heads, head_dim 128) 1,500 queries take 822 us against 956, 2,048
  // 1,133 against 1,255; not 1,024 (657 against 648) or 3,000 (1,602 against 1,569).
  const long long waves = (ctas + num_sms - 1) / num_sms, half_waves = (2 * ctas + num_sms - 1) / num_sms;
  p.even_waves = D <= 128 && waves > 1 && sharing_pays(keys, p.max_q_len) && half_waves * 108 < waves * 200;
  if (p.even_waves) shares = 2;
  if (shares == 1) return launch_t<D, WIN, false>(p, grid, 1, s);
  grid.x *= shares;
  return launch_t<D, WIN, true>(p, grid, shares, s);
}

template <int D>
cudaError_t launch_d(const BlockPrefillParams& p, dim3 grid, long long ctas, int num_sms, cudaStream_t s) {
  return p.window > 0 ? launch_w<D, true>(p, grid, ctas, num_sms, s) : launch_w<D, false>(p, grid, ctas, num_sms, s);
}

}  // namespace

cudaError_t launch_block_prefill(BlockPrefillParams p, int D, int num_sms, cudaStream_t s) {
  // the group's heads in as few equal parts of at most 128 as there can be; whole tokens per CTA
  const int G = p.Hq / p.Hkv;
  p.head_parts = (G + 127) / 128;
  p.part_heads = (G + p.head_parts - 1) / p.head_parts;
  p.part_tokens = 128 / p.part_heads;
  const int tok = p.part_tokens;
  const long long y = static_cast<long long>(p.Hkv) * p.head_parts;
  if (y > 65535) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((p.max_q_len - 1LL) / tok + 1), static_cast<unsigned>(y), p.B);
  // CTAs that have rows, at most: of a ragged batch, far fewer than the grid's
  const long long ctas = std::min<long long>(static_cast<long long>(grid.x) * p.B, static_cast<long long>(p.total_q) / tok + p.B) * y;
  if (D == 64) return launch_d<64>(p, grid, ctas, num_sms, s);
  if (D == 128) return launch_d<128>(p, grid, ctas, num_sms, s);
  return launch_d<256>(p, grid, ctas, num_sms, s);
}

}  // namespace fkv
