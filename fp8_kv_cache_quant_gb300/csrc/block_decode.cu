// Launches of the decode attention over a block-scaled cache (block_decode_kernel.cuh).
#include "block_decode_kernel.cuh"

namespace fkv {
namespace {

template <int D, int G>
cudaError_t launch_t(const BlockDecodeParams& p, int N, cudaStream_t s) {
  using C = BlockDecodeCfg<D, G>;
  CUtensorMap tmk, tmv;
  if (!make_pool_map(&tmk, const_cast<uint8_t*>(p.k_cache), D, p.Hkv >> p.halves, p.num_blocks, C::RB) ||
      !make_pool_map(&tmv, const_cast<uint8_t*>(p.v_cache), D, p.Hkv >> p.halves, p.num_blocks, C::RB))
    return cudaErrorInvalidValue;
  auto kern = block_decode_kernel<D, G, false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(N), dim3(kThreads), C::SMEM, s, p, tmk, tmv);
}

template <int D>
cudaError_t launch_g(const BlockDecodeParams& p, int G, int N, cudaStream_t s) {
  switch (G) {
    case 1: return launch_t<D, 1>(p, N, s);
    case 2: return launch_t<D, 2>(p, N, s);
    case 4: return launch_t<D, 4>(p, N, s);
    case 8: return launch_t<D, 8>(p, N, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int block_decode_ctas_per_sm(int D) { return D <= 128 ? 2 : 1; }

int block_decode_tile_blocks(int D) { return D == 64 ? 16 : 8; }

cudaError_t launch_block_decode(const BlockDecodeParams& p, int D, int N, cudaStream_t s) {
  const int G = p.Hq / p.Hkv;
  if (D == 64) return launch_g<64>(p, G, N, s);
  if (D == 128) return launch_g<128>(p, G, N, s);
  if (D == 256) return launch_g<256>(p, G, N, s);
  return cudaErrorInvalidValue;
}

}  // namespace fkv
