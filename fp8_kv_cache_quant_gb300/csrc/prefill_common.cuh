// What the kernels of the two prefills (prefill_attn.cu, block_prefill.cu) share: the row maximum of a
// score tile, waits under per-warpgroup register budgets, and a bound on what the compiler moves.
#pragma once
#include "common.cuh"
#include "tc.cuh"

namespace fkv {

constexpr float kLog2E4m3Max = 8.807354922057604f;  // log2(448)

FKV_DEV float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Maximum of N values as a tree of three-input maxima (depth log3 N, rather than a chain
// of N / 2 dependent operations).
template <int N>
FKV_DEV float max_tree(const float* v) {
  if constexpr (N == 1) {
    return v[0];
  } else if constexpr (N == 2) {
    return fmaxf(v[0], v[1]);
  } else {
    constexpr int A = (N + 2) / 3, B = (N - A + 1) / 2;
    return fmax3(max_tree<A>(v), max_tree<B>(v + A), max_tree<N - A - B>(v + A + B));
  }
}

// The waits of the prefill kernels take their timed path inline: warpgroups under different
// register budgets cannot be served by one out-of-line function (and inline waits measured faster in
// fp8_prefill_attn at head_dim 256 too, where the budgets are alike).
FKV_DEV bool pf_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns = kPipeWaitNs) { return wait_ns<true>(bar, parity, limit_ns); }
FKV_DEV bool pf_wait_warp(uint64_t* bar, uint32_t parity) { return wait_warp<true>(bar, parity); }

// An empty statement that "uses and redefines" 32 values: placed after the arithmetic on them,
// it keeps the compiler from moving that arithmetic below the next TMEM load (which would
// keep every chunk's loaded values live at once).
FKV_DEV void pin32(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}

}  // namespace fkv
