// Paged GQA decode attention over a block-scaled e4m3 cache on tcgen05 tensor cores: FP8 products
// with the bf16 query and P each as two e4m3 terms, FP32 accumulation in tensor memory, each
// tile's partial promoted into FP32 registers, the context split evenly over the CTAs.
//
// Mathematics.  With q' = q 2^-k (k per head, so that the row's largest magnitude lies in (224, 448])
// and q' = hi + lo, hi the nearest e4m3 value, the score of key j is
//   x_j = (hi . k8_j + lo . k8_j) * ks[block(j)] * c,   c = 2^k softmax_scale log2(e);
// hi + lo is q' down to 2^-17 of the row's largest element (split4_query).  Per tile, with y_j = x_j + L[block(j)], L = log2 vs, and the tile's maximum R_t of y,
//   P_j = 2^(y_j - R_t) * 448 = hi + lo, hi its leading 3 fraction bits,   O_t = sum_j (hi + lo)_j v8_j,
// and the running state is r' = max(r, R_t), acc = acc 2^(r - r') + O_t 2^(R_t - r'),
// l = l 2^(r - r') + 2^(R_t - r') sum_j P_j / 448 * 2^(o - L[block(j)]); the output 2^o acc / (448 l).  P is taken against the
// largest p vs of the tile's visible keys, whichever key has it: it loses what lies below 2^-17 of
// that, and is otherwise within 2^-8 of its value.  o keeps l within float32's range: block_scales in
// block_common.cuh.
//
// The products are taken transposed, keys and head_dim on the MMA's M side, the G query heads on N:
//   S^T [128 keys][16] = K8 . (hi | lo)^T,   O^T [128 d][16] = V8^T . (hi | lo)^T
// so that the cache tiles are the A operands as TMA lands them; the threads that read S^T and O^T
// add column 8 + h to column h.  (hi and lo accumulating into the same columns instead takes twice
// the products: 68 against 63 us for the layer of 8 x 16k-24k tokens, 32/8 heads, head_dim 128, when it was
// tried.)  head_dim 64: tiles of 256 keys (two S^T products), an M = 64 P.V product whose row r sits
// in TMEM lane 32 (r / 16) + r % 16; otherwise tiles of 128 keys.  A group of 16 heads is two units of
// 8 that read the same K and V.
//
// Work.  The decode reads every cached byte once, so the CTAs should all read the same number.  The
// context lengths are known on the GPU alone (a captured graph replays with others), so the
// split is made there: the tiles of all (sequence, KV head) units in a row, each unit's led by a blank
// one that stands for the time its beginning takes, W places in all; CTA k of N takes places
// floor(k W / N) .. floor((k + 1) W / N) - 1, N the CTAs that are resident at once (or W).  A range that
// spans several units is walked as one pipeline (the copies run ahead across the border).  A unit in
// one piece is written by its CTA; the others' pieces go to the workspace as (o / l, log2-sum-exp),
// piece (k, unit u) at row k + u, and the CTA that completes a unit merges it once it is through with
// its own range (all end at the same time).
//
// CTA = 10 warps:
//   0-3   softmax: the query's terms; per tile thread i owns key i (and 128 + i): score, mask, the
//         heads' tile maxima, P's terms, the factors of acc and O_t;
//   4-7   correction: thread i owns head_dim row i (and 128 + i): acc, then the piece, the merge; and a
//         quarter each of V's copies, whose stage is free when O_t has come;
//   8     K copies (a block per lane) and the tile's scales, read a tile ahead and staged;
//   9     TMEM; polls the barriers and issues S^T and P.V products as they become possible.
//
// What bounds it: HBM, around a fixed 12-15 us of ramp, last pieces and merge (groups of one head: 178 MB of
// head_dim 64 take 40 us, 356 MB of head_dim 128 63, 7.3 TB/s on the difference).  8 x 16k-24k tokens, 32/8
// heads, head_dim 128: 63 us, 5.4 TB/s; 8 x 8k-32k, 64/8 heads, head_dim 64: 47 us (six more when warp 9 copied
// V as well and was busy all the time); one sequence of 4,096: 10.6 us.  Two CTAs per SM with three stages
// of K and V; three CTAs with two stages, at 64 registers, are within 1.5 % of it either way.
// Every wait is bounded in time; a timeout records FKV_FAULT_TIMEOUT, lets the CTA's copies and
// products drain and returns (its pieces are then undefined, its units still counted).
//
// SHARED: the decode of what sequences do not share (block_shared.cu): keys from p.shared[b].x on, and a unit of a sequence
// that shares is not merged here: its pieces, the first one's place and their number in p.units, are left for the join.
#pragma once
#include <type_traits>

#include "block_common.cuh"
#include "tc.cuh"

namespace fkv {
namespace {

template <int D, int G>
struct BlockDecodeCfg {
  static constexpr int BN = D == 64 ? 256 : 128;  // keys per tile
  static constexpr int TPB = BN / 16;             // pool blocks per tile
  static constexpr int NHALF = BN / 128;          // S^T products (M = 128 keys) per tile
  static constexpr int LO = 8;                    // first row (column) of the residual terms
  static constexpr int NP = 2 * LO;               // the MMA's N
  static constexpr int NL = G <= 4 ? 4 : LO;      // columns of a term that are read back
  static constexpr int RB = D < 128 ? D : 128;    // bytes of one swizzled row
  static constexpr int SWZ = RB == 128 ? 2 : 4;   // descriptor swizzle mode (128 / 64 bytes)
  static constexpr int NSUB = D / RB;             // column blocks of a K / V row
  static constexpr int KSUB = BN * RB;            // bytes of one column block of a K / V tile
  static constexpr int KTILE = BN * D;            // bytes of a K or V tile
  static constexpr int MPV = D < 128 ? D : 128;   // M of one P.V product
  static constexpr int NS = D <= 128 ? 3 : 2;  // K / V stages
  static constexpr int QSUB = NP * RB;          // bytes of one column block of the query tile
  // P is stored key by key, MN-major: a key's 16 bytes (8 heads' hi, 8 heads' lo) are one store of the
  // thread that owns the key
  static constexpr int PTILE = BN * 16;
  static constexpr int TM_S = 0;                  // S^T buffers: columns [0, 2 NHALF NP)
  static constexpr int TM_O = 2 * NHALF * NP;     // O_t^T buffers
  static constexpr int TM_COLS = TM_O + 2 * NSUB * NP <= 64 ? 64 : TM_O + 2 * NSUB * NP <= 128 ? 128 : 256;
  // scales of a tile, ring of slots: the K copies run at most NS + 2 tiles ahead of the softmax's
  // release of an S buffer, which follows its reading of the scales
  static constexpr int SCN = NS + 2;
  static constexpr int SCF = 3 * TPB + 4;         // ks [TPB], L [TPB], 2^(o - L) [TPB], o, BlockScale's rare and change
  // shared memory (bytes)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + NSUB * QSUB;
  static constexpr int OFF_K = OFF_P + 2 * PTILE;
  static constexpr int OFF_V = OFF_K + NS * KTILE;
  static constexpr int OFF_RED = OFF_V + NS * KTILE;  // [2][4 warps][LO] floats
  static constexpr int OFF_F = OFF_RED + 2 * 4 * LO * 4;  // factors of acc and O_t [2][2][LO]
  static constexpr int MLF = 2 * LO + 4;                  // r, l [LO] and o of a piece
  static constexpr int OFF_ML = OFF_F + 2 * 2 * LO * 4;   // [2][MLF]
  static constexpr int OFF_QS = OFF_ML + 2 * MLF * 4;     // c of the query rows [LO]
  static constexpr int OFF_SC = OFF_QS + LO * 4;
  static constexpr int OFF_BAR = OFF_SC + SCN * SCF * 4;
  static constexpr int NBAR = 24 + 3 * NS + SCN;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 40;
  static constexpr uint32_t IDESC_QK = idesc_e4m3_f32(128, NP, 0, 0);  // K and query K-major
  static constexpr uint32_t IDESC_PV = idesc_e4m3_f32(MPV, NP, 1, 1);  // V and P MN-major
  static constexpr int CTAS = D <= 128 ? 2 : 1;   // per SM
  static_assert(OFF_K % 1024 == 0 && OFF_P % 1024 == 0 && OFF_BAR % 8 == 0, "tile alignment of the swizzles");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory of the resident CTAs");
};

constexpr int kThreads = 320;

// Keys of sequence b: [lo, T), blocks [blk0, blk_end), n tiles of TPB blocks from blk0.
struct Seq {
  int T, lo, n;
  bool shares;  // SHARED: the sequence's keys before lo are another kernel's
};

template <int TPB, bool SHARED>
FKV_DEV Seq seq_of(const BlockDecodeParams& p, int b, bool report) {
  Seq s;
  s.T = p.ctx[b];
  if (s.T < 0 || s.T > p.max_blocks * 16LL) {
    if (report) raise_fault(p.fault, FKV_FAULT_CONTEXT);
    s.T = s.T < 0 ? 0 : p.max_blocks * 16;
  }
  s.lo = p.window > 0 ? max(0, s.T - p.window) : 0;
  s.shares = false;
  if constexpr (SHARED) {
    const int keys = p.shared[b].x;
    s.shares = keys > 0;
    s.lo = min(max(s.lo, keys), s.T);
  }
  s.n = (((s.T + 15) >> 4) - (s.lo >> 4) + TPB - 1) / TPB;
  if constexpr (SHARED) s.n = s.lo < s.T ? s.n : 0;
  return s;
}

// A place in a CTA's range of tiles.
template <int TPB, bool SHARED>
struct Cursor {
  int b, g, t;       // tile t of unit (b, g)
  Seq s;
  int left;          // tiles of the range from this one on
  int piece;         // units begun before this one in the range

  FKV_DEV bool piece_ends() const { return t + 1 == s.n || left == 1; }
  FKV_DEV void advance(const BlockDecodeParams& p) {
    if (--left <= 0) return;
    if (++t < s.n) return;
    t = 0;
    ++piece;
    if (++g == p.Hkv) {
      g = 0;
      do s = seq_of<TPB, SHARED>(p, ++b, false);
      while (s.n == 0);
    }
  }
  FKV_DEV int block0() const { return (s.lo >> 4) + t * TPB; }                       // the tile's first block
  FKV_DEV int blocks() const { return min(TPB, ((s.T + 15) >> 4) - block0()); }      // and how many it has
};

// The range of CTA k: its first tile and their number, the place w0 of that tile, W (places in all, below
// 2^31) and N, the CTAs that have places.  Every lane of a warp takes part.
template <int TPB, bool SHARED>
FKV_DEV Cursor<TPB, SHARED> first_tile(const BlockDecodeParams& p, int k, int& N, int& w0, int& W, bool report) {
  const int lane = threadIdx.x & 31;
  auto places = [](int n) { return n > 0 ? n + 1 : 0; };
  auto seq = [&](int b0, bool rep) { return b0 + lane < p.B ? seq_of<TPB, SHARED>(p, b0 + lane, rep) : Seq{0, 0, 0, false}; };
  const Seq s0 = seq(0, report);
  int total = __reduce_add_sync(0xffffffffu, places(s0.n));
  for (int b0 = 32; b0 < p.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, places(seq(b0, report).n));
  W = total * p.Hkv;
  N = min(static_cast<int>(gridDim.x), W);
  Cursor<TPB, SHARED> c;
  c.left = c.b = c.g = c.t = c.piece = 0;
  c.s = Seq{0, 0, 0, false};
  w0 = 0;
  if (k >= N) return c;
  const int each = W / N, rest = W - each * N;  // floor(k W / N) = k each + floor(k rest / N)
  w0 = k * each + k * rest / N;
  const int w1 = (k + 1) * each + (k + 1) * rest / N;
  int base = 0;  // places of the sequences before b0
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const Seq s = b0 == 0 ? s0 : seq(b0, false);
    int before = places(s.n);  // inclusive sums over the lanes
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + before * p.Hkv > w0);
    if (past != 0) {
      const int j = __ffs(past) - 1;  // the first sequence that ends behind w0
      c.b = b0 + j;
      c.s.T = __shfl_sync(0xffffffffu, s.T, j);
      c.s.lo = __shfl_sync(0xffffffffu, s.lo, j);
      c.s.n = __shfl_sync(0xffffffffu, s.n, j);
      c.s.shares = SHARED && __shfl_sync(0xffffffffu, s.shares, j);
      const int rem = w0 - base - __shfl_sync(0xffffffffu, before - places(s.n), j) * p.Hkv;
      c.g = rem / (c.s.n + 1);
      c.t = rem - c.g * (c.s.n + 1) - 1;
      if (c.t < 0) {  // a blank place: its unit's first tile is next
        c.t = 0;
        ++w0;
      }
      // the tiles among places w0 .. w1 - 1: blanks lie at the units' first places
      int at = w0 - c.t - 1, blanks = 0;  // the blank place of the current unit
      int b = c.b, g = c.g, n = c.s.n;
      for (;;) {
        at += n + 1;
        if (at >= w1) break;
        ++blanks;
        if (++g == p.Hkv) {
          g = 0;
          do n = ++b < p.B ? seq_of<TPB, SHARED>(p, b, false).n : 0;
          while (n == 0 && b < p.B);
        }
      }
      c.left = w1 - w0 - blanks;
      return c;
    }
    base += __shfl_sync(0xffffffffu, before, 31) * p.Hkv;
  }
  return c;
}

// The CTA whose range holds place w: floor(((w + 1) N - 1) / W).
FKV_DEV int cta_of(int w, int W, int N) {
  const unsigned long long x = static_cast<unsigned long long>(w + 1) * N - 1;
  return static_cast<int>(x >> 32 ? x / W : static_cast<uint32_t>(x) / static_cast<uint32_t>(W));
}

// Add 1 to a counter with release and acquire semantics at GPU scope: what this CTA wrote before the
// barrier in front of it is visible to whom the sum orders behind it.
FKV_DEV int count_acq_rel(int32_t* p) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

FKV_DEV void tmem_ld4(uint32_t addr, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr));
}

// The heads' columns of both terms: NL of hi, NL of lo.
template <typename C>
FKV_DEV void load_terms(uint32_t col, float (&v)[2 * C::NL]) {
  if constexpr (C::NL == 4) {
    tmem_ld4(col, v);
    tmem_ld4(col + C::LO, v + 4);
  } else {
    tmem_ld16(col, v);
  }
}

FKV_DEV void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

FKV_DEV float warp_max_f(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The merge of a unit's pieces, rows row0 .. row0 + ns - 1 of the workspace, by the whole CTA:
// o = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M) in FP32.  First the heads' weights (a warp per head)
// into shared memory; then groups of threads, one thread per four outputs, take a share of the
// pieces each, eight at a time so that a round trip to L2 serves eight (the first eight are requested
// before the weights), and the groups' sums are added.  A piece whose sums are NaN has lse +inf, so that the output is NaN.
template <int D, int G>
FKV_DEV void merge_pieces(const BlockDecodeParams& p, int unit, long long row0, int ns, float* scratch) {
  constexpr int QUADS = G * D / 4, PARTS = QUADS <= kThreads ? kThreads / QUADS : 1, U = 8;
  float* inv_s = scratch;             // [G]
  float4* o_s = reinterpret_cast<float4*>(scratch + 16);  // [PARTS][QUADS]
  float* w_s = scratch + 16 + 4 * PARTS * QUADS;          // [G][ns]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = threadIdx.x / QUADS, q0 = PARTS > 1 ? threadIdx.x - part * QUADS : threadIdx.x;
  const int sb = PARTS > 1 ? part * ns / PARTS : 0, se = PARTS > 1 ? (part + 1) * ns / PARTS : ns;
  // pieces s .. s + U - 1 (the last one again behind it) of quad qd
  auto load = [&](float4 (&x)[U], int qd, int s, int s1) {
    const float* src = p.o_part + row0 * G * D + 4 * qd;
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = __ldcg(reinterpret_cast<const float4*>(src + static_cast<size_t>(min(s + u, s1 - 1)) * G * D));
  };
  float4 first[U];  // this thread's first pieces, on their way while the weights are made
  if (PARTS == 1 ? q0 < QUADS : part < PARTS && sb < se) load(first, q0, sb, se);
  for (int h = warp; h < G; h += kThreads / 32) {
    const float* lse = p.lse_part + row0 * G + h;
    float M = -INFINITY;
    for (int s = lane; s < ns; s += 32) {
      const float v = __ldcg(lse + static_cast<size_t>(s) * G);
      w_s[h * ns + s] = v;
      M = fmaxf(M, v);
    }
    M = warp_max_f(M);
    float W = 0.f;
    for (int s = lane; s < ns; s += 32) {
      const float w = ex2(w_s[h * ns + s] - M);
      w_s[h * ns + s] = w;
      W += w;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) W += __shfl_xor_sync(0xffffffffu, W, off);
    if (lane == 0) inv_s[h] = 1.f / W;
  }
  __syncthreads();
  __nv_bfloat16* out = p.out + static_cast<size_t>(unit) * G * D;  // (b * Hkv + g) * G rows of D
  auto sum = [&](int qd, int s0, int s1) -> float4 {
    const float* w = w_s + (qd / (D / 4)) * ns;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = s0; s < s1; s += U) {
      float4 x[U];
      if (qd == q0 && s == s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = first[u];
      } else {
        load(x, qd, s, s1);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float wu = s + u < s1 ? w[s + u] : 0.f;
        o.x = fmaf(wu, x[u].x, o.x);
        o.y = fmaf(wu, x[u].y, o.y);
        o.z = fmaf(wu, x[u].z, o.z);
        o.w = fmaf(wu, x[u].w, o.w);
      }
    }
    return o;
  };
  auto store = [&](int qd, float4 o) {
    const float inv = inv_s[qd / (D / 4)];
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(out + 4 * qd);
    dst[0] = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    dst[1] = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  };
  if constexpr (PARTS == 1) {
    for (int qd = threadIdx.x; qd < QUADS; qd += kThreads) store(qd, sum(qd, 0, ns));
  } else {
    const int qd = q0;
    if (part < PARTS) o_s[part * QUADS + qd] = sum(qd, sb, se);
    __syncthreads();
    if (part == 0) {
      float4 o = o_s[qd];
#pragma unroll
      for (int j = 1; j < PARTS; ++j) {
        const float4 x = o_s[j * QUADS + qd];
        o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
      }
      store(qd, o);
    }
  }
}

template <int D, int G, bool SHARED>
__global__ void __launch_bounds__(kThreads, (BlockDecodeCfg<D, G>::CTAS))
    block_decode_kernel(const __grid_constant__ BlockDecodeParams p, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
  using C = BlockDecodeCfg<D, G>;
  constexpr int TPB = C::TPB, LO = C::LO;
  using Place = Cursor<TPB, SHARED>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sP = smem + C::OFF_P;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  float* red_s = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* f_s = reinterpret_cast<float*>(smem + C::OFF_F);
  float* ml_s = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* qs_s = reinterpret_cast<float*>(smem + C::OFF_QS);
  float* sc_s = reinterpret_cast<float*>(smem + C::OFF_SC);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  // tiles are counted u = 0, 1, ... over the CTA's range, pieces likewise
  uint64_t* q_full = bars + 0;     // the query of piece r
  uint64_t* s_full = bars + 1;     // [2] S^T(u) in buffer u % 2
  uint64_t* s_free = bars + 3;     // [2]
  uint64_t* p_full = bars + 5;     // [2] P^T(u) in tile u % 2
  uint64_t* p_free = bars + 7;     // [2]
  uint64_t* o_full = bars + 9;     // [2] O_t^T(u) in buffer u % 2
  uint64_t* o_free = bars + 11;    // [2]
  uint64_t* mma_done = bars + 13;
  uint64_t* red_full = bars + 14;  // [2] the 4 warps' values of reduction r in slot r % 2
  uint64_t* f_full = bars + 16;    // [2] factors of tile u in slot u % 2
  uint64_t* f_free = bars + 18;    // [2]
  uint64_t* l_full = bars + 20;    // [2] r, l and o of piece r in slot r % 2 ...
  uint64_t* l_free = bars + 22;    // [2] ... and taken
  uint64_t* k_full = bars + 24;
  uint64_t* k_empty = k_full + C::NS;
  uint64_t* v_full = k_empty + C::NS;
  uint64_t* sc_full = v_full + C::NS;  // [SCN] scales of tile u in slot u % SCN
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* last_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  volatile int* pend_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);  // [2] {unit, first CTA, pieces}

  const int k = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // barriers and tensor memory need no input: they are set up before waiting for the kernels
  // before this one
  if (warp == 8 && lane == 0) {
    // barriers signalled by the softmax or correction warps count warps (one arrival each)
    mbar_init(q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_free[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&red_full[i], 4);
      mbar_init(&f_full[i], 4);
      mbar_init(&f_free[i], 4);
      mbar_init(&l_full[i], 4);
      mbar_init(&l_free[i], 4);
    }
    mbar_init(mma_done, 1);
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
    }
    for (int s = 0; s < C::SCN; ++s) mbar_init(&sc_full[s], 1);
    *abort_s = 0;
    pend_s[2] = pend_s[5] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  // (SHARED too: the kernel before this one is the shared part's, whose results are not read here, but only behind this wait is what the plan
  // before it wrote sure to be visible)
  griddep_wait();
  int N, w0, W;
  Place at = first_tile<TPB, SHARED>(p, k, N, w0, W, k == 0 && warp == 0);
  const int n = at.left;  // tiles of this CTA
  // the table's entry of block `lane` of a tile, read ahead of its use and looked at only there (a
  // check at the load would hold the warp for the load's latency)
  auto block_id = [&](const Place& c) -> int {
    if (c.left <= 0 || lane >= c.blocks()) return 0;
    return p.block_table[static_cast<size_t>(c.b) * p.max_blocks + c.block0() + lane];
  };
  // an id out of range reads block 0 and is reported
  auto checked = [&](int id) -> int {
    if (id >= 0 && id < p.num_blocks) return id;
    raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
    return 0;
  };
  // lane j's copies of block j of a tile
  auto copy_tile = [&](const CUtensorMap* map, uint8_t* dst, const Place& c, int id, uint64_t* full) {
    const int nblk = c.blocks();
    if (lane == 0) mbar_arrive_expect_tx(full, nblk * 16 * D);
    __syncwarp();
    if (lane < nblk) {
#pragma unroll
      for (int s = 0; s < C::NSUB; ++s) tma_load_4d(dst + s * C::KSUB + lane * 16 * C::RB, map, s * C::RB, 0, c.g >> p.halves, id, full);
    }
  };
  // The loads that the first tile waits for go out before the CTA's barrier and before the first copies of K
  // and V, which fill the memory system's queues for some microseconds: the query rows (softmax
  // warps, 8 threads per row), the first tiles' block ids (warp 8).
  constexpr int NCH = (D / 16 + 7) / 8;  // 16-element chunks of a query row per thread
  uint32_t in[NCH][8];
  auto load_query = [&](const Place& c) {
    const int row = threadIdx.x >> 3;
#pragma unroll
    for (int cc = 0; cc < NCH; ++cc) {
      const int ch = (threadIdx.x & 7) + 8 * cc;
#pragma unroll
      for (int j = 0; j < 8; ++j) in[cc][j] = 0u;
      if (row < G && ch < D / 16) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(c.b) * p.Hq + c.g * G + row) * D) + 2 * ch;
        const uint4 a = src[0], a2 = src[1];
        in[cc][0] = a.x; in[cc][1] = a.y; in[cc][2] = a.z; in[cc][3] = a.w;
        in[cc][4] = a2.x; in[cc][5] = a2.y; in[cc][6] = a2.z; in[cc][7] = a2.w;
      }
    }
  };
  if (warp < 4 && n > 0) load_query(at);
  const int n0 = min(C::NS, n);  // tiles whose copies warp 8 issues first, K and V
  int ids[C::NS];
  if (warp == 8 && n > 0) {
    Place c = at;
#pragma unroll
    for (int j = 0; j < C::NS; ++j) {
      ids[j] = block_id(c);
      if (j + 1 < C::NS) c.advance(p);
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the next kernel may take its place on the SMs from here on (not before this CTA has its tensor memory)
  griddep_launch_dependents();

  // sequences without keys: zero rows, spread over the CTAs
  if (warp >= 4 && warp < 8)
    for (int b = k; b < p.B; b += gridDim.x) {
      const Seq s = seq_of<TPB, SHARED>(p, b, false);
      if (s.n != 0 || s.shares) continue;  // (what is shared, the join writes)
      for (int x = threadIdx.x - 128; x < p.Hq * D / 8; x += 128)
        reinterpret_cast<uint4*>(p.out + static_cast<size_t>(b) * p.Hq * D)[x] = make_uint4(0u, 0u, 0u, 0u);
    }

  if (n == 0) {
    // more CTAs than tiles
  } else if (warp < 4) {
    // ============================================================ softmax warpgroup
    const int i = threadIdx.x;  // key i of a tile (TMEM lane i)
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float m[G], lsum[G];  // r and (this thread's keys only) l
    bool ok = true;
    bool fresh = true;  // the next tile begins a piece
    for (int u = 0; ok && u < n; ++u) {
      if (fresh) {
        // ---- the piece's query: head h's row scaled to (224, 448], as two terms (the products with the
        // last piece's query are done: their S was read).  8 threads per row.  A row with a NaN or
        // an infinity makes its scores, and so its output, NaN.
        fresh = false;
        const int row = i >> 3;
        if (at.piece > 0) load_query(at);
        uint32_t amax = 0;
#pragma unroll
        for (int cc = 0; cc < NCH; ++cc)
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = max(amax, max((in[cc][j] << 16) & 0x7FFF0000u, in[cc][j] & 0x7FFF0000u));
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const int e = query_exponent(amax);  // q = q' * 2^e
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        if ((i & 7) == 0 && row < G)
          qs_s[row] = amax < 0x7F800000u ? p.sm_scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23)
                                         : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int cc = 0; cc < NCH; ++cc) {
          const int c = (i & 7) + 8 * cc;
          if (c >= D / 16 || row >= LO) continue;
          uint32_t wh[4], wl[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x0 = bf16x2_to_f2(in[cc][2 * j]), x1 = bf16x2_to_f2(in[cc][2 * j + 1]);
            split4_query(make_float2(x0.x * down, x0.y * down), make_float2(x1.x * down, x1.y * down), wh[j], wl[j]);
          }
          const int byte = c * 16;
          uint8_t* sub = sQ + (byte / C::RB) * C::QSUB;
          *reinterpret_cast<uint4*>(sub + swz(static_cast<uint32_t>(row * C::RB + byte % C::RB), C::RB)) =
              make_uint4(wh[0], wh[1], wh[2], wh[3]);
          *reinterpret_cast<uint4*>(sub + swz(static_cast<uint32_t>((LO + row) * C::RB + byte % C::RB), C::RB)) =
              make_uint4(wl[0], wl[1], wl[2], wl[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(q_full);
        if (!wait_warp(q_full, at.piece & 1)) { ok = false; break; }  // every warp's rows and c are there
#pragma unroll
        for (int h = 0; h < G; ++h) {
          m[h] = -INFINITY;
          lsum[h] = 0.f;
        }
        // the next unit's query towards L2 (its rows follow; i sweeps them in 32-byte steps)
        if (at.left > at.s.n - at.t && (at.g + 1 < p.Hkv || at.b + 1 < p.B) && i * 16 < G * D)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + (static_cast<size_t>(at.b) * p.Hkv + at.g + 1) * G * D + i * 16));
      }
      if ((u & 7) == 7 && abort_warp(abort_s)) { ok = false; break; }
      const int sb = u & 1;
      if (!wait_warp(&s_full[sb], (u >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      float x[C::NHALF][G];  // the scores of key i + 128 hh of the tile
      uint32_t whi[C::NHALF][2], wlo[C::NHALF][2];  // P's codes
      float sv[2 * C::NL];
      auto load_s = [&](int hh) {
        const uint32_t col = lane_base + C::TM_S + (sb * C::NHALF + hh) * C::NP;
        load_terms<C>(col, sv);
      };
      load_s(0);
      if (!wait_warp(&sc_full[u % C::SCN], (u / C::SCN) & 1)) { ok = false; break; }
      const float* slot = sc_s + (u % C::SCN) * C::SCF;
      float ks[C::NHALF], lv[C::NHALF], iv[C::NHALF], pmax[C::NHALF];
      bool valid[C::NHALF];
#pragma unroll
      for (int hh = 0; hh < C::NHALF; ++hh) {
        ks[hh] = slot[8 * hh + (i >> 4)];
        lv[hh] = slot[TPB + 8 * hh + (i >> 4)];
        iv[hh] = slot[2 * TPB + 8 * hh + (i >> 4)];
        pmax[hh] = iv[hh] > 0.f ? 448.f : 0.f;  // (0: a scale that counts as zero)
        const int key = at.block0() * 16 + 128 * hh + i;
        valid[hh] = key >= at.s.lo && key < at.s.T;
      }
      const float o = slot[3 * TPB], rare = slot[3 * TPB + 1], change = slot[3 * TPB + 2];
#pragma unroll
      for (int hh = 0; hh < C::NHALF; ++hh) {
        tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < G; ++h) x[hh][h] = sv[h] + sv[C::NL + h];
        if (hh + 1 < C::NHALF) load_s(hh + 1);
      }
      tc_fence_before();
      mbar_arrive_warp(&s_free[sb]);
      // the heads' maxima of y over the tile's keys: within the warp, then across the 4
      const int rr = u + at.piece;  // reductions before this one (each piece ended with one of its own)
      float* red = red_s + (rr & 1) * 4 * LO;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        float wm = -INFINITY;
#pragma unroll
        for (int hh = 0; hh < C::NHALF; ++hh) {
          x[hh][h] = valid[hh] ? fmaf(x[hh][h], qs_s[h] * ks[hh], lv[hh]) : -INFINITY;  // (c in shared memory: registers)
          wm = hh == 0 ? x[hh][h] : fmaxf(wm, x[hh][h]);
        }
        wm = warp_max_f(wm);
        if (lane == 0) red[warp * LO + h] = wm;
      }
      // reduction rr uses slot rr % 2 (its use before, rr - 2, was read by every warp before that
      // warp's arrival for rr - 1)
      if (lane == 0) mbar_arrive(&red_full[rr & 1]);
      if (!wait_warp(&red_full[rr & 1], (rr >> 1) & 1)) { ok = false; break; }
      const int pb = u & 1;
      if (u >= 2 && !wait_warp(&p_free[pb], ((u >> 1) - 1) & 1)) { ok = false; break; }
      if (u >= 2 && !wait_warp(&f_free[pb], ((u >> 1) - 1) & 1)) { ok = false; break; }
      // four heads at a time (a word of codes): maxima, P's terms, factors
      auto heads = [&](auto rarely) {
#pragma unroll
        for (int h4 = 0; h4 < G; h4 += 4) {
          constexpr int HN = G < 4 ? G : 4;
          float tm[4];
          {
            const float4 r0 = *reinterpret_cast<const float4*>(red + h4), r1 = *reinterpret_cast<const float4*>(red + LO + h4);
            const float4 r2 = *reinterpret_cast<const float4*>(red + 2 * LO + h4), r3 = *reinterpret_cast<const float4*>(red + 3 * LO + h4);
            tm[0] = fmaxf(fmaxf(r0.x, r1.x), fmaxf(r2.x, r3.x));
            tm[1] = fmaxf(fmaxf(r0.y, r1.y), fmaxf(r2.y, r3.y));
            tm[2] = fmaxf(fmaxf(r0.z, r1.z), fmaxf(r2.z, r3.z));
            tm[3] = fmaxf(fmaxf(r0.w, r1.w), fmaxf(r2.w, r3.w));
          }
          float pv[C::NHALF][4], al[4], be[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            al[j] = be[j] = 0.f;
            if (j >= HN) {
#pragma unroll
              for (int hh = 0; hh < C::NHALF; ++hh) pv[hh][j] = 0.f;
              continue;
            }
            const int h = h4 + j;
            // one of the two factors is 1, the other 2^-|m - tmax|
            const float e = ex2(-fabsf(m[h] - tm[j]));
            const float alpha = m[h] > tm[j] ? 1.f : e, corr = m[h] > tm[j] ? e : 1.f;
            float psum = 0.f;
#pragma unroll
            for (int hh = 0; hh < C::NHALF; ++hh) {
              const float w = valid[hh] ? ex2(x[hh][h] - tm[j]) : 0.f;
              psum = fmaf(w, fabsf(iv[hh]), psum);
              pv[hh][j] = w * pmax[hh];
            }
            if constexpr (decltype(rarely)::value) {
              const RareFactors f = rare_factors(m[h], lsum[h], tm[j], change);
              lsum[h] = lsum[h] * f.l * f.l * f.l + psum * f.lt * f.lt * f.lt;
              al[j] = f.alpha;
              be[j] = f.beta;
            } else {
              lsum[h] = fmaf(lsum[h], alpha, psum * corr);
              m[h] = fmaxf(m[h], tm[j]);
              al[j] = alpha;
              be[j] = corr;
            }
          }
          if (i == 0) {
            *reinterpret_cast<float4*>(f_s + pb * 2 * LO + h4) = make_float4(al[0], al[1], al[2], al[3]);
            *reinterpret_cast<float4*>(f_s + pb * 2 * LO + LO + h4) = make_float4(be[0], be[1], be[2], be[3]);
          }
          // the codes of heads h4 .. h4 + 3: words h4 / 4 (hi) and LO / 4 + h4 / 4 (lo) of the key's bytes
#pragma unroll
          for (int hh = 0; hh < C::NHALF; ++hh) {
            uint32_t hi, lo;
            split4<false>(make_float2(pv[hh][0], pv[hh][1]), make_float2(pv[hh][2], pv[hh][3]), hi, lo);
            whi[hh][h4 / 4] = hi;
            wlo[hh][h4 / 4] = lo;
          }
        }
      };
      if (rare == 0.f) heads(std::false_type());
      else heads(std::true_type());
#pragma unroll
      for (int hh = 0; hh < C::NHALF; ++hh) {
        uint8_t* key = sP + pb * C::PTILE + (128 * hh + i) * 16;
        *reinterpret_cast<uint4*>(key) = make_uint4(whi[hh][0], G > 4 ? whi[hh][1] : 0u, wlo[hh][0], G > 4 ? wlo[hh][1] : 0u);
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(&p_full[pb]);
      mbar_arrive_warp(&f_full[pb]);
      if (at.piece_ends()) {
        // ---- the piece's r, l (summed over the 128 key threads) and o for the correction
        const int r = at.piece, re = rr + 1;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float s = lsum[h];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
          if (lane == 0) red_s[(re & 1) * 4 * LO + warp * LO + h] = s;
        }
        if (lane == 0) mbar_arrive(&red_full[re & 1]);
        if (!wait_warp(&red_full[re & 1], (re >> 1) & 1)) { ok = false; break; }
        if (r >= 2 && !wait_warp(&l_free[r & 1], ((r >> 1) - 1) & 1)) { ok = false; break; }
        if (i == 0) {
          const float* red2 = red_s + (re & 1) * 4 * LO;
#pragma unroll
          for (int h = 0; h < G; ++h) {
            ml_s[(r & 1) * C::MLF + h] = m[h];
            ml_s[(r & 1) * C::MLF + LO + h] = (red2[h] + red2[LO + h]) + (red2[2 * LO + h] + red2[3 * LO + h]);
          }
          ml_s[(r & 1) * C::MLF + 2 * LO] = o;
        }
        mbar_arrive_warp(&l_full[r & 1]);
        fresh = true;
      }
      at.advance(p);
    }
    tmem_ld_wait();  // no load left in flight on an early exit: the tensor memory is freed below
    if (!ok) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
  } else if (warp < 8) {
    // ============================================================ correction warpgroup
    const int i = threadIdx.x - 128;  // TMEM lane i
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp - 4) * 32) << 16);
    // the head_dim row this lane holds (and 128 + it): lane i itself for M = 128; for M = 64 lanes 0-15 of
    // each warp hold rows 16 (warp - 4) + lane
    const bool has_row = C::MPV == 128 || lane < 16;
    const int d = C::MPV == 128 ? i : (warp - 4) * 16 + lane;
    float acc[C::NSUB][G];
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
      for (int s2 = 0; s2 < C::NSUB; ++s2) acc[s2][h] = 0.f;
    // V's copies: blocks v0 .. v0 + VB - 1 of a tile, a block per lane, its id read a tile ahead
    constexpr int VB = TPB / 4;
    const int v0 = (warp - 4) * VB;
    Place vat = at;
    for (int j = 0; j < n0; ++j) vat.advance(p);
    auto v_id = [&]() -> int {
      if (vat.left <= 0 || lane >= VB || v0 + lane >= vat.blocks()) return 0;
      return p.block_table[static_cast<size_t>(vat.b) * p.max_blocks + vat.block0() + v0 + lane];
    };
    int tv = n0, vid = v_id();  // the next tile to copy
    auto copy_v = [&]() {
      const int st = tv % C::NS, nblk = min(max(vat.blocks() - v0, 0), VB), id = checked(vid);
      if (lane == 0) mbar_arrive_expect_tx(&v_full[st], nblk * 16 * D);
      __syncwarp();
      if (lane < nblk) {
#pragma unroll
        for (int s = 0; s < C::NSUB; ++s)
          tma_load_4d(sV + st * C::KTILE + s * C::KSUB + (v0 + lane) * 16 * C::RB, &tmv, s * C::RB, 0, vat.g >> p.halves, id, &v_full[st]);
      }
      ++tv;
      vat.advance(p);
      vid = v_id();
    };
    bool ok = true;
    int w = w0;  // the tile's place
    for (int u = 0; u < n; ++u) {
      if ((u & 7) == 7 && abort_warp(abort_s)) ok = false;
      const int ob = u & 1;
      if (ok) ok = wait_warp(&f_full[ob], (u >> 1) & 1);
      float alpha[G], beta[G];
      if (ok) {
#pragma unroll
        for (int h = 0; h < G; ++h) {
          alpha[h] = f_s[ob * 2 * LO + h];
          beta[h] = f_s[ob * 2 * LO + LO + h];
        }
        mbar_arrive_warp(&f_free[ob]);
        ok = wait_warp(&o_full[ob], (u >> 1) & 1);
      }
      if (ok) {
        tc_fence_after();
        float o[C::NSUB][2 * C::NL];
#pragma unroll
        for (int s2 = 0; s2 < C::NSUB; ++s2) {
          const uint32_t col = lane_base + C::TM_O + (ob * C::NSUB + s2) * C::NP;
          load_terms<C>(col, o[s2]);
        }
        if (tv < n) copy_v();  // the P.V of tile u = tv - NS is done with its stage
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive_warp(&o_free[ob]);
#pragma unroll
        for (int s2 = 0; s2 < C::NSUB; ++s2)
#pragma unroll
          for (int h = 0; h < G; ++h) acc[s2][h] = fmaf(acc[s2][h], alpha[h], beta[h] * (o[s2][h] + o[s2][C::NL + h]));
      }
      if (at.piece_ends()) {
        // ---- the piece's result: 2^o acc / (448 l), and its log2-sum-exp r - o + log2 l
        const int r = at.piece;
        const int unit = at.b * p.Hkv + at.g;
        const int u0 = w - at.t;  // the place of the unit's first tile
        const int k0 = cta_of(u0, W, N), ns = cta_of(u0 + at.s.n - 1, W, N) - k0 + 1;
        const bool shares = SHARED && at.s.shares;
        if (shares && i == 0 && k == k0) p.units[unit] = make_int2(k0, ns);
        if (ok) ok = wait_warp(&l_full[r & 1], (r >> 1) & 1);
        if (ok) {
          const long long row = static_cast<long long>(k) + unit;
          const float* ml = ml_s + (r & 1) * C::MLF;
          const float o = ml[2 * LO], so = pow2i(o);
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float mh = ml[h], L = ml[LO + h];
            const float inv = 1.f / (448.f * L);
            if (ns == 1 && !shares) {
              if (has_row) {
#pragma unroll
                for (int s2 = 0; s2 < C::NSUB; ++s2)
                  p.out[(static_cast<size_t>(at.b) * p.Hq + at.g * G + h) * D + s2 * 128 + d] = __float2bfloat16(acc[s2][h] * inv * so);
              }
            } else {
              if (has_row) {
#pragma unroll
                for (int s2 = 0; s2 < C::NSUB; ++s2) p.o_part[(row * G + h) * D + s2 * 128 + d] = acc[s2][h] * inv * so;
              }
              if (i == 0) p.lse_part[row * G + h] = L > 0.f ? mh - o + lg2(L) : INFINITY;
            }
#pragma unroll
            for (int s2 = 0; s2 < C::NSUB; ++s2) acc[s2][h] = 0.f;
          }
          mbar_arrive_warp(&l_free[r & 1]);
        }
        if (ns > 1 && i == 0 && !shares) {
          // to be counted (after a timeout too: the counters return to zero); only a range's first and
          // last pieces can be parts of a unit
          volatile int* pend = pend_s + (r == 0 ? 0 : 3);
          pend[0] = unit;
          pend[1] = k0;
          pend[2] = ns;
        }
      }
      w += at.t + 1 == at.s.n ? 2 : 1;  // a new unit begins with a blank place
      at.advance(p);
    }
    if (!ok) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
      // let the copies land before the CTA can exit (on the way to here without a fault, P.V read them all)
      if (lane == 0)
        for (int s = 0; s < C::NS; ++s)
          if (tv > s) wait_ns(&v_full[s], ((tv - 1 - s) / C::NS) & 1);
      __syncwarp();
    }
  } else if (warp == 8) {
    // ============================================================ K copies and scales
    // K(u) into stage u % NS once the S^T of tile u - NS has read it, the first NS with their V at
    // once; the scales of tile u into their slot.  (A warp's copies go out one after another, 100 cycles each.  SHARED, short ranges
    // mostly: the first tile's scales come before the copies of the tiles behind it, the first P after 8,270 cycles instead of 13,580;
    // longer ranges gain nothing.)
    float ks_n = 0.f, vs_n = 0.f;
    auto read_scales = [&](const Place& c, int j) {
      ks_n = vs_n = 0.f;
      if (c.left > 0 && lane < c.blocks()) {
        const size_t x = static_cast<size_t>(j) * (p.Hkv >> p.halves) + (c.g >> p.halves);
        ks_n = p.k_scale[x];
        vs_n = p.v_scale[x];
      }
    };
    auto copy_first = [&](const Place& c, int x, int st) {  // K and V
      copy_tile(&tmk, sK + st * C::KTILE, c, x, &k_full[st]);
      if (lane > 0 && lane < 4) mbar_arrive(&v_full[st]);  // (a phase has four arrivals)
      copy_tile(&tmv, sV + st * C::KTILE, c, x, &v_full[st]);
    };
    int id = checked(ids[0]);
    read_scales(at, id);
    copy_first(at, id, 0);
    int used = 1;  // tiles whose K copy was issued
    Place nx = at;
    nx.advance(p);
    auto copy_next_ones = [&](Place c) {
#pragma unroll
      for (int j = 1; j < C::NS; ++j) {
        if (j >= n0) break;
        copy_first(c, checked(ids[j]), j);
        if (j + 1 < C::NS) c.advance(p);
      }
      used = n0;
    };
    if constexpr (!SHARED) copy_next_ones(nx);
    int id_next = ids[1];
    ScaleRange range;
    for (int u = 0; u < n; ++u) {
      if (abort_warp(abort_s)) break;
      const float ks = ks_n, vs = vs_n;
      const int id_u = id;
      const Place here = at;
      id = checked(id_next);
      read_scales(nx, id);
      at = nx;
      nx.advance(p);
      id_next = block_id(nx);
      const int st = u % C::NS, use = u / C::NS;
      if (u >= n0) {
        if (!wait_stage_warp(&k_empty[st], (use - 1) & 1, p.stage_wait_ns)) {
          if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
          *abort_s = 1;
          break;
        }
        copy_tile(&tmk, sK + st * C::KTILE, here, id_u, &k_full[st]);
        used = u + 1;
      }
      if (here.t == 0) range = ScaleRange();  // another piece
      const BlockScale sc = block_scales(range, vs, lane < here.blocks());
      float* slot = sc_s + (u % C::SCN) * C::SCF;
      if (lane < TPB) {
        slot[lane] = ks;
        slot[TPB + lane] = sc.lv;
        slot[2 * TPB + lane] = sc.iv;
      }
      if (lane == 0) {
        slot[3 * TPB] = range.o;
        slot[3 * TPB + 1] = sc.rare ? 1.f : 0.f;
        slot[3 * TPB + 2] = sc.change;
      }
      mbar_arrive_warp(&sc_full[u % C::SCN]);
      if (SHARED && u == 0) copy_next_ones(at);
    }
    // let every copy issued here land before the CTA can exit
    if (lane == 0) {
      for (int s = 0; s < C::NS; ++s)
        if (used > s) wait_ns(&k_full[s], ((used - 1 - s) / C::NS) & 1);
      for (int s = 0; s < min(used, n0); ++s)
        if (*abort_s) wait_ns(&v_full[s], 0);
    }
    __syncwarp();
  } else {
    // ============================================================ MMA issuer (warp 9)
    // Lane 0 polls the pipeline's barriers without blocking and issues, in whatever order they
    // become possible, the S^T and the P.V products.
    const uint64_t dK = smem_desc(smem_u32(sK), 16, 8 * C::RB, C::SWZ), dQ = smem_desc(smem_u32(sQ), 16, 8 * C::RB, C::SWZ);
    const uint64_t dV = smem_desc(smem_u32(sV), 8 * C::RB, 8 * C::RB, C::SWZ);
    // P without swizzle: 8 keys of 16 bytes per 128-byte core matrix, the next 8 keys 128 bytes on
    const uint64_t dP = smem_desc(smem_u32(sP), 128, 128, 0);
    int tq = 0, tp = 0;  // next S^T and P.V
    Place qat = at, pat = at;
    bool q_ready = false;  // the query of tile tq's piece is in place
    bool ok = true;
    uint64_t t_idle = 0;
    while (ok && tp < n) {
      int events = 0;  // bit 1: P.V of tile tp ready; bit 2: S^T issued
      if (lane == 0) {
        // S^T(tq) = K8(tq) q^T into buffer tq % 2: K landed, the buffer's previous S read
        if (tq < n && (q_ready || mbar_test_wait(q_full, qat.piece & 1)) &&
            mbar_test_wait(&k_full[tq % C::NS], (tq / C::NS) & 1) &&
            (tq < 2 || mbar_test_wait(&s_free[tq & 1], ((tq >> 1) - 1) & 1))) {
          const int st = tq % C::NS, sb = tq & 1;
          tc_fence_after();
#pragma unroll
          for (int hh = 0; hh < C::NHALF; ++hh)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              const int byte = kk * 32;
              umma_f8(tmem + C::TM_S + (sb * C::NHALF + hh) * C::NP,
                      desc_add(dK, st * C::KTILE + (byte / C::RB) * C::KSUB + hh * 128 * C::RB + byte % C::RB),
                      desc_add(dQ, (byte / C::RB) * C::QSUB + byte % C::RB), C::IDESC_QK, kk > 0 ? 1u : 0u);
            }
          umma_commit(&s_full[sb]);
          umma_commit(&k_empty[st]);
          events |= 4;
        }
        // P.V of tile tp: P written, V landed, the O_t buffer promoted (tile tp - 2)
        if (tp < tq + ((events >> 2) & 1) && mbar_test_wait(&p_full[tp & 1], (tp >> 1) & 1) &&
            mbar_test_wait(&v_full[tp % C::NS], (tp / C::NS) & 1) &&
            (tp < 2 || mbar_test_wait(&o_free[tp & 1], ((tp >> 1) - 1) & 1)))
          events |= 2;
      }
      events = __shfl_sync(0xffffffffu, events, 0);
      if (events & 4) {
        ++tq;
        q_ready = !qat.piece_ends();
        qat.advance(p);
      }
      if (events & 2) {
        const int st = tp % C::NS, pb = tp & 1;
        // keys past the context, and before a window, may hold any bytes (NaN codes) or were not
        // loaded: zero their V rows, since 0 * NaN would poison the product even though their P is 0
        const int kbase = pat.block0() * 16;
        const int keep_lo = max(pat.s.lo - kbase, 0), keep_hi = min(pat.s.T - kbase, C::BN);
        if (keep_lo > 0 || keep_hi < C::BN) {
          constexpr int CPR = C::RB / 16;  // 16-byte chunks per row
          for (int x = lane; x < (keep_lo + C::BN - keep_hi) * C::NSUB * CPR; x += 32) {
            const int c = x % CPR, s = (x / CPR) % C::NSUB, j = x / (CPR * C::NSUB);
            const int r = j < keep_lo ? j : keep_hi + j - keep_lo;
            *reinterpret_cast<uint4*>(sV + st * C::KTILE + s * C::KSUB + r * C::RB + c * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          tc_fence_after();
          // O_t^T(tp) = V8(tp)^T P(tp)^T into buffer tp % 2, one product per column block
#pragma unroll
          for (int s = 0; s < C::NSUB; ++s)
#pragma unroll
            for (int kk = 0; kk < C::BN / 32; ++kk)
              umma_f8(tmem + C::TM_O + (pb * C::NSUB + s) * C::NP, desc_add(dV, st * C::KTILE + s * C::KSUB + kk * 32 * C::RB),
                      desc_add(dP, pb * C::PTILE + kk * 32 * 16), C::IDESC_PV, kk > 0 ? 1u : 0u);
          umma_commit(&o_full[pb]);
          umma_commit(&p_free[pb]);
        }
        __syncwarp();
        ++tp;
        pat.advance(p);
      }
      if (events != 0) {
        t_idle = 0;
        continue;
      }
      if (abort_warp(abort_s)) break;
      const uint64_t now = globaltimer_ns();
      if (t_idle == 0) t_idle = now;
      if (__any_sync(0xffffffffu, now - t_idle > kPipeWaitNs)) ok = false;
      __nanosleep(32);  // leave the issue slots to the softmax warp sharing this SM quarter
    }
    if (!ok) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
    // every product issued by this warp completes before TMEM is released
    if (lane == 0) {
      umma_commit(mma_done);
      wait_ns(mma_done, 0);
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  // the CTA that brings a unit's last piece merges it and returns its counter to zero
  for (int j = 0; j < 2; ++j) {
    const int unit = pend_s[3 * j], k0 = pend_s[3 * j + 1], ns = pend_s[3 * j + 2];
    if (ns == 0) continue;
    if (threadIdx.x == 0) {
      const int old = count_acq_rel(&p.done[k0]);  // (CTA k0 begins no other unit that goes on behind its range)
      if (old >= ns) raise_fault(p.fault, FKV_FAULT_WORKSPACE);
      if (old == ns - 1) p.done[k0] = 0;
      *last_s = old == ns - 1;
    }
    __syncthreads();
    if (*last_s) {
      merge_pieces<D, G>(p, unit, static_cast<long long>(k0) + unit, ns, reinterpret_cast<float*>(sK));
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace fkv
