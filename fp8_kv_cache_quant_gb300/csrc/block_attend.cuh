// A tile of query rows over a block-scaled e4m3 cache on tcgen05 tensor cores, for the prefill (block_prefill.cu) and for what
// the sequences of a decode share (block_shared.cu): FP8 products
// with the bf16 query and P each as two e4m3 terms, FP32 accumulation in tensor memory, each
// tile's partial promoted into FP32 registers.
//
// Mathematics.  With q' = q 2^-k (k per row, so that the row's largest magnitude lies in (224, 448])
// and q' = hi + lo, hi the nearest e4m3 value, the scores of a tile of 128 keys are
//   x_j = (hi . k8_j + lo . k8_j) * c * ks[block(j)],   c = 2^k softmax_scale log2(e);
// hi + lo is q' down to 2^-17 of the row's largest element (split4_query).  With y_j = x_j + L[block(j)], L = log2 vs, and the row's maximum R_t of y over the tile,
//   P_j = 448 * 2^(y_j - R_t),  P = hi + lo, hi its leading 3 fraction bits,
//   l_t = sum_blocks 2^(o - L) sum_j P_j,  O_t = sum_j (hi + lo)_j v8_j,
// and the running state is r' = max(r, R_t), acc = acc 2^(r - r') + O_t 2^(R_t - r'),
// l = l 2^(r - r') + l_t 2^(R_t - r'); the output 2^o acc / l.  P is taken against the largest p vs of
// the keys that the row sees in the tile, so that no other key's scale enters its arithmetic: it loses what lies
// below 2^-17 of that, and is otherwise within 2^-8 of its value, the precision of a bf16 P.  o keeps l within
// float32's range: block_scales in block_common.cuh.
// hi and lo accumulate into the same S and O_t (two products of K = 32 instead of one), so that
// K and V are used as they lie in the cache, without a pass that widens them to 16 bits.
//
// CTA = (up to 128 rows, KV head, sequence); a row is a (token, query head of the group) pair, so
// that short chunks fill the 128 rows of the products and K / V tiles serve the whole group.
// 16 warps:
//   0-7   softmax: warp w owns rows 32 (w % 4) + 16 (w / 4) .. + 15, lanes l and l + 16 each half of
//         a row's columns (16x32bx2 TMEM loads): the query's two terms (prologue); then per tile
//         the maximum, P's two terms into shared memory, the row's factors of acc and O_t;
//   8-11  correction: acc in registers (at head_dim 256 its second half in TMEM), epilogue;
//   12    K copies (a block per lane) and the tile's scales: ks, L, 2^(o - L) and o, read one tile
//         ahead and staged in shared memory;
//   13    allocates TMEM, issues S = q' K8^T;    14  issues O_t = P V8;    15  V copies.
// TMEM: two S buffers and two O_t buffers up to head_dim 128; at head_dim 256 one S buffer, two
// 128-column O_t buffers for the halves of head_dim, and the second half of acc.
// Few rows (drafted tokens, short chunks) over a long context: a cluster of up to 8 CTAs shares
// the rows' key tiles, and the partial results meet through distributed shared memory, where each
// CTA merges its share of the rows (kClusters).
// Sequences that share a prefix: the rows are those of a group's members, the keys a share of the prefix, and the
// result, float32 and with its log-sum-exp, goes to the workspace (kPieces).
// Every wait is bounded in time; a timeout records FKV_FAULT_TIMEOUT, lets the CTA's copies and
// products drain and returns.
#pragma once
#include "block_common.cuh"
#include "prefill_common.cuh"
#include "tc.cuh"

namespace fkv {
namespace {

constexpr float kHuge = 3e38f;  // minus this: the maximum of no scores

template <int D>
struct BlockPrefillCfg {
  static constexpr int BM = 128, BN = 128;          // rows of a CTA, keys of a tile
  static constexpr int NBLK = BN / 16;              // blocks of a tile
  static constexpr int RB = D < 128 ? D : 128;      // bytes of one swizzled row
  static constexpr int NSUB = D / RB;               // sub-tiles along head_dim
  static constexpr int SWZ = RB == 128 ? 2 : 4;     // descriptor swizzle mode (128 B / 64 B)
  static constexpr int SUB = 128 * RB;              // bytes of one 128-row sub-tile (Q, K or V)
  static constexpr int TILE = 128 * D;              // bytes of a term of Q, or of a K or V tile
  static constexpr int NS = D <= 128 ? 3 : 2;       // K / V stages
  static constexpr int DN = D < 128 ? D : 128;      // columns of one P.V product
  static constexpr int NH = D / DN;                 // P.V passes per tile
  static constexpr int PTERM = BM * BN;             // bytes of one term of P
  static constexpr int PBUF = D <= 128 ? 2 : 1;     // P buffers (two do not fit at head_dim 256)
  static constexpr int SBUF = D <= 128 ? 2 : 1;     // S buffers in TMEM
  static constexpr int HC = BN / 2;                 // columns of a softmax thread
  static constexpr int SW = 8;                      // softmax warps
  static constexpr int THREADS = 512;
  static constexpr int TM_OT = 128 * SBUF, TM_OH = TM_OT + 2 * DN;  // O_t buffers; second half of acc
  static constexpr int TM_COLS = 512;
  // scales of a tile in a ring of slots: the K copies run at most SBUF + NS tiles ahead of the
  // softmax (a stage is refilled once its S was computed, an S buffer once it was read)
  static constexpr int SCN = D <= 128 ? 8 : 4;
  static constexpr int SCF = 32;                    // floats per slot: ks [8], L [8], 2^(o - L) [8], o, BlockScale's rare, change
  static_assert(SCN > SBUF + NS, "a slot is rewritten only after the softmax is done with it");
  // registers per thread of the warpgroups (launch: 128 each): softmax, correction, copies and MMA (head_dim 64
  // spills at 120: 485 against 481 us for 2,048 queries over 8,192 keys, 64/8 heads)
  static constexpr int REG_LAUNCH = 128, REG_SOFT = D > 64 ? 120 : 128, REG_CORR = D > 64 ? 232 : 144,
                       REG_MISC = 4 * REG_LAUNCH - 2 * REG_SOFT - REG_CORR;
  static_assert(REG_SOFT <= REG_LAUNCH && REG_CORR >= REG_LAUNCH && REG_MISC <= REG_LAUNCH && REG_MISC >= 24 &&
                    REG_SOFT % 8 == 0 && REG_CORR % 8 == 0 && REG_MISC % 8 == 0,
                "setmaxnreg budgets");
  // shared memory (bytes)
  static constexpr int OFF_Q = 0;                   // hi, lo
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + NS * TILE;
  static constexpr int OFF_P = OFF_V + NS * TILE;   // per buffer: hi, lo
  static constexpr int OFF_F = OFF_P + PBUF * 2 * PTERM;  // factors [2][128] float2 (acc, O_t); last: (1 / l, 2^o)
  static constexpr int OFF_SC = OFF_F + 2 * BM * 8;
  static constexpr int OFF_BAR = OFF_SC + SCN * SCF * 4;
  static constexpr int NBAR = 18 + 4 * NS + SCN;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr uint32_t IDESC_QK = idesc_e4m3_f32(128, BN, 0, 0);
  static constexpr uint32_t IDESC_PV = idesc_e4m3_f32(128, DN, 0, 1);
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
  static_assert(TM_OH + D - DN <= 512, "TMEM budget");
};

FKV_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
FKV_DEV uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster: earlier writes of all are visible behind it.
FKV_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared location `p` in CTA `rank` of the cluster, and loads from there.
FKV_DEV uint32_t peer_address(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
FKV_DEV float peer_ld(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
FKV_DEV float4 peer_ld4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Where a tile's keys and values go: by itself to the output, shared by a cluster's CTAs, or as a piece.
enum TileMode { kAlone, kClusters, kPieces };

// kPieces: the KV head, the sequence whose row of the block table names the keys, the first of them that any row may see, and the piece's
// place: o [D / 4][128 rows] of four columns and lse [128] (base 2; -kHuge: the row saw nothing, +infinity: NaN).
struct Piece {
  int g, table_row, kv_lo;
  float4* o;
  float* lse;
};

// Query tile qt of sequence blockIdx.z and KV head blockIdx.y (kPieces: of rows r0 ..., Lq tokens of different sequences, each of which
// sees keys below T unless its context is shorter than T: then none); kClusters: a cluster's CTAs, `shares` of them at most, share
// its keys.
template <int D, bool WIN, TileMode MODE>
FKV_DEV void attend_tile(const BlockPrefillParams& p, const CUtensorMap& tmk, const CUtensorMap& tmv, int r0, int Lq, int T, int qt,
                         int share, int shares, const Piece& piece = Piece()) {
  constexpr bool SPLIT = MODE == kClusters, PIECES = MODE == kPieces;
  using C = BlockPrefillCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sP = smem + C::OFF_P;
  float2* sF = reinterpret_cast<float2*>(smem + C::OFF_F);
  float* sSc = reinterpret_cast<float*>(smem + C::OFF_SC);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars + 0;
  uint64_t* s_full = bars + 1;      // [2] S(t) in buffer t % SBUF
  uint64_t* s_free = bars + 3;      // [2]
  uint64_t* p_full = bars + 5;      // [2] P(t) in buffer t % PBUF
  uint64_t* p_free = bars + 7;      // [2]
  uint64_t* o_full = bars + 9;      // [2] P.V pass n in buffer n % 2
  uint64_t* o_free = bars + 11;     // [2]
  uint64_t* mma_done = bars + 13;
  uint64_t* f_full = bars + 14;     // [2] factors of tile t in slot t % 2 (tile n_t: the rows' l)
  uint64_t* f_free = bars + 16;     // [2]
  uint64_t* k_full = bars + 18;
  uint64_t* k_empty = k_full + C::NS;
  uint64_t* v_full = k_empty + C::NS;
  uint64_t* v_empty = v_full + C::NS;
  uint64_t* sc_full = v_empty + C::NS;  // [SCN] scales of tile t in slot t % SCN
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  // query heads [h_first, h_first + GC) of KV head g: the whole group, or a part of it when it has
  // more than 128 heads
  const int g = PIECES ? piece.g : blockIdx.y / p.head_parts, part = PIECES ? 0 : blockIdx.y - g * p.head_parts;
  const int GC = p.part_heads, h_first = part * GC;
  const int tok = p.part_tokens;              // tokens per CTA
  const int b = PIECES ? piece.table_row : blockIdx.z;
  const int q0 = qt * tok;  // first token of the CTA
  const int toks = min(tok, Lq - q0);
  const int pos0 = T - Lq + q0;  // absolute position of the first token (may be negative when not causal)
  const int kv_end = !PIECES && p.causal ? min(T, pos0 + toks) : T;  // keys [kv_lo, kv_end) matter
  const int kv_lo = PIECES ? piece.kv_lo : WIN ? max(0, pos0 - p.window + 1) : 0;
  // tiles u = 0 .. n_t-1 are tb + u; SPLIT: this CTA's share of them
  const int tb0 = kv_lo / C::BN, n_all = (kv_end + C::BN - 1) / C::BN - tb0;
  if constexpr (SPLIT) {
    // two tiles at least for each that shares; the others of the cluster have no part
    if (!p.even_waves) shares = max(1, min(shares, n_all / 2));
    if (share >= shares) {
      griddep_launch_dependents();
      if (shares > 1) {
        cluster_sync();
        cluster_sync();
      }
      return;
    }
  }
  const int tb = tb0 + share * n_all / shares;
  const int n_t = tb0 + (share + 1) * n_all / shares - tb;
  const int nblk_seq = (T + 15) >> 4;

  if (threadIdx.x == 0) {
    // barriers signalled by the softmax or correction warps count warps (one arrival each)
    mbar_init(q_full, C::SW);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], C::SW);
      mbar_init(&p_full[i], C::SW);
      mbar_init(&p_free[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&f_full[i], C::SW);
      mbar_init(&f_free[i], 4);
    }
    mbar_init(mma_done, 2);  // one commit from each MMA warp
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < C::SCN; ++s) mbar_init(&sc_full[s], 1);
    *abort_s = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();

  if (warp < C::SW) {
    // ============================================================ softmax warps
    if constexpr (C::REG_SOFT < C::REG_LAUNCH) regs_dec<C::REG_SOFT>();
    const int hf = lane >> 4;                                  // column half
    const int rb = (warp & 3) * 32 + (warp >> 2) * 16;         // first TMEM lane
    const int i = rb + (lane & 15);                            // row (TMEM lane i)
    const int it = i / GC, h = h_first + i - it * GC;          // its token and head of the group
    const bool row_ok = it < toks && h < G;
    const bool live = __any_sync(0xffffffffu, row_ok);         // the warp has a row to work on
    const int pos = pos0 + it;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(rb) << 16);
    const int c0 = hf * C::HC;                                 // first column of this thread's half
    float cst;                                                 // c of the row
    // ---- prologue: the row's two terms in the swizzled Q tiles, half of the row per thread
    {
      constexpr int NCH = D / 16;  // 16-byte chunks (8 elements) of half a row
      uint4 w[NCH];
      uint32_t amax = 0;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<long long>(r0 + q0 + it) * p.Hq + g * G + h) * D) + hf * NCH;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        w[c] = row_ok ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t in[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = max(amax, max((in[j] << 16) & 0x7FFF0000u, in[j] & 0x7FFF0000u));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
      const int k = query_exponent(amax);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      // a row with a NaN or an infinity makes its scores, and so its output, NaN
      cst = amax < 0x7F800000u ? p.sm_scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + k) << 23)
                               : __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int c = 0; c < NCH; c += 2) {  // 16 elements: 16 bytes of each term
        const uint32_t in[8] = {w[c].x, w[c].y, w[c].z, w[c].w, w[c + 1].x, w[c + 1].y, w[c + 1].z, w[c + 1].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 x0 = bf16x2_to_f2(in[2 * j]), x1 = bf16x2_to_f2(in[2 * j + 1]);
          x0.x *= down; x0.y *= down; x1.x *= down; x1.y *= down;
          split4_query(x0, x1, hi[j], lo[j]);
        }
        const int byte = hf * (D / 2) + c * 8;
        uint8_t* dst = sQ + (byte / C::RB) * C::SUB + swz(static_cast<uint32_t>(i * C::RB + byte % C::RB), C::RB);
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + C::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(q_full);
    }
    // keys [lo_row, lim_row) visible
    int lim_row = (!PIECES && p.causal && row_ok) ? min(T, pos + 1) : T, lo_row = (!PIECES && WIN && row_ok) ? max(0, pos - p.window + 1) : 0;
    if constexpr (PIECES) {
      // (a context beyond the table is that of the whole table, as for the keys of its own)
      const int ctx = row_ok ? static_cast<int>(min(static_cast<long long>(p.ctx[r0 + q0 + it]), p.max_blocks * 16LL)) : T;
      if (ctx < T) lim_row = 0;
      if (WIN) lo_row = max(0, ctx - p.window);
    }
    float m = -kHuge, l = 0.f;  // r, and l of this thread's columns only
    bool ok = true;
    for (int t = 0; t < n_t; ++t) {
      if ((t & 7) == 7 && abort_warp(abort_s)) { ok = false; break; }
      const int sb = t % C::SBUF, pb = t % C::PBUF;
      if (!pf_wait_warp(&s_full[sb], (t / C::SBUF) & 1)) { ok = false; break; }
      tc_fence_after();
      if (!live) {
        // a warp without rows takes part in the barriers only (what its rows of P hold reaches no
        // other row)
        mbar_arrive_warp(&s_free[sb]);
        if (t >= C::PBUF && !pf_wait_warp(&p_free[pb], ((t / C::PBUF) - 1) & 1)) { ok = false; break; }
        if (t >= 2 && !pf_wait_warp(&f_free[t & 1], ((t >> 1) - 1) & 1)) { ok = false; break; }
        mbar_arrive_warp(&f_full[t & 1]);
        mbar_arrive_warp(&p_full[pb]);
        continue;
      }
      const uint32_t sc = lane_base + 128 * sb;
      float v[C::HC];
#pragma unroll
      for (int c = 0; c < C::HC / 32; ++c) tmem_ld32_16x2<C::HC>(sc + 32 * c, *reinterpret_cast<float(*)[32]>(v + 32 * c));
      const bool p_ready = t < C::PBUF || mbar_test_wait(&p_free[pb], ((t / C::PBUF) - 1) & 1);
      const bool f_ready = t < 2 || mbar_test_wait(&f_free[t & 1], ((t >> 1) - 1) & 1);
      // this half's four blocks: ks, L, 2^(o - L)
      if (!pf_wait_warp(&sc_full[t % C::SCN], (t / C::SCN) & 1)) { ok = false; break; }
      const float* scl = sSc + (t % C::SCN) * C::SCF + 4 * hf;
      const float4 ks4 = *reinterpret_cast<const float4*>(scl), lv4 = *reinterpret_cast<const float4*>(scl + 8),
                   iv4 = *reinterpret_cast<const float4*>(scl + 16);
      const float rare = sSc[(t % C::SCN) * C::SCF + 25];
      // (plus 2^-126, so that a hidden score of -inf stays one where the product is zero: a row of zeros, a
      // K scale of zero; |S| < 2^26, so that this adds less than 2^-100 to a score)
      constexpr float kLeast = 1.17549435e-38f;
      const float cb[4] = {fmaf(cst, ks4.x, kLeast), fmaf(cst, ks4.y, kLeast), fmaf(cst, ks4.z, kLeast), fmaf(cst, ks4.w, kLeast)};
      const int kbase = (tb + t) * C::BN + c0;  // key of this thread's first column
      const int lim = lim_row - kbase, lo = WIN ? lo_row - kbase : -(1 << 30);
      const bool full = lim >= C::HC && (!WIN || lo <= 0);
      const bool wfull = __all_sync(0xffffffffu, full);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive_warp(&s_free[sb]);
      // hidden scores become -inf (2^(-inf) = 0 is the zero the mask asks for), under a test that
      // the whole warp takes alike
      if (!wfull) {
#pragma unroll
        for (int j = 0; j < C::HC; ++j)
          if (j >= lim || j < lo) v[j] = -INFINITY;
      }
      const float lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w};
      float iv[4] = {iv4.x, iv4.y, iv4.z, iv4.w};
      float tmax = -kHuge;  // (finite, so that a row that sees nothing of the tile adds zeros)
#pragma unroll
      for (int k = 0; k < 4; ++k) tmax = fmaxf(tmax, fmaf(max_tree<16>(v + 16 * k), cb[k], lv[k]));
      tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 16));
      // one of the two factors is 1, the other 2^-|m - tmax|
      const float e = ex2(-fabsf(m - tmax));
      float alpha = m > tmax ? 1.f : e, corr = m > tmax ? e : 1.f;
      // the sum's factors: the same, but in a rare tile (block_scales; the same in every thread)
      if (rare == 0.f) {
        l *= alpha;
#pragma unroll
        for (int k = 0; k < 4; ++k) iv[k] *= corr;
        m = fmaxf(m, tmax);
      } else {
        const RareFactors f = rare_factors(m, l, tmax, sSc[(t % C::SCN) * C::SCF + 26]);
        l = l * f.l * f.l * f.l;
#pragma unroll
        for (int k = 0; k < 4; ++k) iv[k] = iv[k] * f.lt * f.lt * f.lt;
        alpha = f.alpha;
        corr = f.beta;
      }
      if (!__all_sync(0xffffffffu, p_ready) && !pf_wait_warp(&p_free[pb], ((t / C::PBUF) - 1) & 1)) { ok = false; break; }
      uint8_t* P = sP + pb * 2 * C::PTERM;
      const float top = tmax - kLog2E4m3Max;
      const float nb[4] = {lv[0] - top, lv[1] - top, lv[2] - top, lv[3] - top};
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // block k: 16 columns, 16 bytes of each term
        const float2 c2 = make_float2(cb[k], cb[k]), n2 = make_float2(nb[k], nb[k]);
        float2 sum = make_float2(0.f, 0.f);
        uint32_t hi[4], lw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 x0 = __ffma2_rn(make_float2(v[16 * k + 4 * j], v[16 * k + 4 * j + 1]), c2, n2);
          float2 x1 = __ffma2_rn(make_float2(v[16 * k + 4 * j + 2], v[16 * k + 4 * j + 3]), c2, n2);
          x0.x = ex2(x0.x); x0.y = ex2(x0.y); x1.x = ex2(x1.x); x1.y = ex2(x1.y);
          sum = __fadd2_rn(sum, __fadd2_rn(x0, x1));
          split4<true>(x0, x1, hi[j], lw[j]);
        }
        l = fmaf(sum.x + sum.y, fabsf(iv[k]), l);
        uint8_t* dst = P + swz(static_cast<uint32_t>(i * 128 + c0 + 16 * k), 128);
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + C::PTERM) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
      if (rare != 0.f) {  // a scale that counts as zero has no P (unrolled here: 1,098 us on 2,048 queries over 32,768 keys
                          // at head_dim 128, rolled 1,141, behind the factors 1,118)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (iv[k] > 0.f) continue;
          uint8_t* dst = P + swz(static_cast<uint32_t>(i * 128 + c0 + 16 * k), 128);
          *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(dst + C::PTERM) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (!__all_sync(0xffffffffu, f_ready) && !pf_wait_warp(&f_free[t & 1], ((t >> 1) - 1) & 1)) { ok = false; break; }
      if (hf == 0) sF[(t & 1) * C::BM + i] = make_float2(alpha, corr);
      mbar_arrive_warp(&f_full[t & 1]);
      fence_proxy_async_smem();
      mbar_arrive_warp(&p_full[pb]);
    }
    tmem_ld_wait();  // no load left in flight on an early exit
    // ---- the rows' 1 / l and 2^o take the factor slot after the last tile's; SPLIT: the log2-sum-exp
    // (log2 448 too large in every share; -kHuge for a row that sees nothing) lies over the query, whose
    // products are done (without a tile: which every warp has written)
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    const float o = n_t > 0 ? sSc[((n_t - 1) % C::SCN) * C::SCF + 24] : 0.f;
    if (ok && n_t >= 2) ok = pf_wait_warp(&f_free[n_t & 1], ((n_t >> 1) - 1) & 1);
    if (SPLIT && ok && n_t == 0) ok = pf_wait_warp(q_full, 0);
    if (ok) {
      if (hf == 0) {
        sF[(n_t & 1) * C::BM + i] = make_float2(l == 0.f ? 0.f : 1.f / l, pow2i(o));  // (a row that sees no key: zero)
        if constexpr (SPLIT) reinterpret_cast<float*>(sQ)[i] = l == 0.f ? -kHuge : m - o + lg2(l);
        if constexpr (PIECES) piece.lse[i] = l == 0.f ? -kHuge : l > 0.f ? m - o + lg2(l) - kLog2E4m3Max : INFINITY;
      }
      mbar_arrive_warp(&f_full[n_t & 1]);
    } else {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
  } else if (warp < C::SW + 4) {
    // ============================================================ correction warpgroup
    regs_inc<C::REG_CORR>();
    const int i = threadIdx.x - 32 * C::SW;    // row (TMEM lane i)
    const int it = i / GC, h = h_first + i - it * GC;
    const bool row_ok = it < toks && h < G;
    const bool live = __any_sync(0xffffffffu, row_ok);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp - C::SW) * 32) << 16);
    bool ok = true;
    float O[C::DN];  // acc, columns [0, DN)
#pragma unroll
    for (int j = 0; j < C::DN; ++j) O[j] = 0.f;
    for (int t = 0; t < n_t; ++t) {
      if ((t & 7) == 7 && abort_warp(abort_s)) { ok = false; break; }
      if (!pf_wait_warp(&f_full[t & 1], (t >> 1) & 1)) { ok = false; break; }
      const float2 f = sF[(t & 1) * C::BM + i];
      mbar_arrive_warp(&f_free[t & 1]);
      const float2 a2 = make_float2(f.x, f.x), b2 = make_float2(f.y, f.y);
#pragma unroll
      for (int hn = 0; hn < C::NH; ++hn) {
        const int n = C::NH * t + hn, ob = n & 1;
        if (!pf_wait_warp(&o_full[ob], (n >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t src = lane_base + C::TM_OT + ob * C::DN;
        if (!live) {
          // no rows
        } else if (hn == 0) {
#pragma unroll
          for (int c = 0; c < C::DN / 32; ++c) {
            float o[32];
            tmem_ld32(src + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 x = __fmul2_rn(make_float2(o[j], o[j + 1]), b2);
              const float2 r = __ffma2_rn(make_float2(O[32 * c + j], O[32 * c + j + 1]), a2, x);
              O[32 * c + j] = r.x;
              O[32 * c + j + 1] = r.y;
            }
            pin32(O + 32 * c);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < C::DN / 32; ++c) {
            float o[32], acc[32];
            const uint32_t dst = lane_base + C::TM_OH + 32 * c;
            tmem_ld32(src + 32 * c, o);
            if (t > 0) tmem_ld32(dst, acc);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 x = __fmul2_rn(make_float2(o[j], o[j + 1]), b2);
              const float2 r = t > 0 ? __ffma2_rn(make_float2(acc[j], acc[j + 1]), a2, x) : x;
              acc[j] = r.x;
              acc[j + 1] = r.y;
            }
            tmem_st32(dst, acc);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive_warp(&o_free[ob]);
      }
      if (!ok) break;
    }
    // ---- epilogue (every lane loads; rows past the chunk do not store): 2^o acc / l as bf16, or
    // with SPLIT in float32, into shared memory over the K and V stages, whose copies and products are
    // all done: four columns of a row at [column / 4][row]
    if (ok) ok = pf_wait_warp(&f_full[n_t & 1], (n_t >> 1) & 1);
    if (!ok) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    } else {
      const float2 f = sF[(n_t & 1) * C::BM + i];
      __nv_bfloat16* dst = p.out + (static_cast<long long>(r0 + q0 + it) * p.Hq + g * G + h) * D;
      float4* part = reinterpret_cast<float4*>(sK);
      auto store32 = [&](int c, const float* x) {
        if (!row_ok) return;
        if constexpr (PIECES) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            piece.o[(8 * c + j) * C::BM + i] =
                make_float4(x[4 * j] * f.x * f.y, x[4 * j + 1] * f.x * f.y, x[4 * j + 2] * f.x * f.y, x[4 * j + 3] * f.x * f.y);
          return;
        }
        if (SPLIT && shares > 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            part[(8 * c + j) * C::BM + i] =
                make_float4(x[4 * j] * f.x * f.y, x[4 * j + 1] * f.x * f.y, x[4 * j + 2] * f.x * f.y, x[4 * j + 3] * f.x * f.y);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * j] * f.x * f.y, x[2 * j + 1] * f.x * f.y);
            w[j] = *reinterpret_cast<const uint32_t*>(&y);
          }
          uint4* o4 = reinterpret_cast<uint4*>(dst + 32 * c);
#pragma unroll
          for (int j = 0; j < 4; ++j) o4[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
      };
#pragma unroll
      for (int c = 0; c < C::DN / 32; ++c) store32(c, O + 32 * c);
      if constexpr (C::NH == 2) {
#pragma unroll 1
        for (int c = 0; c < C::DN / 32; ++c) {
          float acc[32];
          if (n_t > 0) {
            tmem_ld32(lane_base + C::TM_OH + 32 * c, acc);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[j] = 0.f;
          }
          store32(C::DN / 32 + c, acc);
        }
      }
    }
  } else {
    if constexpr (C::REG_MISC < C::REG_LAUNCH) regs_dec<C::REG_MISC>();
    if (warp == 12 || warp == 15) {
      // ============================================================ copies: K (12), V (15)
      // Lane j < 8 copies the tile's j-th block; block ids are read two tiles ahead, scales (K
      // warp) one.
      const bool is_k = warp == 12;
      uint64_t* full = is_k ? k_full : v_full;
      uint64_t* empty = is_k ? k_empty : v_empty;
      uint8_t* base = is_k ? sK : sV;
      const CUtensorMap* map = is_k ? &tmk : &tmv;
      const int* trow = p.block_table + static_cast<size_t>(b) * p.max_blocks;
      int last[C::NS];  // last use of each stage whose copies were issued
#pragma unroll
      for (int s = 0; s < C::NS; ++s) last[s] = -1;
      // block id, -1 past the sequence and before the first visible key's block, whose table entry may
      // name a block no longer (copied from block 0, its keys masked)
      auto block_id = [&](int t) -> int {
        const int lb = (tb + t) * C::NBLK + lane;
        if (lane >= C::NBLK || t >= n_t || lb >= nblk_seq || lb < kv_lo >> 4) return -1;
        const int id = trow[lb];
        if (id >= 0 && id < p.num_blocks) return id;
        raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
        return 0;
      };
      ScaleRange range;
      float ks_n = 0.f, vs_n = 0.f;
      auto read_scales = [&](int id) {
        ks_n = vs_n = 0.f;
        if (is_k && id >= 0) {
          const size_t at = static_cast<size_t>(id) * p.Hkv + g;
          ks_n = p.k_scale[at];
          vs_n = p.v_scale[at];
        }
      };
      int id = block_id(0), id_next = block_id(1);
      read_scales(id);
      for (int t = 0; t < n_t; ++t) {
        if (abort_warp(abort_s)) break;
        const float ks = ks_n, vs = vs_n;
        const int id_t = max(id, 0);
        read_scales(id_next);
        id = id_next;
        id_next = block_id(t + 2);
        const int st = t % C::NS, use = t / C::NS;
        bool ok = true;
        if (lane == 0 && use > 0) ok = pf_wait(&empty[st], (use - 1) & 1, p.stage_wait_ns);
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) {
          if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
          *abort_s = 1;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[st], C::TILE);
        __syncwarp();
        if (lane < C::NBLK) {
          uint8_t* dst = base + st * C::TILE + lane * 16 * C::RB;
#pragma unroll
          for (int s = 0; s < C::NSUB; ++s) tma_load_4d(dst + s * C::SUB, map, s * C::RB, 0, g, id_t, &full[st]);
        }
        last[st] = use;
        if (is_k) {
          // the tile's scales, those of blocks that no row of this CTA sees left out
          const int lb = (tb + t) * C::NBLK + lane;
          const BlockScale sc = block_scales(range, vs, lane < C::NBLK && lb >= kv_lo >> 4 && lb < (kv_end + 15) >> 4);
          float* slot = sSc + (t % C::SCN) * C::SCF;
          if (lane < C::NBLK) {
            slot[lane] = ks;
            slot[8 + lane] = sc.lv;
            slot[16 + lane] = sc.iv;
          }
          if (lane == 0) {
            slot[24] = range.o;
            slot[25] = sc.rare ? 1.f : 0.f;
            slot[26] = sc.change;
          }
          mbar_arrive_warp(&sc_full[t % C::SCN]);
        }
      }
      // let every issued copy land before the CTA can exit
      if (lane == 0)
        for (int s = 0; s < C::NS; ++s)
          if (last[s] >= 0) pf_wait(&full[s], last[s] & 1);
      __syncwarp();
    } else {
      // ============================================================ MMA issuers: S (13), P.V (14)
      const uint64_t dQ = smem_desc(smem_u32(sQ), 16, 8 * C::RB, C::SWZ);
      const uint64_t dK = smem_desc(smem_u32(sK), 16, 8 * C::RB, C::SWZ);
      const uint64_t dV = smem_desc(smem_u32(sV), 8 * C::RB, 8 * C::RB, C::SWZ);
      const uint64_t dP = smem_desc(smem_u32(sP), 16, 1024, 2);
      bool ok = true;
      if (warp == 13) {
        ok = pf_wait_warp(q_full, 0);
        for (int t = 0; ok && t < n_t; ++t) {
          if ((t & 7) == 7 && abort_warp(abort_s)) break;
          const int st = t % C::NS, sb = t % C::SBUF;
          ok = pf_wait_warp(&k_full[st], (t / C::NS) & 1);
          if (ok && t >= C::SBUF) ok = pf_wait_warp(&s_free[sb], ((t / C::SBUF) - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            // S(t) = hi K8^T + lo K8^T
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {
                const int byte = kk * 32;
                const uint32_t off = (byte / C::RB) * C::SUB + (byte % C::RB);
                umma_f8(tmem + 128 * sb, desc_add(dQ, term * C::TILE + off), desc_add(dK, st * C::TILE + off), C::IDESC_QK,
                        (term > 0 || kk > 0) ? 1u : 0u);
              }
            umma_commit(&s_full[sb]);
            umma_commit(&k_empty[st]);
          }
          __syncwarp();
        }
      } else {
        int n = 0;  // P.V passes issued
        for (int t = 0; ok && t < n_t; ++t) {
          if ((t & 7) == 7 && abort_warp(abort_s)) break;
          const int st = t % C::NS, pb = t % C::PBUF;
          ok = pf_wait_warp(&p_full[pb], (t / C::PBUF) & 1) && pf_wait_warp(&v_full[st], (t / C::NS) & 1);
          if (!ok) break;
          // keys past the context, and before a window, may hold any bytes (NaN codes): zero their V
          // rows, since 0 * NaN would poison the product even though their P is 0
          const int kbase = (tb + t) * C::BN;
          const int keep_lo = max(kv_lo - kbase, 0), keep_hi = min(T - kbase, C::BN);
          if (keep_lo > 0 || keep_hi < C::BN) {
            constexpr int CPR = C::RB / 16;  // 16-byte chunks of a row
            for (int x = lane; x < C::BN * C::NSUB * CPR; x += 32) {
              const int c = x % CPR, s = (x / CPR) % C::NSUB, r = x / (CPR * C::NSUB);
              if (r < keep_lo || r >= keep_hi)
                *reinterpret_cast<uint4*>(sV + st * C::TILE + s * C::SUB + r * C::RB + c * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int hn = 0; hn < C::NH; ++hn, ++n) {
            // O_t buffer n % 2 is free once the correction took pass n - 2
            const int ob = n & 1;
            if (n >= 2 && !pf_wait_warp(&o_free[ob], ((n >> 1) - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int kk = 0; kk < C::BN / 32; ++kk)
                  umma_f8(tmem + C::TM_OT + ob * C::DN, desc_add(dP, pb * 2 * C::PTERM + term * C::PTERM + kk * 32),
                          desc_add(dV, st * C::TILE + hn * C::SUB + kk * 32 * C::RB), C::IDESC_PV,
                          (term > 0 || kk > 0) ? 1u : 0u);
              umma_commit(&o_full[ob]);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (lane == 0) {
            umma_commit(&v_empty[st]);
            umma_commit(&p_free[pb]);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
        *abort_s = 1;
      }
      // every product issued by either warp completes before TMEM is released
      if (lane == 0) {
        umma_commit(mma_done);
        pf_wait(mma_done, 0);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  if (SPLIT && shares > 1) {
    // the shares (o, lse)_r of every row: M = max lse_r, out = sum 2^(lse_r - M) o_r / sum 2^(lse_r - M), by the
    // softmax warps, whose register budget holds it
    cluster_sync();
    const int rows = toks * GC;
    constexpr int kMergers = 32 * C::SW;
    for (int e = warp < C::SW ? share * kMergers + threadIdx.x : rows * D; e < rows * (D / 4); e += kMergers * shares) {
      const int c = e / rows, i = e - c * rows;
      const int it = i / GC, h = h_first + i - it * GC;
      if (h >= G) continue;
      float M = -kHuge, L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r = 0; r < shares; ++r) {
        const float lse = peer_ld(peer_address(reinterpret_cast<float*>(sQ) + i, r));
        const float4 x = peer_ld4(peer_address(reinterpret_cast<float4*>(sK) + c * C::BM + i, r));
        const float mx = fmaxf(M, lse), a = ex2(M - mx), w = ex2(lse - mx);
        M = mx;
        L = fmaf(L, a, w);
        o.x = fmaf(o.x, a, w * x.x);
        o.y = fmaf(o.y, a, w * x.y);
        o.z = fmaf(o.z, a, w * x.z);
        o.w = fmaf(o.w, a, w * x.w);
      }
      const float f = 1.f / L;
      __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out + (static_cast<long long>(r0 + q0 + it) * p.Hq + g * G + h) * D + 4 * c);
      dst[0] = __floats2bfloat162_rn(o.x * f, o.y * f);
      dst[1] = __floats2bfloat162_rn(o.z * f, o.w * f);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
}

}  // namespace
}  // namespace fkv
