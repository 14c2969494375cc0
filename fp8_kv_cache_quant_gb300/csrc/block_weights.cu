// The attention weight that the cached keys of a block-scaled pool receive from a chunk of queries, summed over the
// queries and the heads of a KV head's group, on tcgen05 tensor cores.
//
// Mathematics.  A row r is a (token, head of the group) pair, r = token * G + head; x_rj = q_r . k_j * ks_j * c, c =
// softmax_scale log2(e), in base 2.  lse_r = log2 sum_j 2^(x_rj) over the keys that the row sees, and
//   w_j = sum_r 2^(x_rj - lse_r).
// No weight is final before every key of a row has been scored, so the keys are gone over twice.  Products are FP8: the
// bf16 query as two e4m3 terms on its row's own power of two (split4_query), K as it lies in the cache, FP32 sums.
//
// Few rows (at most 16 per sequence and KV head: decode steps, drafts): one walk over K writes the scores, 16 to 64 bytes a key
// where K has 64 to 256, and the rows' sums; a second kernel reads them back (from L2 as a rule) and adds up (score_kernel,
// gather_kernel).
// More rows: a score costs an exponential, which the GPU makes 32 of per clock and SM, in each of two passes, and writing it
// down would cost more than making it again.  query_kernel lays the rows out in tiles of 128 as the products want
// them; pass 0 takes rows as the MMA's M side (a thread owns a row, its maximum and sum stay in registers), pass 1 keys (a
// thread owns a key, the sum over the rows stays in a register), so that neither needs a sum across threads in its loop.
//
// Work.  Lengths are known on the GPU alone.  The steps of a pass (a tile against a tile) of all units (sequence, KV head, row tile
// or key tile) stand in a row, and every resident CTA takes the same number of them; a unit in several CTAs' ranges is joined by the
// one that brings its last piece, in the order of the pieces, so that the same sizes give the same bits.
//
// What bounds it.  Few rows: K's bytes, and the scores' way through L2: 8 sequences of 16k-24k tokens, 32/8 heads of 128, 44 us (163 MB
// of K; 34 us score_kernel and 10 gather_kernel one by one, cold).  More rows: a step of pass 0 (128 rows against 128 keys) takes 1,150
// cycles, its products 540 and its exponentials 512, and a piece's end and beginning in pass 1 as much as its 256 keys; 32 queries of
// four sequences of 7k-16k, 32/8 heads of 128, 54 us, of which each pass needs 5 to find its work and its first tiles; a whole prompt of
// 4,001 tokens, 8/1 heads of 256, 95 us, where the products and the copies of the rows' tiles (64 KB each) set the pace.
// Every wait is bounded in time; a timeout records FKV_FAULT_TIMEOUT, lets the CTA's copies and products drain and returns.
#include "block_common.cuh"
#include "prefill_common.cuh"
#include "tc.cuh"

namespace fkv {
namespace {

constexpr float kHuge = 3e38f;  // minus this: the maximum of no scores

// Sequence b's rows and keys; rows 0: nothing to do.  back: the starts decrease behind it.
struct WeightsSeq {
  int r0, rows, T;
  bool back;
  FKV_DEV int end() const { return rows > 0 ? r0 + rows : 0; }
};
FKV_DEV WeightsSeq weights_seq(const BlockWeightsParams& p, int b, bool report) {
  WeightsSeq s;
  s.r0 = p.cu[b];
  s.rows = p.cu[b + 1] - s.r0;
  s.back = s.rows < 0;
  s.T = p.ctx[b];
  const long long most = min(p.max_blocks * 16LL, static_cast<long long>(p.weights_len));
  if (s.T < 0 || s.T > most) {
    if (report) raise_fault(p.fault, FKV_FAULT_CONTEXT);
    s.T = s.T < 0 ? 0 : static_cast<int>(most);
  }
  if (s.rows < 0 || s.rows > p.max_q_len || s.rows > s.T || s.r0 < 0 || s.r0 + static_cast<long long>(s.rows) > p.total_q) {
    if (report) raise_fault(p.fault, FKV_FAULT_QLEN);
    s.rows = 0;
  }
  return s;
}

// ---------------------------------------------------------------- the division of the work

// What a kernel divides: kRows: row tiles against the key tiles (of 128) that they see (pass 0); kKeys: key tiles of KT keys against
// the row tiles that see them (pass 1); kScores: all of a KV head's key tiles of KT keys as one unit.
enum Kind { kRows, kKeys, kScores };

// A piece: the steps of a unit that a CTA takes.  (Rows and keys of a sequence are below 2^31, rows times G at most 2^30.)
// The row tiles have their places in the workspace by the sequences' first rows (tile_index).  Where the starts decrease, a sequence
// whose rows do not lie behind those of all earlier ones would share places with them, and is left out (kRows, kKeys).
template <Kind K, int KT>
struct Walk {
  int G;
  int b, g, t, of;        // unit t of the `of` of (sequence b, KV head g)
  int r0, rows, T;        // the sequence
  int s, n, count;        // steps s .. s + n - 1 of its count; n 0: behind the range
  int left;               // steps of the range behind this piece
  int piece;              // pieces before this one
  int top;                // the rows of sequences up to this one end at or before it (0 where the starts do not decrease)
  long long unit0;        // the place of the unit's first step

  FKV_DEV void set(const WeightsSeq& q) {
    r0 = q.r0;
    rows = q.rows;
    T = q.T;
    of = rows == 0 ? 0 : K == kRows ? tiles() : K == kKeys ? (T + KT - 1) / KT : 1;
  }
  FKV_DEV int old() const { return T - rows; }
  FKV_DEV int tiles() const { return (rows * G + 127) / 128; }
  // the first step's tile: 0, or the first row tile that sees key tile x
  FKV_DEV int first(int x) const { return K == kKeys ? max(KT * x - old(), 0) * G / 128 : 0; }
  FKV_DEV int first() const { return first(t); }
  FKV_DEV int steps(int x) const {
    if (K == kScores) return (T + KT - 1) / KT;
    if (K == kKeys) return tiles() - first(x);
    return (old() + (min(128 * (x + 1), rows * G) - 1) / G) / 128 + 1;
  }
  FKV_DEV bool whole() const { return n == count; }
  FKV_DEV void next(const BlockWeightsParams& p) {
    n = 0;
    if (left == 0) return;
    ++piece;
    unit0 += count;
    if (++t == of) {
      t = 0;
      if (++g == p.Hkv) {
        g = 0;
        do {
          WeightsSeq q = weights_seq(p, ++b, false);
          if constexpr (K != kScores) {
            const int end = q.end();
            if (q.r0 < top) q.rows = 0;
            top = max(top, end);
          }
          set(q);
        } while (of == 0);
      }
    }
    count = steps(t);
    s = 0;
    n = min(count, left);
    left -= n;
  }
};

// The range of CTA k of the grid: its first piece, and W and N, the steps in all and the CTAs that have some.  By one warp.
template <Kind K, int KT>
FKV_DEV Walk<K, KT> first_piece(const BlockWeightsParams& p, int k, long long& W, int& N, bool report) {
  const int lane = threadIdx.x & 31;
  Walk<K, KT> a;
  a.G = p.Hq / p.Hkv;
  a.b = a.g = a.t = a.s = a.n = a.count = a.left = a.piece = a.top = 0;
  a.unit0 = 0;
  a.set(WeightsSeq{0, 0, 0, false});
  auto sum = [](long long x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
  };
  auto upto = [&](long long x) {  // inclusive sums over the lanes
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    return x;
  };
  // a sequence's steps for one KV head: by one lane where it has few units, by all of them where it may have many
  const bool by_lane = K != kRows || p.max_q_len * static_cast<long long>(a.G) <= 512;
  auto steps_of = [&](const WeightsSeq& q) -> long long {
    Walk<K, KT> c = a;
    c.set(q);
    if (c.of == 0) return 0;
    if constexpr (K == kScores) {
      return c.steps(0);
    } else if constexpr (K == kKeys) {
      // key tiles that begin before the chunk or with it are seen by every row tile, those behind by KT / 128 G fewer each
      const int nt = c.tiles(), nk = c.of, t1 = min(c.old() / KT + 1, nk), n = nk - t1;
      const long long G = c.G;
      const long long skipped = KT / 128 * G * (static_cast<long long>(t1) * n + static_cast<long long>(n) * (n - 1) / 2) - n * ((c.old() * G + 127) / 128);
      return static_cast<long long>(nt) * nk - skipped;
    } else {
      long long x = 0;
      for (int t = by_lane ? 0 : lane; t < c.of; t += by_lane ? 1 : 32) x += c.steps(t);
      return by_lane ? x : sum(x);
    }
  };
  const int db = by_lane ? 32 : 1;
  auto seq_at = [&](int b0, bool rep) {
    const int b = by_lane ? b0 + lane : b0;
    return b < p.B ? weights_seq(p, b, rep && (by_lane || lane == 0)) : WeightsSeq{0, 0, 0, false};
  };
  // where the starts decrease: the sequence left out if it does not lie behind those before it, whose rows end at top
  bool back = false;
  int top = 0;
  auto check = [&](WeightsSeq& q) {  // returns where the rows up to this lane's sequence end
    if (!by_lane) {
      const int end = q.end();
      if (q.r0 < top) q.rows = 0;
      return top = max(top, end);
    }
    int end = max(top, q.end());
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, off);
      if (lane >= off) end = max(end, y);
    }
    const int before = __shfl_up_sync(0xffffffffu, end, 1);
    if (q.r0 < (lane > 0 ? before : top)) q.rows = 0;
    top = __shfl_sync(0xffffffffu, end, 31);
    return end;
  };
  long long first32 = 0;
#pragma unroll 1
  for (int go = 0; go < 2; ++go) {
    bool decrease = false;
    W = 0;
    for (int b0 = 0; b0 < p.B; b0 += db) {
      WeightsSeq q = seq_at(b0, report && go == 0);
      decrease = decrease || q.back;
      if (back) check(q);
      const long long x = steps_of(q);
      if (b0 == 0) first32 = x;
      W += by_lane ? sum(x) : x;
    }
    if (K == kScores || go > 0 || !__any_sync(0xffffffffu, decrease)) break;
    back = true;
  }
  W *= p.Hkv;
  N = static_cast<int>(min(static_cast<long long>(gridDim.x), W));
  if (k >= N) return a;
  const bool small = W < (1LL << 31) / N;
  const long long w0 = small ? static_cast<uint32_t>(W) * k / static_cast<uint32_t>(N) : W * k / N;
  const long long w1 = small ? static_cast<uint32_t>(W) * (k + 1) / static_cast<uint32_t>(N) : W * (k + 1) / N;
  long long base = 0, mine = 0;  // places before sequence b, and one KV head's of it
  top = 0;
  for (int b0 = 0;; b0 += db) {
    long long x = first32;
    int end = 0;
    if (back || b0 > 0) {
      WeightsSeq q = seq_at(b0, false);
      if (back) end = check(q);
      x = steps_of(q);
    }
    const long long y = by_lane ? upto(x) : x;
    const unsigned past = __ballot_sync(0xffffffffu, base + y * p.Hkv > w0);
    if (past != 0) {
      const int j = by_lane ? __ffs(past) - 1 : 0;
      a.b = b0 + j;
      a.top = __shfl_sync(0xffffffffu, end, j);
      mine = __shfl_sync(0xffffffffu, x, j);
      base += (__shfl_sync(0xffffffffu, y, j) - mine) * p.Hkv;
      break;
    }
    base += __shfl_sync(0xffffffffu, y, 31) * p.Hkv;
  }
  a.set(weights_seq(p, a.b, false));
  const long long in = w0 - base;
  a.g = small ? static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(mine)) : static_cast<int>(in / mine);
  const long long rem = in - a.g * mine;
  long long before = 0;  // steps of the units before t0
  for (int t0 = 0; t0 < a.of; t0 += 32) {
    const int n = t0 + lane < a.of ? a.steps(t0 + lane) : 0;
    const long long y = before + upto(n);
    const unsigned past = __ballot_sync(0xffffffffu, y > rem);
    if (past != 0) {
      const int j = __ffs(past) - 1;
      a.t = t0 + j;
      a.count = __shfl_sync(0xffffffffu, n, j);
      a.s = static_cast<int>(rem - (__shfl_sync(0xffffffffu, y, j) - a.count));
      break;
    }
    before = __shfl_sync(0xffffffffu, y, 31);
  }
  a.unit0 = w0 - a.s;
  a.n = static_cast<int>(min(static_cast<long long>(a.count - a.s), w1 - w0));
  a.left = static_cast<int>(w1 - w0 - a.n);
  return a;
}

// The division as the CTA's warps share it.
template <Kind K, int KT>
struct Division {
  Walk<K, KT> first;
  long long W;
  int N;
};

// The CTA whose range holds place w: the largest k with floor(W k / N) <= w.
FKV_DEV int cta_of(long long w, long long W, int N) { return static_cast<int>(((w + 1) * N - 1) / W); }

// A unit's pieces lie at place 2 k0 + 1 (the CTA that begins it, whose last unit it is) and at 2 k of those behind it.
FKV_DEV long long piece_place(int k, int k0) { return k == k0 ? 2LL * k + 1 : 2LL * k; }

// Add 1 to a counter with release and acquire semantics at GPU scope.
FKV_DEV int count_piece(int32_t* p) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

// Index of row tile i of (b, g) among the tiles of the workspace, r0 the sequence's first row.
FKV_DEV size_t tile_index(const BlockWeightsParams& p, int r0, int b, int g, int i) {
  return (static_cast<size_t>(r0) * (p.Hq / p.Hkv) / 128 + b + i) * p.Hkv + g;
}

// The block ids and K scales of the key tiles that a range of steps goes through, for the warp that copies them: as many tiles as a warp
// has lanes for their blocks (a batch) are read at once, the ids two batches and the scales one ahead.  Tile by tile and one ahead, a step
// took a round trip to memory, 1.0 us, whatever else it did.
template <Kind K, int KT>
struct KeyFeed {
  static constexpr int TB = KT / 16, BATCH = 32 / TB;
  struct Read {
    int id, g;
    bool in;
  };
  Walk<K, KT> ahead;    // the piece, and which of its steps, whose tile this lane reads next
  int step;
  Read now, next, last;
  float ks, ks_next;
  int taken;

  static FKV_DEV int blocks_of(const Walk<K, KT>& a, int tile) { return min(TB, ((a.T + 15) >> 4) - TB * tile); }
  FKV_DEV void skip(const BlockWeightsParams& p, int x) {  // x key tiles on
    if (K == kKeys) {
#pragma unroll 1
      for (; x > 0 && ahead.n > 0; --x) ahead.next(p);
    } else {
      step += x;
#pragma unroll 1
      while (ahead.n > 0 && step >= ahead.n) {
        step -= ahead.n;
        ahead.next(p);
      }
    }
  }
  FKV_DEV Read read(const BlockWeightsParams& p) {
    const int j = (threadIdx.x & 31) % TB, tile = K == kKeys ? ahead.t : ahead.s + step;
    Read x = {0, ahead.g, ahead.n > 0 && j < blocks_of(ahead, tile)};
    if (x.in) x.id = p.block_table[static_cast<size_t>(ahead.b) * p.max_blocks + TB * tile + j];
    skip(p, BATCH);
    return x;
  }
  // an id out of range reads block 0 and is reported
  static FKV_DEV float scale_of(Read& x, const BlockWeightsParams& p) {
    if (!x.in) return 0.f;
    if (x.id < 0 || x.id >= p.num_blocks) {
      raise_fault(p.fault, FKV_FAULT_BLOCK_ID);
      x.id = 0;
    }
    return p.k_scale[static_cast<size_t>(x.id) * p.Hkv + x.g];
  }
  FKV_DEV void begin(const Walk<K, KT>& at, const BlockWeightsParams& p) {
    ahead = at;
    step = 0;
    skip(p, (threadIdx.x & 31) / TB);
    now = read(p);
    next = read(p);
    ks = scale_of(now, p);
    last = read(p);
    ks_next = scale_of(next, p);
    taken = 0;
  }
  // the next tile's: lane j < TB has block j's
  FKV_DEV void take(const BlockWeightsParams& p, int& id, float& scale) {
    const int j = taken % BATCH;
    if (taken > 0 && j == 0) {
      now = next;
      ks = ks_next;
      next = last;
      ks_next = scale_of(next, p);
      last = read(p);
    }
    const int from = TB * j + (threadIdx.x & 31) % TB;
    id = __shfl_sync(0xffffffffu, now.id, from);
    scale = __shfl_sync(0xffffffffu, ks, from);
    ++taken;
  }
};

template <int D>
struct Shape {
  static constexpr int RB = D < 128 ? D : 128;   // bytes of one swizzled row
  static constexpr int NSUB = D / RB;            // sub-tiles along head_dim
  static constexpr int SWZ = RB == 128 ? 2 : 4;  // descriptor swizzle mode (128 B / 64 B)
  static constexpr int SUB = 128 * RB;           // bytes of one 128-row sub-tile
  static constexpr int TILE = 128 * D;           // bytes of 128 keys, or of a term of 128 query rows
};

// Bytes of a tile's parameters: (c, c, -lse, -lse) of two rows at a time.
constexpr int kRowBytes = 128 * 8;

// ---------------------------------------------------------------- query_kernel

// The rows of every tile as two e4m3 terms in the products' layout, c of each; -lse of the rows that there are not is
// -infinity, which makes their weights zero.  A CTA takes 16 rows of a tile, 8 threads each.
template <int D>
__global__ void __launch_bounds__(128) query_kernel(const BlockWeightsParams p) {
  using S = Shape<D>;
  griddep_wait();
  griddep_launch_dependents();
  const int G = p.Hq / p.Hkv, lane = threadIdx.x & 31, g = blockIdx.y;
  const int tile = blockIdx.x / 8, row0 = (blockIdx.x & 7) * 16;
  if (blockIdx.x == 0 && g == 0)
    for (int i = threadIdx.x; i < 2 * p.slots; i += 128) p.done[i] = 0;
  // the first sequence that has this tile
  WeightsSeq s = {0, 0, 0, false};
  int b = -1;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    if (b0 + lane < p.B) s = weights_seq(p, b0 + lane, false);
    else s.rows = 0;
    const long long i = tile - (static_cast<long long>(s.r0) * G / 128 + b0 + lane);
    const unsigned has = __ballot_sync(0xffffffffu, i >= 0 && i * 128 < static_cast<long long>(s.rows) * G);
    if (has != 0) {
      const int j = __ffs(has) - 1;
      b = b0 + j;
      s.r0 = __shfl_sync(0xffffffffu, s.r0, j);
      s.rows = __shfl_sync(0xffffffffu, s.rows, j);
      break;
    }
    if (__any_sync(0xffffffffu, s.rows > 0 && i < 0)) break;  // (those behind it that are not left out begin behind it)
  }
  if (b < 0) return;
  const long long R = static_cast<long long>(s.rows) * G;
  const long long i = tile - (static_cast<long long>(s.r0) * G / 128 + b);
  const int row = row0 + (threadIdx.x >> 3);
  const long long r = i * 128 + row;
  constexpr int NCH = (D / 16 + 7) / 8;  // 16-element chunks of a row per thread
  uint32_t in[NCH][8];
  uint32_t amax = 0;
#pragma unroll
  for (int cc = 0; cc < NCH; ++cc) {
    const int ch = (threadIdx.x & 7) + 8 * cc;
#pragma unroll
    for (int j = 0; j < 8; ++j) in[cc][j] = 0u;
    if (r < R && ch < D / 16) {
      const long long token = r / G;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + ((s.r0 + token) * p.Hq + g * G + (r - token * G)) * D) + 2 * ch;
      const uint4 x = src[0], y = src[1];
      in[cc][0] = x.x; in[cc][1] = x.y; in[cc][2] = x.z; in[cc][3] = x.w;
      in[cc][4] = y.x; in[cc][5] = y.y; in[cc][6] = y.z; in[cc][7] = y.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, max((in[cc][j] << 16) & 0x7FFF0000u, in[cc][j] & 0x7FFF0000u));
  }
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const int e = query_exponent(amax);  // q = q' 2^e
  const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const size_t at = tile_index(p, s.r0, b, g, static_cast<int>(i));
  if ((threadIdx.x & 7) == 0) {
    // a row with a NaN or an infinity makes its scores NaN
    float* out = p.rows + at * 256 + (row >> 1) * 4 + (row & 1);
    out[0] = r >= R ? 0.f : amax < 0x7F800000u ? p.sm_scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __uint_as_float(0x7FC00000u);
    if (r >= R) out[2] = -INFINITY;
  }
  uint8_t* dst = p.q_tiles + at * 2 * S::TILE;
#pragma unroll
  for (int cc = 0; cc < NCH; ++cc) {
    const int c = (threadIdx.x & 7) + 8 * cc;
    if (c >= D / 16) continue;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x0 = bf16x2_to_f2(in[cc][2 * j]), x1 = bf16x2_to_f2(in[cc][2 * j + 1]);
      split4_query(make_float2(x0.x * down, x0.y * down), make_float2(x1.x * down, x1.y * down), hi[j], lo[j]);
    }
    const int byte = c * 16;
    uint8_t* x = dst + (byte / S::RB) * S::SUB + swz(static_cast<uint32_t>(row * S::RB + byte % S::RB), S::RB);
    *reinterpret_cast<uint4*>(x) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(x + S::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ---------------------------------------------------------------- the two passes over many rows

// The unit's own tile stays (pass 0: 128 rows, both terms; pass 1: 256 keys, two products of 128), the others stream past it.  One CTA per
// SM.  Sixteen warps read the scores: in pass 0 a thread one row's for 64 keys, in pass 1 two keys' for 64 rows (whose c and lse it reads
// from shared memory once for both: one key per thread was bound by that, 2,000 cycles per 256 keys and 128 rows).  Eight of them take
// every other step, so that a piece's end, a chain of barriers, is passed by eight while the others compute (128 rows a
// unit, head_dim 128: 53.1 us a call with turns in pass 0 alone, 51.3 with both, then); in pass 1 at head_dim 256, whose products set the pace and wait for the scores' two buffers,
// all sixteen take every step, 32 rows a thread (a prompt of 4,001 tokens, 8/1 heads: 91 us against 97 then).  A wait that need not wait takes 100 to 200 cycles, a step's products 540 (head_dim
// 128), so the readers wait as seldom as they can, and two warps issue the products of the steps in turn.
template <int D, Kind K>
struct PassCfg : Shape<D> {
  using S = Shape<D>;
  static constexpr int KT = K == kRows ? 128 : 256;             // keys of a unit or step
  static constexpr int NT = KT / 128;                           // products per step
  static constexpr int QT = 2 * S::TILE;                        // both terms of a row tile
  static constexpr int STAY = K == kRows ? QT : 2 * S::TILE;
  static constexpr int STREAM = K == kRows ? S::TILE : QT + kRowBytes;
  static constexpr int NY = K == kRows ? 2 : D == 256 ? 1 : 3;  // buffers of the one, stages of the other
  static constexpr int NS = K == kRows ? (D == 256 ? 2 : 8) : (D == 256 ? 2 : 3);
  static constexpr int SBUF = 4 / NT;                           // buffers of a step's scores, 128 NT columns each
  static constexpr int READERS = 16, THREADS = 32 * (READERS + 3);
  static constexpr bool TURNS = K == kRows || D <= 128;         // eight readers every other step
  static constexpr int COLS = TURNS ? 64 : 32;                  // columns of a reader
  // K scales in slots: of steps 4 b .. 4 b + 3 (pass 0; the copies run at most NS + SBUF steps ahead), or of piece r (pass 1: NY ahead of
  // the products, which are SBUF steps ahead of the readers)
  static constexpr int SCN = 8, SCB = K == kRows ? 4 : 1;
  static constexpr int SCF = K == kRows ? 32 : 16;
  static constexpr int OFF_STAY = 0;
  static constexpr int OFF_STREAM = OFF_STAY + NY * STAY;
  static constexpr int OFF_SC = OFF_STREAM + NS * STREAM;
  static constexpr int JOIN = 4 * 128 * 8;                      // the column parts' results [4][128] float2, [4][256] float, twice
  static constexpr int OFF_JOIN = OFF_SC + SCN * SCF * 4;
  static constexpr int OFF_BAR = OFF_JOIN + 2 * JOIN;
  static constexpr int NBAR = 2 * NY + 2 * SBUF + 2 * NS + SCN + 6;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 64;
  static constexpr uint32_t IDESC = idesc_e4m3_f32(128, 128, 0, 0);
  static_assert(SCN * SCB > (K == kRows ? NS + SBUF + SCB : NY + SBUF + 1) && OFF_BAR % 8 == 0, "a slot is rewritten only after its readers are done");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Warps 0 .. 15 read the scores, 16 copies, 17 and 18 issue the products.
template <int D, Kind K>
__global__ void __launch_bounds__((PassCfg<D, K>::THREADS), 1)
    pass_kernel(const __grid_constant__ BlockWeightsParams p, const __grid_constant__ CUtensorMap tmk) {
  using C = PassCfg<D, K>;
  using Place = Walk<K, C::KT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sStay = smem + C::OFF_STAY;
  uint8_t* sStream = smem + C::OFF_STREAM;
  float* sSc = reinterpret_cast<float*>(smem + C::OFF_SC);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* y_full = bars;              // [NY] the tile of piece r in buffer r % NY
  uint64_t* y_empty = y_full + C::NY;
  uint64_t* s_full = y_empty + C::NY;   // [SBUF] the scores of step u in buffer u % SBUF
  uint64_t* s_free = s_full + C::SBUF;
  uint64_t* x_full = s_free + C::SBUF;  // [NS] the streamed tile of step u in stage u % NS
  uint64_t* x_empty = x_full + C::NS;
  uint64_t* sc_full = x_empty + C::NS;  // [SCN]
  uint64_t* mma_done = sc_full + C::SCN;  // [2]
  uint64_t* j_full = mma_done + 2;      // [2] the column parts' results of piece r in buffer r % 2 ...
  uint64_t* j_free = j_full + 2;        // [2] ... and taken
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* last_s = abort_s + 1;
  volatile int* pend_s = abort_s + 2;  // [2] {pieces, first CTA, b, g, t} of the range's first and last unit, if they have several

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NY; ++i) {
      mbar_init(&y_full[i], 1);
      mbar_init(&y_empty[i], 2);  // (both issuing warps)
    }
    for (int i = 0; i < C::SBUF; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], C::TURNS ? C::READERS / 2 : C::READERS);
    }
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_empty[i], K == kKeys ? 1 + (C::TURNS ? C::READERS / 2 : C::READERS) : 1);  // (the rows' parameters are read by the readers)
    }
    for (int i = 0; i < C::SCN; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&mma_done[i], 1);
      mbar_init(&j_full[i], C::READERS);
      mbar_init(&j_free[i], K == kRows ? 4 : 8);
    }
    *abort_s = 0;
    pend_s[0] = pend_s[5] = 0;
    fence_mbar_init();
  }
  // The kernel before this one lets it start when itself has waited for what came before, so that only it holds tensor memory, all of
  // which it has.  Everything else is read behind the wait for it, the sequences and the table too, which are older: only what is behind
  // a kernel's own wait is sure to be visible to it.
  if (warp == C::READERS + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  __shared__ Division<K, C::KT> division;
  if (warp == 0) {
    Division<K, C::KT> d;
    d.first = first_piece<K, C::KT>(p, k, d.W, d.N, K == kRows && k == 0);
    if (lane == 0) division = d;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int32_t* done = p.done + (K == kRows ? 0 : p.slots);
  Place at = division.first;
  int u = 0;  // steps so far
  KeyFeed<K, C::KT> feed;
  if (warp == C::READERS && at.n > 0) feed.begin(at, p);
  griddep_launch_dependents();

  if (warp < C::READERS) {
    // ============================================================ the scores' readers
    // tensor memory lane i, columns c_part .. + COLS - 1; taking turns, part >> 1 the steps' parity
    const int part = warp >> 2, i = (warp & 3) * 32 + lane;
    const int c_part = C::TURNS ? 64 * (part & 1) : 32 * part;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c_part;
    bool ok = true;
    while (ok && at.n > 0) {
      if (K == kKeys && C::TURNS && at.n == 1 && (u & 1) != part >> 1) {  // the other eight warps' alone
        ++u;
        at.next(p);
        continue;
      }
      // pass 0: the row's sum l of 2^(x - m) (of this thread's columns).  m need not be the maximum, only near enough that no sum
      // overflows: it is the largest score of the first columns, and moves when a sum of 32 reaches 2^60.
      float m = -kHuge, l = 0.f;
      float2 acc[C::NT];                      // pass 1: the keys' sums
      float mine[C::NT];                      // c of the row; ks of the keys
      int limit[C::NT];                       // keys that the row sees; the first row that sees the key
      if constexpr (K == kRows) {
        const int r = 128 * at.t + i;
        const bool is_row = r < at.rows * at.G;
        limit[0] = is_row ? at.old() + r / at.G + 1 : 0;
        mine[0] = is_row ? p.rows[tile_index(p, at.r0, at.b, at.g, at.t) * 256 + (i >> 1) * 4 + (i & 1)] : 0.f;
      } else {
        if (!wait_warp(&sc_full[at.piece % C::SCN], (at.piece / C::SCN) & 1)) ok = false;
#pragma unroll
        for (int h = 0; h < C::NT; ++h) {
          mine[h] = sSc[(at.piece % C::SCN) * C::SCF + 8 * h + (i >> 4)];
          limit[h] = max(C::KT * at.t + 128 * h + i - at.old(), 0) * at.G;
          acc[h] = make_float2(0.f, 0.f);
        }
      }
      const int end = u + at.n;
      if constexpr (K == kRows) {
        int c0 = 128 * (at.s + ((u ^ (part >> 1)) & 1)) + 64 * (part & 1);  // this thread's first key in its first step
        for (int v0 = u + ((u ^ (part >> 1)) & 1); ok && v0 < end; v0 += 2, c0 += 256) {
          const int sb = v0 % C::SBUF;
          if ((v0 & 6) == 6 && abort_warp(abort_s)) { ok = false; break; }
          if (!wait_warp(&sc_full[(v0 / C::SCB) % C::SCN], (v0 / (C::SCB * C::SCN)) & 1) || !wait_warp(&s_full[sb], (v0 / C::SBUF) & 1)) { ok = false; break; }
          tc_fence_after();
          const bool any_partly = __any_sync(0xffffffffu, limit[0] < c0 + 64);
          const float* ks = sSc + ((v0 / C::SCB) % C::SCN) * C::SCF + 8 * (v0 % C::SCB) + 4 * (part & 1);
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            float v[32];
            tmem_ld32(lane_base + 128 * sb + c, v);
            const float2 ks2 = *reinterpret_cast<const float2*>(ks + c / 16);
            tmem_ld_wait();
            if (c == 32) {
              tc_fence_before();
              mbar_arrive_warp(&s_free[sb]);
            }
            if (any_partly) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (c0 + c + j >= limit[0]) v[j] = -INFINITY;
            }
            // (plus 2^-126, so that a hidden score of -inf stays one where the product is zero)
            constexpr float kLeast = 1.17549435e-38f;
            const float a = fmaf(mine[0], ks2.x, kLeast), b2 = fmaf(mine[0], ks2.y, kLeast);
            // the sum against m; a sum of 2^60 and above, or NaN, moves its row's m to the maximum and is made again (the rows of
            // which it is not true stay as they are)
#pragma unroll 1
            for (bool again = false;; again = true) {
              const float2 a2 = make_float2(a, a), bb = make_float2(b2, b2), t2 = make_float2(-m, -m);
              float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 x = __ffma2_rn(make_float2(v[j], v[j + 1]), a2, t2), y = __ffma2_rn(make_float2(v[16 + j], v[17 + j]), bb, t2);
                s0 = __fadd2_rn(s0, make_float2(ex2(x.x), ex2(x.y)));
                s1 = __fadd2_rn(s1, make_float2(ex2(y.x), ex2(y.y)));
              }
              s0 = __fadd2_rn(s0, s1);
              const float sum = s0.x + s0.y;
              const bool over = !again && !(sum < 1.152921504606847e18f);
              if (!__any_sync(0xffffffffu, over)) {
                l += sum;
                break;
              }
              const float top = over ? fmaxf(m, fmaxf(max_tree<16>(v) * a, max_tree<16>(v + 16) * b2)) : m;
              l *= ex2(m - top);
              m = top;
            }
          }
        }
      } else {
        const int off = C::TURNS ? (u ^ (part >> 1)) & 1 : 0;
        int c0 = 128 * (at.first() + at.s + off) + c_part;  // this thread's first row
        for (int v0 = u + off; ok && v0 < end; v0 += C::TURNS ? 2 : 1, c0 += C::TURNS ? 256 : 128) {
          const int sb = v0 % C::SBUF, st = v0 % C::NS;
          if ((v0 & 6) == 6 && abort_warp(abort_s)) { ok = false; break; }
          const bool any_partly = __any_sync(0xffffffffu, limit[0] > c0 || limit[C::NT - 1] > c0);
          if (!wait_warp(&s_full[sb], (v0 / C::SBUF) & 1)) { ok = false; break; }
          tc_fence_after();
          const float4* rp = reinterpret_cast<const float4*>(sStream + st * C::STREAM + C::QT) + c_part / 2;
#pragma unroll 1
          for (int c = 0; c < C::COLS; c += 16) {
            float v[C::NT][16];
#pragma unroll
            for (int h = 0; h < C::NT; ++h) tmem_ld16(lane_base + 128 * (C::NT * sb + h) + c, v[h]);
            tmem_ld_wait();
            if (c == C::COLS - 16) {
              tc_fence_before();
              mbar_arrive_warp(&s_free[sb]);
            }
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float4 r = rp[(c + j) / 2];
#pragma unroll
              for (int h = 0; h < C::NT; ++h) {
                const float2 x = __ffma2_rn(__fmul2_rn(make_float2(v[h][j], v[h][j + 1]), make_float2(mine[h], mine[h])), make_float2(r.x, r.y), make_float2(r.z, r.w));
                v[h][j] = ex2(x.x);
                v[h][j + 1] = ex2(x.y);
              }
            }
            if (any_partly) {  // (a hidden score has no weight, whatever its row's sum is)
#pragma unroll
              for (int h = 0; h < C::NT; ++h)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (c0 + c + j < limit[h]) v[h][j] = 0.f;
            }
#pragma unroll
            for (int h = 0; h < C::NT; ++h)
#pragma unroll
              for (int j = 0; j < 16; j += 2) acc[h] = __fadd2_rn(acc[h], make_float2(v[h][j], v[h][j + 1]));
          }
          mbar_arrive_warp(&x_empty[st]);
        }
      }
      u = end;
      if (!ok) break;
      // ---- the column parts of the piece meet in shared memory (pass 1, a piece of one step: those of eight warps, which arrive twice)
      const bool alone = K == kKeys && C::TURNS && at.n == 1;
      const int jb = at.piece & 1;
      float2* row_join = reinterpret_cast<float2*>(smem + C::OFF_JOIN + jb * C::JOIN);
      float* key_join = reinterpret_cast<float*>(row_join);
      if (at.piece > 1 && !wait_warp(&j_free[jb], ((at.piece >> 1) - 1) & 1)) { ok = false; break; }
      if constexpr (K == kRows) {
        row_join[part * 128 + i] = make_float2(m, l);
      } else {
#pragma unroll
        for (int h = 0; h < C::NT; ++h) key_join[part * 256 + 128 * h + i] = acc[h].x + acc[h].y;
      }
      mbar_arrive_warp(&j_full[jb]);
      if (alone) mbar_arrive_warp(&j_full[jb]);
      if (K == kRows ? warp < 4 : ((C::TURNS ? end - 1 : 0) & 1) == part >> 1) {
        if (!wait_warp(&j_full[jb], (at.piece >> 1) & 1)) { ok = false; break; }
        int k0 = k, ns = 1;
        if (!at.whole()) {
          k0 = cta_of(at.unit0, division.W, division.N);
          ns = cta_of(at.unit0 + at.count - 1, division.W, division.N) - k0 + 1;
        }
        const long long place = piece_place(k, k0);
        if constexpr (K == kRows) {
          float top = -kHuge, sum = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 y = row_join[x * 128 + i];
            const float mx = fmaxf(top, y.x);
            sum = sum * ex2(top - mx) + y.y * ex2(y.x - mx);
            top = mx;
          }
          if (ns > 1) p.pieces[place * 128 + i] = make_float2(top, sum);
          else if (limit[0] > 0) p.rows[tile_index(p, at.r0, at.b, at.g, at.t) * 256 + (i >> 1) * 4 + (i & 1) + 2] = -(top + lg2(sum));
        } else {
          const int j = threadIdx.x & 255, key = C::KT * at.t + j;
          const float* mine_join = key_join + 512 * (part >> 1) + j;
          float sum = mine_join[0] + mine_join[256];
          if (!alone) sum = part >> 1 ? (key_join[j] + key_join[256 + j]) + sum : sum + (key_join[512 + j] + key_join[768 + j]);
          if (ns > 1) {
            p.sums[place * C::KT + j] = sum;
          } else if (key < at.T) {
            float* w = p.weights + (static_cast<size_t>(at.b) * p.Hkv + at.g) * p.weights_len + key;
            *w = key < at.old() && p.decay != 0.f ? fmaf(p.decay, *w, sum) : sum;
          }
        }
        mbar_arrive_warp(&j_free[jb]);
        if (ns > 1 && threadIdx.x == (K == kRows ? 0 : 256 * (part >> 1))) {
          volatile int* pend = pend_s + (k == k0 ? 5 : 0);
          pend[0] = ns;
          pend[1] = k0;
          pend[2] = at.b;
          pend[3] = at.g;
          pend[4] = at.t;
        }
      }
      at.next(p);
    }
    tmem_ld_wait();  // no load left in flight on an early exit
    if (!ok) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
  } else if (warp == C::READERS) {
    // ============================================================ copies
    using Feed = KeyFeed<K, C::KT>;
    int stay_pieces = 0;            // pieces whose tile was requested
    size_t held[C::NS];             // pass 1: the row tile that a stage holds
#pragma unroll
    for (int s = 0; s < C::NS; ++s) held[s] = ~static_cast<size_t>(0);
    // The keys of tile `tile` (a block per lane; blocks behind the sequence are left as they are: their keys are hidden, or their sums
    // not stored) and their scales.
    auto copy_keys = [&](uint8_t* dst, uint64_t* full, int tile, int x) {  // x: the step (pass 0) or piece
      int id;
      float ks;
      feed.take(p, id, ks);
      const int nblk = Feed::blocks_of(at, tile);
      if (lane == 0) mbar_arrive_expect_tx(full, nblk * 16 * D);
      __syncwarp();
      if (lane < nblk) {
#pragma unroll
        for (int s = 0; s < C::NSUB; ++s)
          tma_load_4d(dst + (lane >> 3) * C::TILE + s * C::SUB + (lane & 7) * 16 * C::RB, &tmk, s * C::RB, 0, at.g, id, full);
      }
      if (x % C::SCB == 0) {
        const int slot = (x / C::SCB) % C::SCN;
        if (K == kRows) sSc[slot * C::SCF + lane] = feed.ks;  // (a batch: the scales of four steps)
        else if (lane < Feed::TB) sSc[slot * C::SCF + lane] = ks;
        mbar_arrive_warp(&sc_full[slot]);
      }
    };
    bool ok = true;
    while (ok && at.n > 0) {
      const int yb = at.piece % C::NY;
      if (at.piece >= C::NY && !wait_warp(&y_empty[yb], (at.piece / C::NY - 1) & 1, p.stage_wait_ns)) { ok = false; break; }
      size_t tile = tile_index(p, at.r0, at.b, at.g, K == kRows ? at.t : at.first() + at.s);
      if constexpr (K == kRows) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&y_full[yb], C::QT);
          bulk_g2s(sStay + yb * C::STAY, p.q_tiles + tile * C::QT, C::QT, &y_full[yb]);
        }
        __syncwarp();
      } else {
        copy_keys(sStay + yb * C::STAY, &y_full[yb], at.t, at.piece);
      }
      stay_pieces = at.piece + 1;
      const int end = u + at.n;
      for (int x = 0; u < end; ++u, ++x, tile += p.Hkv) {
        if (abort_warp(abort_s)) { ok = false; break; }
        const int st = u % C::NS;
        if (u >= C::NS && !wait_warp(&x_empty[st], (u / C::NS - 1) & 1, p.stage_wait_ns)) { ok = false; break; }
        uint8_t* dst = sStream + st * C::STREAM;
        if constexpr (K == kRows) {
          copy_keys(dst, &x_full[st], at.s + x, u);
        } else {
          bool same = false;
#pragma unroll
          for (int s = 0; s < C::NS; ++s) {
            if (s != st) continue;
            same = held[s] == tile;
            held[s] = tile;
          }
          if (lane == 0) {
            if (same) {
              mbar_arrive(&x_full[st]);
            } else {
              mbar_arrive_expect_tx(&x_full[st], C::QT + kRowBytes);
              bulk_g2s(dst, p.q_tiles + tile * C::QT, C::QT, &x_full[st]);
              bulk_g2s(dst + C::QT, p.rows + tile * 256, kRowBytes, &x_full[st]);
            }
          }
          __syncwarp();
        }
      }
      if (ok) at.next(p);
    }
    if (!ok) {
      if (lane == 0 && *abort_s == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
    // let every copy land before the CTA can exit
    if (lane == 0) {
      for (int s = 0; s < C::NS; ++s)
        if (u > s) wait_ns(&x_full[s], ((u - 1 - s) / C::NS) & 1);
      for (int s = 0; s < C::NY; ++s)
        if (stay_pieces > s) wait_ns(&y_full[s], ((stay_pieces - 1 - s) / C::NY) & 1);
    }
    __syncwarp();
  } else {
    // ============================================================ products
    // Warp w the steps of its parity.  A piece's tile is free when both warps' products with it are done.
    const int w = warp - C::READERS - 1;
    const uint64_t dY = smem_desc(smem_u32(sStay), 16, 8 * C::RB, C::SWZ), dX = smem_desc(smem_u32(sStream), 16, 8 * C::RB, C::SWZ);
    bool ok = true;
    while (ok && at.n > 0) {
      const int yb = at.piece % C::NY, end = u + at.n;
      ok = wait_warp(&y_full[yb], (at.piece / C::NY) & 1);
      for (int v0 = u + ((u ^ w) & 1); ok && v0 < end; v0 += 2) {
        if ((v0 & 6) == 6 && abort_warp(abort_s)) { ok = false; break; }
        const int st = v0 % C::NS, sb = v0 % C::SBUF;
        ok = wait_warp(&x_full[st], (v0 / C::NS) & 1);
        if (ok && v0 >= C::SBUF) ok = wait_warp(&s_free[sb], (v0 / C::SBUF - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < C::NT; ++h)
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk) {
                const int byte = kk * 32;
                const uint32_t off = (byte / C::RB) * C::SUB + (byte % C::RB);
                umma_f8(tmem + 128 * (C::NT * sb + h), desc_add(dY, yb * C::STAY + (K == kRows ? term : h) * C::TILE + off),
                        desc_add(dX, st * C::STREAM + (K == kKeys ? term : 0) * C::TILE + off), C::IDESC, (term > 0 || kk > 0) ? 1u : 0u);
              }
          umma_commit(&s_full[sb]);
          umma_commit(&x_empty[st]);
        }
        __syncwarp();
      }
      u = end;
      if (!ok) break;
      if (elect_one()) umma_commit(&y_empty[yb]);
      __syncwarp();
      at.next(p);
    }
    if (!ok) {
      if (lane == 0 && *abort_s == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
    if (elect_one()) umma_commit(&mma_done[w]);  // every product issued here completes before the tensor memory is released
    __syncwarp();
    wait_warp(&mma_done[w], 0);
  }
  __syncthreads();
  if (warp == C::READERS + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // the CTA that brings a unit's last piece joins them
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const int ns = pend_s[5 * j], k0 = pend_s[5 * j + 1], b = pend_s[5 * j + 2], g = pend_s[5 * j + 3], t = pend_s[5 * j + 4];
    if (ns == 0) continue;
    if (threadIdx.x == 0) *last_s = count_piece(&done[k0]) == ns - 1;
    __syncthreads();
    const int i = threadIdx.x;
    if (*last_s && i < (K == kRows ? 128 : C::KT)) {
      const WeightsSeq s = weights_seq(p, b, false);
      if constexpr (K == kRows) {
        float m = -kHuge, l = 0.f;
#pragma unroll 4
        for (int x = 0; x < ns; ++x) {
          const float2 y = __ldcg(p.pieces + piece_place(k0 + x, k0) * 128 + i);
          const float top = fmaxf(m, y.x);
          l = l * ex2(m - top) + y.y * ex2(y.x - top);
          m = top;
        }
        if (128 * t + i < s.rows * (p.Hq / p.Hkv)) p.rows[tile_index(p, s.r0, b, g, t) * 256 + (i >> 1) * 4 + (i & 1) + 2] = -(m + lg2(l));
      } else {
        float sum = 0.f;
#pragma unroll 4
        for (int x = 0; x < ns; ++x) sum += __ldcg(p.sums + piece_place(k0 + x, k0) * C::KT + i);
        const int key = C::KT * t + i;
        if (key < s.T) {
          float* w = p.weights + (static_cast<size_t>(b) * p.Hkv + g) * p.weights_len + key;
          *w = key < s.T - s.rows && p.decay != 0.f ? fmaf(p.decay, *w, sum) : sum;
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- few rows

// RN: rows (4, 8 or 16) that a key's scores are kept for.
template <int D, int RN>
struct ScoreCfg : Shape<D> {
  using S = Shape<D>;
  static constexpr int LO = RN < 8 ? 8 : RN;                    // first row (column) of the query's second term
  static constexpr int NP = 2 * LO;                             // the MMA's N
  static constexpr int NHALF = D == 64 ? 2 : 1;                 // products of 128 keys per tile
  static constexpr int BN = 128 * NHALF, TPB = BN / 16;         // keys and blocks of a tile
  static constexpr int KSUB = BN * S::RB, KTILE = BN * D;
  static constexpr int NS = D <= 128 ? 4 : 3;
  static constexpr int CTAS = D <= 128 ? 3 : 2;
  static constexpr int SCN = 8;
  static constexpr int QSUB = NP * S::RB;
  static constexpr int TM_COLS = 2 * NHALF * NP <= 32 ? 32 : 2 * NHALF * NP <= 64 ? 64 : 128;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = (OFF_Q + S::NSUB * QSUB + 1023) / 1024 * 1024;
  static constexpr int OFF_SC = OFF_K + NS * KTILE;
  static constexpr int OFF_C = OFF_SC + SCN * TPB * 4;          // c of the rows [16]
  static constexpr int OFF_RED = OFF_C + 16 * 4;                // [2][4 warps][RN] float2
  static constexpr int OFF_BAR = OFF_RED + 2 * 4 * RN * 8;
  static constexpr int NBAR = 7 + 2 * NS + SCN;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr uint32_t IDESC = idesc_e4m3_f32(128, NP, 0, 0);
  static_assert(SCN > NS + 2 && OFF_BAR % 8 == 0, "slots");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory of the resident CTAs");
};

constexpr int kScoreThreads = 192;  // warps 0-3 read the scores, 4 copies, 5 issues the products

FKV_DEV void tmem_ld4(uint32_t addr, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr));
}

// The scores of the rows of every (sequence, KV head) for its keys, [key][RN] in base 2 (-infinity where the row does not
// see the key), and each piece's maxima and sums.  The products are taken transposed, S^T = K8 (hi | lo)^T: a thread owns a key, and
// keeps its own running maximum and sum of every row, which meet at a piece's end.
template <int D, int RN>
__global__ void __launch_bounds__(kScoreThreads, (ScoreCfg<D, RN>::CTAS))
    score_kernel(const __grid_constant__ BlockWeightsParams p, const __grid_constant__ CUtensorMap tmk) {
  using C = ScoreCfg<D, RN>;
  using Place = Walk<kScores, C::BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  float* sSc = reinterpret_cast<float*>(smem + C::OFF_SC);
  float* sC = reinterpret_cast<float*>(smem + C::OFF_C);
  float2* sRed = reinterpret_cast<float2*>(smem + C::OFF_RED);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars + 0;    // the query of piece r
  uint64_t* s_full = bars + 1;    // [2]
  uint64_t* s_free = bars + 3;    // [2]
  uint64_t* mma_done = bars + 5;
  uint64_t* r_full = bars + 6;    // the warps' results of piece r
  uint64_t* k_full = bars + 7;
  uint64_t* k_empty = k_full + C::NS;
  uint64_t* sc_full = k_empty + C::NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.x;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 4);
    mbar_init(r_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::SCN; ++i) mbar_init(&sc_full[i], 1);
    *abort_s = 0;
    fence_mbar_init();
  }
  griddep_wait();  // (the tensor memory is taken after it, as in pass_kernel)
  if (warp == 5) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  __shared__ Division<kScores, C::BN> division;
  if (warp == 0) {
    Division<kScores, C::BN> d;
    d.first = first_piece<kScores, C::BN>(p, k, d.W, d.N, k == 0);
    if (lane == 0) division = d;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  Place at = division.first;
  const int G = at.G;
  int u = 0;  // steps so far

  if (warp < 4) {
    // ============================================================ the scores' readers
    const int i = threadIdx.x;  // key i (and 128 + i) of a tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float m[RN], l[RN];
    // the piece's unit: its first CTA and its pieces, which that CTA writes down
    auto put_unit = [&]() {
      int2 unit = make_int2(k, 1);
      if (!at.whole()) {
        unit.x = cta_of(at.unit0, division.W, division.N);
        unit.y = cta_of(at.unit0 + at.count - 1, division.W, division.N) - unit.x + 1;
      }
      if (lane == 0 && k == unit.x) p.units[at.b * p.Hkv + at.g] = unit;
      return unit;
    };
    bool ok = true;
    while (ok && at.n > 0) {
      // ---- the piece's query: row r scaled to (224, 448], as two terms, 8 threads per row (the products with the
      // last piece's query are done: their scores were read)
      const int row = i >> 3, R = at.rows * G;
      constexpr int NCH = (D / 16 + 7) / 8;
      uint32_t in[NCH][8];
      uint32_t amax = 0;
#pragma unroll
      for (int cc = 0; cc < NCH; ++cc) {
        const int ch = (i & 7) + 8 * cc;
#pragma unroll
        for (int j = 0; j < 8; ++j) in[cc][j] = 0u;
        if (row < R && ch < D / 16) {
          const int token = row / G;
          const uint4* src = reinterpret_cast<const uint4*>(p.q + ((static_cast<size_t>(at.r0) + token) * p.Hq + at.g * G + (row - token * G)) * D) + 2 * ch;
          const uint4 x = src[0], y = src[1];
          in[cc][0] = x.x; in[cc][1] = x.y; in[cc][2] = x.z; in[cc][3] = x.w;
          in[cc][4] = y.x; in[cc][5] = y.y; in[cc][6] = y.z; in[cc][7] = y.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, max((in[cc][j] << 16) & 0x7FFF0000u, in[cc][j] & 0x7FFF0000u));
      }
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      const int e = query_exponent(amax);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if ((i & 7) == 0)
        sC[row] = amax < 0x7F800000u ? p.sm_scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int cc = 0; cc < NCH; ++cc) {
        const int c = (i & 7) + 8 * cc;
        if (c >= D / 16 || row >= C::LO) continue;
        uint32_t wh[4], wl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x0 = bf16x2_to_f2(in[cc][2 * j]), x1 = bf16x2_to_f2(in[cc][2 * j + 1]);
          split4_query(make_float2(x0.x * down, x0.y * down), make_float2(x1.x * down, x1.y * down), wh[j], wl[j]);
        }
        const int byte = c * 16;
        uint8_t* sub = sQ + (byte / C::RB) * C::QSUB;
        *reinterpret_cast<uint4*>(sub + swz(static_cast<uint32_t>(row * C::RB + byte % C::RB), C::RB)) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
        *reinterpret_cast<uint4*>(sub + swz(static_cast<uint32_t>((C::LO + row) * C::RB + byte % C::RB), C::RB)) =
            make_uint4(wl[0], wl[1], wl[2], wl[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(q_full);
      if (!wait_warp(q_full, at.piece & 1)) { ok = false; break; }  // every warp's rows and c are there
#pragma unroll
      for (int r = 0; r < RN; ++r) {
        m[r] = -kHuge;
        l[r] = 0.f;
      }
      const int end = u + at.n;
      for (int x0 = 0; ok && u < end; ++u, ++x0) {
        if ((u & 7) == 7 && abort_warp(abort_s)) { ok = false; break; }
        const int sb = u & 1;
        if (!wait_warp(&sc_full[u % C::SCN], (u / C::SCN) & 1) || !wait_warp(&s_full[sb], (u >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int hh = 0; hh < C::NHALF; ++hh) {
          float v[2 * RN];
          const uint32_t col = lane_base + (sb * C::NHALF + hh) * C::NP;
          if constexpr (RN == 4) {
            tmem_ld4(col, v);
            tmem_ld4(col + C::LO, v + 4);
          } else if constexpr (RN == 8) {
            tmem_ld16(col, v);
          } else {
            tmem_ld32(col, v);
          }
          const float ks = sSc[(u % C::SCN) * C::TPB + 8 * hh + (i >> 4)];
          const int key = C::BN * (at.s + x0) + 128 * hh + i;
          tmem_ld_wait();
          if (hh + 1 == C::NHALF) {
            tc_fence_before();
            mbar_arrive_warp(&s_free[sb]);
          }
          // the first row that sees the key (none behind the sequence)
          const int from = key < at.T ? max(key - (at.T - at.rows), 0) * G : RN;
#pragma unroll
          for (int r = 0; r < RN; ++r) {
            float x = (v[r] + v[RN + r]) * (sC[r] * ks);
            if (r < from) x = -INFINITY;
            v[r] = x;
            // one exponential: of the smaller against the larger
            const float e = ex2(-fabsf(x - m[r]));
            l[r] = x > m[r] ? fmaf(l[r], e, 1.f) : l[r] + e;
            m[r] = fmaxf(m[r], x);
          }
          if (key < at.T) {
            float4* dst = reinterpret_cast<float4*>(p.scores + ((static_cast<size_t>(at.b) * p.Hkv + at.g) * p.max_blocks * 16 + key) * RN);
#pragma unroll
            for (int r = 0; r < RN; r += 4) dst[r / 4] = make_float4(v[r], v[r + 1], v[r + 2], v[r + 3]);
          }
        }
      }
      if (!ok) break;
      // ---- the warps' maxima and sums meet in shared memory; behind this barrier no warp reads the piece's query constants
      float2* red = sRed + (at.piece & 1) * 4 * RN;
#pragma unroll
      for (int r = 0; r < RN; ++r) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          const float m2 = __shfl_xor_sync(0xffffffffu, m[r], off), l2 = __shfl_xor_sync(0xffffffffu, l[r], off), top = fmaxf(m[r], m2);
          l[r] = l[r] * ex2(m[r] - top) + l2 * ex2(m2 - top);
          m[r] = top;
        }
        if (lane == 0) red[warp * RN + r] = make_float2(m[r], l[r]);
      }
      mbar_arrive_warp(r_full);
      if (!wait_warp(r_full, at.piece & 1)) { ok = false; break; }
      if (warp == 0) {
        const int2 unit = put_unit();
        const int k0 = unit.x, ns = unit.y;
        if (lane < RN) {
          float M = -kHuge, L = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 y = red[w * RN + lane];
            const float top = fmaxf(M, y.x);
            L = L * ex2(M - top) + y.y * ex2(y.x - top);
            M = top;
          }
          // (a unit in one piece has a place of its own: a CTA may have many)
          p.pieces[(ns == 1 ? 2LL * p.slots + static_cast<long long>(at.b) * p.Hkv + at.g : piece_place(k, k0)) * 16 + lane] = make_float2(M, L);
        }
      }
      at.next(p);
    }
    tmem_ld_wait();
    if (!ok) {
      if (lane == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
      // what the gather finds its pieces by is there all the same (what they hold is then anything)
      if (warp == 0)
        for (; at.n > 0; at.next(p)) put_unit();
    }
  } else if (warp == 4) {
    // ============================================================ K copies and scales
    using Feed = KeyFeed<kScores, C::BN>;
    Feed feed;
    if (at.n > 0) feed.begin(at, p);
    bool ok = true;
    for (; ok && at.n > 0; at.next(p)) {
      const int end = u + at.n;
      for (int x = 0; u < end; ++u, ++x) {
        const int st = u % C::NS;
        if (abort_warp(abort_s) || (u >= C::NS && !wait_warp(&k_empty[st], (u / C::NS - 1) & 1, p.stage_wait_ns))) { ok = false; break; }
        int id;
        float ks;
        feed.take(p, id, ks);
        const int nblk = Feed::blocks_of(at, at.s + x);
        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], nblk * 16 * D);
        __syncwarp();
        if (lane < nblk) {
#pragma unroll
          for (int s = 0; s < C::NSUB; ++s) tma_load_4d(sK + st * C::KTILE + s * C::KSUB + lane * 16 * C::RB, &tmk, s * C::RB, 0, at.g, id, &k_full[st]);
        }
        if (lane < C::TPB) sSc[(u % C::SCN) * C::TPB + lane] = ks;
        mbar_arrive_warp(&sc_full[u % C::SCN]);
      }
    }
    if (!ok) {
      if (lane == 0 && *abort_s == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
    if (lane == 0)
      for (int s = 0; s < C::NS; ++s)
        if (u > s) wait_ns(&k_full[s], ((u - 1 - s) / C::NS) & 1);
    __syncwarp();
  } else {
    // ============================================================ products
    const uint64_t dK = smem_desc(smem_u32(sK), 16, 8 * C::RB, C::SWZ), dQ = smem_desc(smem_u32(sQ), 16, 8 * C::RB, C::SWZ);
    bool ok = true;
    for (; ok && at.n > 0; at.next(p)) {
      const int end = u + at.n;
      ok = wait_warp(q_full, at.piece & 1);
      for (; ok && u < end; ++u) {
        if ((u & 7) == 7 && abort_warp(abort_s)) { ok = false; break; }
        const int st = u % C::NS, sb = u & 1;
        ok = wait_warp(&k_full[st], (u / C::NS) & 1);
        if (ok && u >= 2) ok = wait_warp(&s_free[sb], ((u >> 1) - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int hh = 0; hh < C::NHALF; ++hh)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              const int byte = kk * 32;
              umma_f8(tmem + (sb * C::NHALF + hh) * C::NP,
                      desc_add(dK, st * C::KTILE + (byte / C::RB) * C::KSUB + hh * 128 * C::RB + byte % C::RB),
                      desc_add(dQ, (byte / C::RB) * C::QSUB + byte % C::RB), C::IDESC, kk > 0 ? 1u : 0u);
            }
          umma_commit(&s_full[sb]);
          umma_commit(&k_empty[st]);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (lane == 0 && *abort_s == 0) raise_fault(p.fault, FKV_FAULT_TIMEOUT);
      *abort_s = 1;
    }
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    wait_warp(mma_done, 0);
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

constexpr int kGatherThreads = 256, kGatherKeys = 4 * kGatherThreads;

// w_j from the scores: grid (kGatherKeys keys each, KV heads, sequences).  A thread's scores and weights are on their way while the rows'
// sums, a chain of round trips, are put together.
template <int RN>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const BlockWeightsParams p) {
  __shared__ float lse_s[16];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z, g = blockIdx.y, G = p.Hq / p.Hkv;
  const WeightsSeq s = weights_seq(p, b, false);
  if (s.rows == 0 || static_cast<long long>(blockIdx.x) * kGatherKeys >= s.T) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t unit = static_cast<size_t>(b) * p.Hkv + g;
  const int2 at = p.units[unit];
  constexpr int KEYS = kGatherKeys / kGatherThreads;
  const float4* scores = reinterpret_cast<const float4*>(p.scores + unit * p.max_blocks * 16 * RN);
  float* weights = p.weights + unit * p.weights_len;
  const long long key0 = static_cast<long long>(blockIdx.x) * kGatherKeys + threadIdx.x;
  float4 y[KEYS][RN / 4];
  float old[KEYS];
#pragma unroll
  for (int x = 0; x < KEYS; ++x) {
    const long long key = key0 + x * kGatherThreads;
#pragma unroll
    for (int r = 0; r < RN / 4; ++r) y[x][r] = key < s.T ? scores[key * (RN / 4) + r] : make_float4(0.f, 0.f, 0.f, 0.f);
    old[x] = key < s.T - s.rows && p.decay != 0.f ? weights[key] : 0.f;
  }
  for (int r = warp; r < RN; r += kGatherThreads / 32) {
    float m = -kHuge, l = 0.f;
    for (int x = lane; x < at.y; x += 32) {
      const float2 y = p.pieces[(at.y == 1 ? 2LL * p.slots + static_cast<long long>(unit) : piece_place(at.x + x, at.x)) * 16 + r];
      const float top = fmaxf(m, y.x);
      l = l * ex2(m - top) + y.y * ex2(y.x - top);
      m = top;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, off), l2 = __shfl_xor_sync(0xffffffffu, l, off), top = fmaxf(m, m2);
      l = l * ex2(m - top) + l2 * ex2(m2 - top);
      m = top;
    }
    if (lane == 0) lse_s[r] = r < s.rows * G ? m + lg2(l) : INFINITY;
  }
  __syncthreads();
  float lse[RN];
#pragma unroll
  for (int r = 0; r < RN; ++r) lse[r] = lse_s[r];
#pragma unroll
  for (int x = 0; x < KEYS; ++x) {
    const long long key = key0 + x * kGatherThreads;
    if (key >= s.T) break;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < RN / 4; ++r) {
      const float v[4] = {y[x][r].x, y[x][r].y, y[x][r].z, y[x][r].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += v[j] == -INFINITY ? 0.f : ex2(v[j] - lse[4 * r + j]);
    }
    weights[key] = key < s.T - s.rows && p.decay != 0.f ? fmaf(p.decay, old[x], sum) : sum;
  }
}

// ---------------------------------------------------------------- launches

constexpr int kFewRows = 16;

// Rows that a key's scores are kept for; 0: too many, pass by pass.
int rows_kept(int max_q_len, int G) {
  const long long R = static_cast<long long>(max_q_len) * G;
  return R <= 4 ? 4 : R <= 8 ? 8 : R <= kFewRows ? 16 : 0;
}

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The workspace's parts; returns its bytes.
size_t lay_out(BlockWeightsParams* p, uint8_t* base, int B, int total_q, int max_q_len, int Hq, int Hkv, int D, long long keys, int slots) {
  const int G = Hq / Hkv, RN = rows_kept(max_q_len, G);
  size_t at = 0;
  auto part = [&](size_t bytes) {
    uint8_t* x = base ? base + at : nullptr;
    at += up256(bytes);
    return x;
  };
  const size_t units = static_cast<size_t>(B) * Hkv;
  if (RN > 0) {
    uint8_t* u = part(units * sizeof(int2));
    uint8_t* pieces = part((2 * static_cast<size_t>(slots) + units) * 16 * sizeof(float2));
    uint8_t* scores = part(units * keys * RN * sizeof(float));
    if (p) {
      p->units = reinterpret_cast<int2*>(u);
      p->pieces = reinterpret_cast<float2*>(pieces);
      p->scores = reinterpret_cast<float*>(scores);
    }
  } else {
    const size_t tiles = (static_cast<size_t>(total_q) * G / 128 + B) * Hkv;
    uint8_t* done = part(2 * static_cast<size_t>(slots) * sizeof(int32_t));
    uint8_t* pieces = part(2 * static_cast<size_t>(slots) * 128 * sizeof(float2));
    uint8_t* sums = part(2 * static_cast<size_t>(slots) * 256 * sizeof(float));
    uint8_t* rows = part(tiles * kRowBytes);
    uint8_t* q = part(tiles * 256 * D);
    if (p) {
      p->done = reinterpret_cast<int32_t*>(done);
      p->pieces = reinterpret_cast<float2*>(pieces);
      p->sums = reinterpret_cast<float*>(sums);
      p->rows = reinterpret_cast<float*>(rows);
      p->q_tiles = q;
    }
  }
  return at;
}

template <typename Kernel>
cudaError_t launch_tc(Kernel kern, int grid, int threads, int smem, const BlockWeightsParams& p, const CUtensorMap& tmk, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(grid), dim3(threads), smem, s, p, tmk);
}

template <int D, int RN>
cudaError_t launch_few(const BlockWeightsParams& p, const CUtensorMap& tmk, int num_sms, cudaStream_t s) {
  using C = ScoreCfg<D, RN>;
  const cudaError_t e = launch_tc(score_kernel<D, RN>, C::CTAS * num_sms, kScoreThreads, C::SMEM, p, tmk, s);
  if (e != cudaSuccess) return e;
  const long long keys = std::min(p.max_blocks * 16LL, static_cast<long long>(p.weights_len));
  if (keys == 0) return cudaSuccess;  // (no weights: the sequences were reported)
  return launch_dependent(gather_kernel<RN>, dim3(static_cast<unsigned>((keys + kGatherKeys - 1) / kGatherKeys), p.Hkv, p.B), dim3(kGatherThreads),
                          0, s, p);
}

template <int D>
cudaError_t launch_d(const BlockWeightsParams& p, int num_sms, cudaStream_t s) {
  CUtensorMap tmk;
  if (!make_pool_map(&tmk, const_cast<uint8_t*>(p.k_cache), D, p.Hkv, p.num_blocks, Shape<D>::RB)) return cudaErrorInvalidValue;
  const int G = p.Hq / p.Hkv, RN = rows_kept(p.max_q_len, G);
  if (RN == 4) return launch_few<D, 4>(p, tmk, num_sms, s);
  if (RN == 8) return launch_few<D, 8>(p, tmk, num_sms, s);
  if (RN == 16) return launch_few<D, 16>(p, tmk, num_sms, s);
  const long long tiles = static_cast<long long>(p.total_q) * G / 128 + p.B;
  if (tiles * 8 > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = launch_dependent(query_kernel<D>, dim3(static_cast<unsigned>(tiles * 8), p.Hkv), dim3(128), 0, s, p);
  if (e != cudaSuccess) return e;
  e = launch_tc(pass_kernel<D, kRows>, num_sms, PassCfg<D, kRows>::THREADS, PassCfg<D, kRows>::SMEM, p, tmk, s);
  if (e != cudaSuccess) return e;
  return launch_tc(pass_kernel<D, kKeys>, num_sms, PassCfg<D, kKeys>::THREADS, PassCfg<D, kKeys>::SMEM, p, tmk, s);
}

// CTAs of a launch, at most.
int slots_of(int num_sms) { return 3 * num_sms; }

}  // namespace

size_t block_weights_workspace(int B, int total_q, int max_q_len, int Hq, int Hkv, int D, long long keys, int num_sms) {
  return lay_out(nullptr, nullptr, B, total_q, max_q_len, Hq, Hkv, D, keys, slots_of(num_sms));
}

cudaError_t launch_block_weights(BlockWeightsParams p, int D, void* workspace, int num_sms, cudaStream_t s) {
  p.slots = slots_of(num_sms);
  lay_out(&p, static_cast<uint8_t*>(workspace), p.B, p.total_q, p.max_q_len, p.Hq, p.Hkv, D, p.max_blocks * 16LL, p.slots);
  if (D == 64) return launch_d<64>(p, num_sms, s);
  if (D == 128) return launch_d<128>(p, num_sms, s);
  return launch_d<256>(p, num_sms, s);
}

}  // namespace fkv
