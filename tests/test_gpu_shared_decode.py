"""fp8_block_shared_decode_attn on the GPU against the float64 softmax of every sequence by itself.

Tolerance of an output element, derived as for the attention over block-scaled pools: with p_j the softmax weights,
P = sum_j p_j |v_j| and V the largest |v_j| of the sequence, P enters the products within 2^-8 (2^-8 P), scores are FP32 sums of
exact products (2^-10 P), weights 2^-17 and more below a tile's largest may be off by a fixed step (2^-10 V), the output
is rounded to bf16 (2^-8 |o|).  The join of the pieces is FP32.  The relative L2 distance is held to 2^-7.

Sharing begins where it saves 64 to 112 MB of keys and values (by head_dim): a case's first group has as many members more, each with a
few tokens of its own, as take it beyond that (`fill`), unless the case is about calls that are too small for it."""
import numpy as np
import pytest
import torch

from helpers import rel_l2
from oracle import blockcache

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    """Groups of sequences behind shared tokens.  groups: (shared tokens, [own tokens of each member]); a negative number
    of own tokens is a member shorter than the shared part.  `alone` sequences behind the last group share nothing."""

    def __init__(self, groups, hq, h, d, seed=0, alone=(), spread=3, q_size=1.0, wide=0, fill=True, window=0, tiles=5):
        rng = np.random.default_rng(seed)
        if fill:
            # members beyond what the rule asks for with pieces of up to `tiles` key tiles
            seen = [min(p, window or p) for p, _ in groups]
            least = (48 + d // 4 + tiles * min(d, 128) // 16) << 20
            have = sum((len(m) - 1) * n for n, (_, m) in zip(seen, groups)) * h * 2 * d
            more = max(0, -(-(least - have) // (seen[0] * h * 2 * d)))
            groups = [(groups[0][0], list(groups[0][1]) + [1 + i % 37 for i in range(more)])] + list(groups[1:])
        self.ctx, self.starts, self.shared, rows, nb = [], [0], [], [], 0

        def blocks(n):
            nonlocal nb
            nb += n
            return list(range(nb - n, nb))
        copies = []
        for p, mine in groups:
            common = blocks(p // 16)
            first = None
            for m in mine:
                t = max(0, p + m)
                own = blocks((t + 15) // 16 - min(p, t) // 16)
                rows.append(common[:min(p, t) // 16] + own)
                if p % 16 and t >= p:
                    if first is None:
                        first = own[0]
                    else:
                        copies.append((first, own[0], p % 16))
                self.ctx.append(t)
            self.starts.append(len(self.ctx))
            self.shared.append(p)
        for t in alone:
            rows.append(blocks((t + 15) // 16))
            self.ctx.append(t)
        nb += 2
        perm = rng.permutation(nb).astype(np.int32)
        self.table = np.full((len(rows), max(1, *(len(r) for r in rows)) + wide), -1, np.int32)
        for b, r in enumerate(rows):
            self.table[b, :len(r)] = perm[r]
        self.pools, self.scales = [], []
        for _ in range(2):
            x = rng.standard_normal((nb, h, 16, d))
            s = 2.0 ** rng.integers(-spread, spread + 1, (nb, h)) * 2.0 ** -7
            p8 = torch.from_numpy((x * 128).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            s = s.astype(np.float32)
            for a, c, n in copies:       # a copied block: the shared tokens' codes and their scale
                p8[perm[c], :, :n], s[perm[c]] = p8[perm[a], :, :n], s[perm[a]]
            for b, t in enumerate(self.ctx):
                if t % 16 and not any(t < q for q in self._shared_of(b)):
                    p8[self.table[b, t // 16], :, t % 16:] = rng.choice([0x7F, 0xFF, 0x7E, 3], p8[0, :, t % 16:].shape)
            p8[perm[nb - 2:]] = 0x7F
            self.pools.append(p8)
            self.scales.append(s)
        self.q = torch.from_numpy((rng.standard_normal((len(rows), hq, d)) * q_size).astype(np.float32)).to(torch.bfloat16)

    def _shared_of(self, b):
        return [p for i, p in enumerate(self.shared) if self.starts[i] <= b < self.starts[i + 1]]

    def cache(self):
        return f.BlockCache(*(torch.from_numpy(p).cuda() for p in self.pools), *(torch.from_numpy(s).cuda() for s in self.scales))

    def run(self, **kw):
        self.fault = torch.zeros(1, dtype=torch.int32, device="cuda")
        return f.fp8_block_shared_decode_attn(self.q.cuda(), self.cache(), _i32(self.table), _i32(self.ctx), _i32(self.starts),
                                              _i32(self.shared), fault=self.fault, **kw)

    def exact(self, softmax_scale=0.0, window=0, device="cuda"):
        """(softmax(q K^T) V, softmax(q K^T) |V|, the largest |V|) of every sequence by itself in float64, the shared tokens of a
        group from the blocks that its first sequence names."""
        batch, hq, d = self.q.shape
        h = self.pools[0].shape[1]
        scale = softmax_scale or d ** -0.5
        pool = [torch.from_numpy(p).to(device).view(torch.float8_e4m3fn) for p in self.pools]
        step = [torch.from_numpy(s).to(device).double() for s in self.scales]
        o, mag, top = (torch.zeros(batch, hq, n, dtype=torch.float64, device=device) for n in (d, d, 1))
        for b, t in enumerate(self.ctx):
            if t == 0:
                continue
            lo = max(0, t - window) if window else 0
            spans = [(b, lo, t)]
            for i, n in enumerate(self.shared):
                n = min(n, self.ctx[self.starts[i]]) if self.starts[i] < self.starts[i + 1] else 0
                if self.starts[i] <= b < self.starts[i + 1] and t >= n > lo:
                    spans = [(self.starts[i], lo, n), (b, n, t)]

            def tokens(p, s):
                x = []
                for row, a, e in spans:
                    ids = torch.from_numpy(self.table[row, a // 16:(e + 15) // 16].astype(np.int64)).to(device)
                    y = p.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * s[ids][:, :, None, None]
                    x.append(y.transpose(1, 2).reshape(-1, h, d)[a % 16:e - a // 16 * 16])
                return torch.cat(x)
            k, v = (tokens(p, s) for p, s in zip(pool, step))
            q = self.q[b].to(device).double().view(h, hq // h, d)
            w = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * scale, -1)
            for dst, x in ((o, v), (mag, v.abs())):
                dst[b] = torch.einsum("hgt,thd->hgd", w, x).reshape(hq, d)
            top[b] = v.abs().amax()
        return (x.cpu().numpy() for x in (o, mag, top))

    def check(self, got=None, **kw):
        if got is None:
            got = self.run(**kw)
            assert int(self.fault) == 0
        kw.pop("workspace", None)
        o, mag, top = self.exact(**kw)
        tol = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -10 * top + 2.0 ** -8 * np.abs(o)
        got = got.float().cpu().numpy().astype(np.float64)
        assert np.all(np.isfinite(got))
        err = np.abs(got - o)
        i = np.unravel_index(int(np.argmax(err - tol)), err.shape)
        assert np.all(err <= tol), f"{err[i]:.3e} above {tol[i]:.3e} at {i} (T {self.ctx[i[0]]})"
        assert rel_l2(got, o) <= 2.0 ** -7


def test_the_oracle_here_is_the_other_tests_one():
    c = Case([(500, [1, 30, 3]), (33, [4, 5])], 8, 2, 64, alone=(0, 70), fill=False)
    a = (c.pools[0], c.pools[1], c.scales[0], c.scales[1], c.table, c.ctx, None)
    q = c.q.float().numpy().astype(np.float64)
    for kw in ({}, {"window": 100}, {"softmax_scale": 0.3}):
        o, mag, _ = c.exact(**kw)
        np.testing.assert_allclose(o, blockcache.attend(q, *a, **kw), rtol=1e-9, atol=1e-12)
        np.testing.assert_allclose(mag, blockcache.p_bound(q, *a, **kw), rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
def test_one_group(d, g):
    if g * d > 2048:
        pytest.skip("group and head_dim beyond the decode's limit")
    Case([(6400, [1, 0, 17, 200, 3, 16, 40, 128])], 2 * g, 2, d, seed=d + g).check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("groups,alone,hq,h", [
    ([(5000, [5, 77]), (2049, [1] * 9), (3333, [600, 0, 30])], (300, 0, 17), 8, 2),
    ([(4099, [1] * 70)], (), 8, 2), ([(100, [10, 10]), (9000, [40] * 5), (0, [33, 1]), (7, [9])], (5000,), 4, 1),
    ([(8000, [3, -100, -7990, -8000, 50])], (), 8, 2), ([(16, [1, 2]), (16 * 400, [300] * 4)], (1,), 16, 8),
])
def test_groups(d, groups, alone, hq, h):
    Case(groups, hq, h, d, seed=len(groups) + hq, alone=alone).check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 50, 700, 6000])
def test_windows(d, window):
    # (a window of 1 or 50 saves too little to be worth sharing)
    Case([(6003, [1, 0, 60, 900, 5, 5]), (4000, [10, 2000, -30])], 16, 8, d, seed=window, fill=window > 50, window=window).check(window=window)


@pytest.mark.parametrize("groups,hq,h,d", [
    ([(1, [0, 0])], 2, 2, 64), ([(33, [1, 2, 3, 4])], 8, 2, 128), ([(2048, [1, 50, 100, 150])], 32, 8, 128),
    ([(2048, [5, 6]), (700, [1, 1, 1]), (0, [16]), (30, [0, 0])], 16, 8, 64),
])
def test_calls_too_small_to_share(groups, hq, h, d):
    c = Case(groups, hq, h, d, seed=len(groups), fill=False)
    c.check()
    assert torch.equal(c.run(), f.fp8_block_decode_attn(c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx)))


@pytest.mark.parametrize("groups,hq,h,d", [
    # a wide table and a batch large enough that only the lengths, on the GPU, tell that sharing does not pay
    ([(160, [1, 2, 3]), (40, [5, 6])], 16, 8, 64), ([(0, [400, 900, 16]), (700, [0, 1])], 8, 8, 128),
])
def test_lengths_too_short_to_share(groups, hq, h, d):
    c = Case(groups, hq, h, d, seed=2, fill=False, wide=2048)
    c.check()
    assert torch.equal(c.run(), f.fp8_block_decode_attn(c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx)))


@pytest.mark.parametrize("groups,hq,h,d", [
    ([(320, [int(x) for x in range(1, 5)]) for _ in range(110)], 8, 4, 128), ([(1280, [1] * 2) for _ in range(80)], 32, 8, 64),
    ([(96, [0, 1, 2]) for _ in range(600)], 8, 8, 64),
])
def test_many_groups(groups, hq, h, d):
    Case(groups, hq, h, d, seed=3).check()


def test_one_long_prefix_of_one_head():
    Case([(60000, [10, 1])], 2, 1, 64, seed=5).check()


def test_scales_far_apart():
    c = Case([(5000, [100, 20, 3, 9])], 8, 2, 128, seed=6, spread=0)
    rng = np.random.default_rng(7)
    for s in c.scales:
        s *= (2.0 ** rng.integers(-40, 1, s.shape)).astype(np.float32)
    c.scales[1][c.table[0, 3:9]] = 0.0
    c.check()


def test_all_shared_and_scale():
    Case([(3000, [0] * 6)], 8, 2, 128, seed=8).check(softmax_scale=0.25)


def test_no_groups():
    c = Case([], 8, 2, 128, seed=9, alone=(100, 700, 0, 33), fill=False)
    c.check()
    want = f.fp8_block_decode_attn(c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx))
    assert torch.equal(c.run(), want)


def test_bad_queries_keep_to_their_rows():
    c = Case([(5000, [40, 3, 9, 70])], 8, 2, 128, seed=10)
    want = c.run()
    c.q[1, 5, 7] = float("nan")
    c.q[2, 0, 1] = float("inf")
    got = c.run()
    assert bool(got[1, 5].isnan().all()) and bool(got[2, 0].isnan().all())
    bad = torch.zeros(len(c.ctx), 8, dtype=torch.bool)
    bad[1, 5] = bad[2, 0] = True
    assert torch.equal(got[~bad], want[~bad])


def test_bad_groups_share_nothing_and_are_reported():
    c = Case([(4000, [40, 3, 9]), (3000, [5, 6])], 8, 2, 128, seed=11)
    n = c.starts[1]
    plain = f.fp8_block_decode_attn(c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx))
    assert not torch.equal(c.run(), plain), "the unspoiled call shares"
    for starts, shared, fault in (([0, n, n - 1], [4000, 3000], f.FAULT_QLEN), ([-1, n, n + 2], [4000, 3000], f.FAULT_QLEN),
                                  ([0, n, n + 3], [4000, 3000], f.FAULT_QLEN), ([0, n, n + 2], [-1, 3000], f.FAULT_CONTEXT),
                                  ([0, n, n + 2], [16 * c.table.shape[1] + 1, 3000], f.FAULT_CONTEXT)):
        c.starts, c.shared = starts, shared
        assert torch.equal(c.run(), plain)
        assert int(c.fault) == fault


def test_bad_blocks_are_reported():
    c = Case([(5000, [40, 3, 9])], 8, 2, 128, seed=12)
    c.table[:, 7] = 1 << 29
    c.pools[0][0], c.pools[1][0] = 0x10, 0x10
    c.run()
    assert int(c.fault) == f.FAULT_BLOCK_ID


def test_one_workspace_for_calls_that_grow_and_shrink():
    big, small = Case([(5000, [40] * 40)], 8, 2, 128, seed=13), Case([(4000, [3, 9]), (6000, [1, 1, 1])], 8, 2, 128, seed=14, alone=(50,))
    ws = f.block_shared_workspace(max(len(big.ctx), len(small.ctx)), 8, big.cache(), 2)
    for c in (big, small, big, small, small):
        c.check(workspace=ws)
    one = big.run(workspace=ws)
    assert torch.equal(one, big.run(workspace=ws)), "the same bits every time"
    plain = f.fp8_block_decode_attn(small.q.cuda(), small.cache(), _i32(small.table), _i32(small.ctx), workspace=ws)
    small.check(plain)
    with pytest.raises(f.FkvError):
        big.run(workspace=ws[:65536])


def test_captured_and_replayed_with_other_groups_and_lengths():
    c = Case([(5000, [40, 300, 9, 1]), (3000, [5, 6])], 8, 2, 128, seed=15)
    cache, q, tab, ctx, starts, shared = c.cache(), c.q.cuda(), _i32(c.table), _i32(c.ctx), _i32(c.starts), _i32(c.shared)
    n = c.starts[1]
    ws, out = f.block_shared_workspace(n + 2, 8, cache, 2), torch.empty_like(q)
    f.fp8_block_shared_decode_attn(q, cache, tab, ctx, starts, shared, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.fp8_block_shared_decode_attn(q, cache, tab, ctx, starts, shared, out=out, workspace=ws)
    g.replay()
    c.check(out)
    c.starts, c.shared, c.ctx = [0, n - 1, n - 1], [4990, 0], [5011, 5300, 5001, 5000] + c.ctx[4:n] + [3001, 2]
    starts.copy_(_i32(c.starts)), shared.copy_(_i32(c.shared)), ctx.copy_(_i32(c.ctx))
    out.zero_()
    g.replay()
    c.check(out)


def test_on_another_stream_beside_another_call():
    c, e = Case([(5000, [40, 300, 9, 1])], 8, 2, 128, seed=16), Case([(4000, [7, 8])], 8, 2, 128, seed=17)
    s = torch.cuda.Stream()
    a = (c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx), _i32(c.starts), _i32(c.shared))
    b = (e.q.cuda(), e.cache(), _i32(e.table), _i32(e.ctx), _i32(e.starts), _i32(e.shared))
    torch.cuda.synchronize()
    for _ in range(20):
        x = f.fp8_block_shared_decode_attn(*a, stream=s)
        y = f.fp8_block_shared_decode_attn(*b)
    torch.cuda.synchronize()
    c.check(x), e.check(y)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_wait_that_runs_out(d):
    """The copies' wait for a free stage given less time than the pipeline takes: reported, and the next call is sound."""
    c = Case([(100000, [100, 300])], 8, 1, d, seed=18, tiles=8)      # (782 key tiles of one KV head: six in a piece)
    cache, q, tab, ctx, starts, shared = c.cache(), c.q.cuda(), _i32(c.table), _i32(c.ctx), _i32(c.starts), _i32(c.shared)
    ws, fault, lib = f.block_shared_workspace(len(c.ctx), q.shape[1], cache, 1), _i32([0]), f.load_library()

    def call():
        return f.fp8_block_shared_decode_attn(q, cache, tab, ctx, starts, shared, workspace=ws, fault=fault)
    ref = call()
    torch.cuda.synchronize()
    assert int(fault) == 0
    assert not torch.equal(ref, f.fp8_block_decode_attn(q, cache, tab, ctx)), "the call shares"
    lib.fkv_set_decode_wait_limit_ns(1)
    try:
        for _ in range(2):
            call()
        torch.cuda.synchronize()
    finally:
        lib.fkv_set_decode_wait_limit_ns(0)
    assert int(fault) == f.FAULT_TIMEOUT
    fault.zero_()
    for _ in range(2):
        assert torch.equal(call(), ref)
    assert int(fault) == 0


def _within(got, o, mag, top):
    """The tolerance above, against an `exact` that was taken before the case was spoiled."""
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), f"not finite: sequences {np.unique(np.nonzero(~np.isfinite(got))[0]).tolist()}"
    assert np.all(np.abs(got - o) <= (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -10 * top + 2.0 ** -8 * np.abs(o))
    assert rel_l2(got, o) <= 2.0 ** -7


@pytest.mark.parametrize("d,members", [(64, 45), (128, 28), (256, 24)])
@pytest.mark.parametrize("longest", [0, -1])
def test_windows_over_evicted_blocks(d, members, longest):
    """What lies before every member's window is gone: blocks taken out of the table, their slots NaN codes.  The group's
    first sequence is the longest one, whose row has lost blocks that others still see, or the last is."""
    w, p = 3000, 4003
    own = [45 + 7 * i for i in range(members)]
    own.insert(0 if longest == 0 else members, 900)
    c = Case([(p, own)], 16, 8, d, seed=d, fill=False)
    exact = list(c.exact(window=w))
    plain = f.fp8_block_decode_attn(c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx), window=w)
    least = min(c.ctx) - w
    assert least % 16 and least > p - w
    row = c.table[int(np.argmin(c.ctx))]
    for pool in c.pools:
        pool[row[:least // 16]] = 0x7F
        pool[row[least // 16], :, :least % 16] = 0x7F
    for b, t in enumerate(c.ctx):
        c.table[b, :(t - w) // 16] = -1
    got = c.run(window=w)
    _within(got, *exact)
    assert int(c.fault) == 0
    assert not torch.equal(got, plain), "the call shares"


@pytest.mark.parametrize("own", [[2999, 2998], [3000, 3500, 4000], [1, 3100]])
def test_windows_that_hardly_reach_the_shared_tokens(own):
    """Members whose windows begin at, behind or just before the end of the shared tokens, beside a group that shares."""
    w = 3000
    Case([(5000, own), (4000, [40 + i for i in range(30)])], 16, 8, 128, seed=len(own), fill=False).check(window=w)


@pytest.mark.parametrize("window", [0, 3000])
def test_a_context_beyond_the_table(window):
    """Reported and clamped to the table, for the shared part's windows too."""
    c = Case([(4000, [880] + [30 + 5 * i for i in range(28)])], 16, 8, 128, seed=19, fill=False)
    assert c.ctx[0] == 16 * c.table.shape[1] == max(c.ctx)
    exact = list(c.exact(window=window))
    within = c.run(window=window)
    c.ctx[0] += 700
    got = c.run(window=window)
    assert int(c.fault) == f.FAULT_CONTEXT
    _within(got, *exact)
    assert torch.equal(got, within)
