"""fp8_block_attn_weights on the GPU against the float64 softmax.

Tolerance of w_j, derived before the first run.  A weight p = 2^(x - lse) is off by what its score and its row's sum
are off by.  A score of row r and key j, in natural units:
  * the query's terms leave at most 2^-17 of the row's largest element: 2^-17 |q|max tau sum_d |k_d|;
  * FP32 sums of 2 D exact products and the scaling: (2 D + 4) 2^-24 tau sum_d |q_d k_d|.
E, the largest of those two together, enters twice (score and sum), ex2 and lg2 and the subtraction add 2^-20, and the row's
and the column's FP32 sums of n terms at most n 2^-24 each (n keys, n rows), what was there before and the decay 2^-23 of
their own sum.  So |error| <= (2 E + 2^-20 + (keys + rows) 2^-24) w_j + 2^-23 |before|, and a number below 2^-100 may be flushed.
Those are worst cases; roundings that are not all alike leave far less: the relative L2 distance of the added part is held to
2^-16 (sqrt(2 D) 2^-24 of scores up to 8, and as much again for the sums)."""
import numpy as np
import pytest
import torch

from oracle import blockcache, longcontext
from test_gpu_block_timeout import _runs_out

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    """A seeded block-scaled cache with chunks of queries: any byte (NaN codes too) behind the sequences."""

    def __init__(self, ctx, new, hq, h, d, seed=0, spread=3, q_size=1.0, wide=0):
        rng = np.random.default_rng(seed)
        n = [(t + 15) // 16 for t in ctx]
        nb = sum(n) + 2
        perm = rng.permutation(nb).astype(np.int32)
        self.table, at = np.full((len(ctx), max(1, *n) + wide), -1, np.int32), 0
        x = rng.standard_normal((nb, h, 16, d))
        self.k_scale = (2.0 ** rng.integers(-spread, spread + 1, (nb, h)) * 2.0 ** -7).astype(np.float32)
        self.k = torch.from_numpy((x * 128).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        for b, m in enumerate(n):
            self.table[b, :m] = perm[at:at + m]
            at += m
        self.k[perm[at:]] = 0x7F
        for b, t in enumerate(ctx):
            if t % 16:
                self.k[self.table[b, t // 16], :, t % 16:] = rng.choice([0x7F, 0xFF, 0x7E, 3], self.k[0, :, t % 16:].shape)
        self.ctx, self.new, self.cu = list(ctx), list(new), np.concatenate(([0], np.cumsum(new)))
        self.q = torch.from_numpy((rng.standard_normal((int(self.cu[-1]), hq, d)) * q_size).astype(np.float32)).to(torch.bfloat16)
        L = self.table.shape[1] * 16 + 5
        self.before = (rng.random((len(ctx), h, L)) * 0.01).astype(np.float32)

    def cache(self):
        k, s = torch.from_numpy(self.k).cuda(), torch.from_numpy(self.k_scale).cuda()
        return f.BlockCache(k, k, s, s)

    def run(self, decay=1.0, weights=None, **kw):
        self.weights = torch.from_numpy(self.before.copy()).cuda() if weights is None else weights
        self.fault = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = f.fp8_block_attn_weights(self.q.cuda(), _i32(self.cu), max(self.new), self.cache(), _i32(self.table), _i32(self.ctx),
                                       self.weights, decay=decay, fault=self.fault, **kw)
        assert got is self.weights or got.data_ptr() == self.weights.data_ptr()
        return self.weights.cpu().numpy().astype(np.float64)

    def check(self, decay=1.0, softmax_scale=0.0, rows=slice(None)):
        got = self.run(decay, softmax_scale=softmax_scale)
        assert int(self.fault) == 0
        q = self.q.float().numpy().astype(np.float64)
        d, hq, h = q.shape[2], q.shape[1], self.k.shape[1]
        tau = softmax_scale or d ** -0.5
        new = longcontext.softmax_weights(q, self.k, self.k_scale, self.table, self.ctx, self.cu, softmax_scale)
        for b, (t, n) in enumerate(zip(self.ctx, self.new)):
            if n == 0:
                assert np.array_equal(got[b], self.before[b].astype(np.float64))
                continue
            assert np.array_equal(got[b, :, t:], self.before[b, :, t:].astype(np.float64)), "behind the sequence"
            want = longcontext.accumulate(self.before[b], new[b], n, decay)[:, :t]
            chunk = np.abs(q[self.cu[b]:self.cu[b + 1]])
            for g in range(h):
                K = np.abs(blockcache.sequence(self.k, self.k_scale, self.table[b], t, g))
                Q = chunk[:, g * (hq // h):(g + 1) * (hq // h)].reshape(-1, d)
                E = tau * float((2.0 ** -17 * Q.max(1)[:, None] * K.sum(1)[None] + (2 * d + 4) * 2.0 ** -24 * (Q @ K.T)).max())
                old = np.zeros(t)
                old[:t - n] = np.abs(decay * self.before[b, g, :t - n])
                tol = (2 * E + 2.0 ** -20 + (t + n * hq // h) * 2.0 ** -24) * new[b][g] + 2.0 ** -23 * (old + new[b][g]) + 2.0 ** -100
                err = np.abs(got[b, g, :t] - want[g])
                i = int(np.argmax(err - tol))
                assert np.all(err <= tol), f"sequence {b} head {g} key {i}: {err[i]:.3e} above {tol[i]:.3e}, w {new[b][g][i]:.3e}"
                if decay == 0.0:
                    rel = np.linalg.norm(got[b, g, :t] - want[g]) / np.linalg.norm(want[g])
                    assert rel <= 2.0 ** -16, f"sequence {b} head {g}: rel_l2 {rel:.2e}"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 2, 3, 4, 7, 8, 16])
def test_one_query_per_sequence(d, g):
    c = Case([1, 15, 16, 17, 127, 128, 129, 300, 700], [1] * 9, 3 * g, 3, d, seed=d + g)
    c.check(1.0)
    c.check(0.0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,new,hq,h", [
    ([400, 9, 130], [3, 9, 1], 8, 2), ([300, 260], [33, 128], 4, 1), ([500, 77, 129, 64], [64, 77, 1, 30], 8, 2),
    ([1000], [300], 6, 2), ([700, 512], [700, 257], 2, 2), ([40, 300], [5, 40], 20, 4), ([200], [3], 160, 1),
])
def test_chunks(d, ctx, new, hq, h):
    c = Case(ctx, new, hq, h, d, seed=len(ctx) + ctx[0])
    c.check(0.0)
    c.check(0.875)


@pytest.mark.parametrize("new", [[1, 1], [40, 33]])
def test_long_contexts(new):
    c = Case([9000, 5003], new, 4, 1, 64, seed=3)
    c.check(0.0)
    c.check(1.0)


def test_many_sequences_some_without_queries():
    rng = np.random.default_rng(0)
    ctx = rng.integers(1, 200, 70).tolist()
    new = [int(rng.integers(0, min(t, 9) + 1)) for t in ctx]
    new[0] = 0
    Case(ctx, new, 4, 2, 64, seed=5).check(0.0)
    Case(ctx, [min(n, 2) for n in new], 8, 2, 128, seed=6, wide=40).check(1.0)


@pytest.mark.parametrize("new", [[1, 1], [50, 20]])
def test_scales_far_apart_and_zero(new):
    c = Case([300, 90], new, 4, 2, 128, seed=8, spread=0)
    c.k_scale[:] = (2.0 ** np.random.default_rng(1).integers(-60, -5, c.k_scale.shape)).astype(np.float32)
    c.k_scale[c.table[0, :4]] = 0.0
    c.check(0.0)
    c.q.zero_()
    c.check(0.0)      # every visible key alike


def test_softmax_scale_and_large_scores():
    c = Case([333, 64], [20, 1], 4, 1, 64, seed=9, q_size=6.0, spread=1)
    c.check(0.0, softmax_scale=0.3)


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 40, 40]])
def test_bad_queries_reach_their_own_head_and_the_keys_they_see(new):
    c = Case([100, 90, 80], new, 4, 2, 64, seed=10)
    i = int(c.cu[1])
    c.q[i, 1, 3] = float("nan")
    got = c.run(0.0)
    seen = 90 - new[1] + 1
    assert np.all(np.isnan(got[1, 0, :seen]))
    ok = got.copy()
    ok[1, 0, :seen] = 0
    assert np.all(np.isfinite(ok))
    c.q[i, 1, 3] = 0
    assert np.array_equal(c.run(0.0)[1, 0, seen:], ok[1, 0, seen:])


def test_decay_zero_does_not_read_what_was_there():
    for new in ([1, 1], [30, 70]):
        c = Case([100, 70], new, 4, 2, 64, seed=11)
        c.before[:] = np.nan
        got = c.run(0.0)
        assert np.all(np.isfinite(got[0, :, :100])) and np.all(np.isfinite(got[1, :, :70]))
        c.before[:] = 0.5
        assert np.array_equal(c.run(0.0)[0, :, :100], got[0, :, :100])


@pytest.mark.parametrize("new", [[1] * 4, [30] * 4])
def test_bad_lengths_and_blocks_are_reported(new):
    c = Case([100, 60, 50, 64], new, 4, 2, 64, seed=12)
    want = c.run(1.0)
    c.ctx = [100, 0, 16 * c.table.shape[1] + 6, 64]       # rows beyond the context; a context beyond the table
    c.table[2] = c.table[0]
    got = c.run(1.0)
    assert int(c.fault) == f.FAULT_QLEN | f.FAULT_CONTEXT
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[3], want[3])
    assert np.array_equal(got[1], c.before[1].astype(np.float64))
    c.ctx = [100, 60, 50, 64]
    c.table[1, 0] = 1 << 30
    c.k[0] = 0x10
    c.run(1.0)
    assert int(c.fault) == f.FAULT_BLOCK_ID


@pytest.mark.parametrize("new", [[1, 1], [64, 5]])
def test_the_same_bits_every_time_and_with_any_workspace(new):
    c = Case([3000, 700], new, 8, 2, 128, seed=13)
    one = c.run(1.0)
    n = f.fp8_block_attn_weights_workspace_size(2, sum(new), max(new), 8, 2, 128, c.table.shape[1])
    for fill in (0, 0xFF):
        ws = torch.full((max(n, 256),), fill, dtype=torch.uint8, device="cuda")
        assert np.array_equal(c.run(1.0, workspace=ws), one)
    with pytest.raises(f.FkvError):
        c.run(1.0, workspace=ws[:n - 1])


@pytest.mark.parametrize("new", [[1, 1], [40, 7]])
def test_captured_and_replayed_with_other_lengths(new):
    c = Case([500, 300], new, 4, 2, 64, seed=14)
    c.run(1.0)
    cache, q, cu, tab, ctx = c.cache(), c.q.cuda(), _i32(c.cu), _i32(c.table), _i32(c.ctx)
    w = torch.from_numpy(c.before.copy()).cuda()
    ws = f.attn_weights_workspace(2, q.shape[0], max(new), 4, cache, tab.shape[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.fp8_block_attn_weights(q, cu, max(new), cache, tab, ctx, w, decay=0.0, workspace=ws)
    c.ctx = [417, 100]
    ctx.copy_(_i32(c.ctx))
    g.replay()
    want = c.run(0.0)
    got = w.cpu().numpy().astype(np.float64)
    for b, t in enumerate(c.ctx):
        assert np.array_equal(got[b, :, :t], want[b, :, :t])


def test_on_another_stream():
    c = Case([800, 300], [16, 1], 4, 2, 128, seed=15)
    want = c.run(1.0)
    s = torch.cuda.Stream()
    args = (c.q.cuda(), _i32(c.cu), 16, c.cache(), _i32(c.table), _i32(c.ctx), torch.from_numpy(c.before.copy()).cuda())
    s.wait_stream(torch.cuda.current_stream())
    got = f.fp8_block_attn_weights(*args, stream=s)
    s.synchronize()
    assert np.array_equal(got.cpu().numpy().astype(np.float64), want)


def _large_pool(sequences, tokens, d):
    """A pool larger than the L2 cache, so that copies wait for memory: 64 x 8,000 tokens are 262 MB of keys."""
    h, per = 512 // d, -(-tokens // 16)
    gen = torch.Generator(device="cuda").manual_seed(d)
    k = torch.randint(0, 256, (sequences * per, h, 16, d), dtype=torch.uint8, device="cuda", generator=gen) & 0xBB
    s = torch.full((sequences * per, h), 2.0 ** -5, device="cuda")
    table = torch.randperm(sequences * per, device="cuda", generator=gen).to(torch.int32).view(sequences, per)
    return h, f.BlockCache(k, k, s, s), table


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [4, 7, 16])
def test_wait_that_runs_out_few_rows(d, g):
    """The copies' wait for a free stage given less time than the pipeline takes, in a workspace of any bytes: reported, and the next
    call is sound."""
    h, cache, table = _large_pool(64, 8000, d)
    q = torch.randn(64, g * h, d, generator=torch.Generator().manual_seed(g)).to(torch.bfloat16).cuda()
    lens, cu = _i32([8000 - 9 * b for b in range(64)]), _i32(range(65))
    ws = f.attn_weights_workspace(64, 64, 1, g * h, cache, table.shape[1])

    def call(fault):
        w = torch.zeros(64, h, 8000, device="cuda")
        ws.fill_(0x7F)
        return f.fp8_block_attn_weights(q, cu, 1, cache, table, lens, w, decay=0.0, workspace=ws, fault=fault)
    _runs_out(call)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sequences,tokens,g,new", [(4, 3000, 16, 160), (64, 8000, 7, 33), (1024, 100, 2, 9)])
def test_wait_that_runs_out_many_rows(d, sequences, tokens, g, new):
    """The same for the two passes over many rows: row tiles that stream past the keys, long contexts, and many short ones, whose
    pieces follow one another faster than their tiles are done with (either pass stops there)."""
    h, cache, table = _large_pool(sequences, tokens, d)
    q = torch.randn(sequences * new, g * h, d, generator=torch.Generator().manual_seed(g)).to(torch.bfloat16).cuda()
    lens, cu = _i32([tokens] * sequences), _i32(np.arange(sequences + 1) * new)
    ws = f.attn_weights_workspace(sequences, sequences * new, new, g * h, cache, table.shape[1])

    def call(fault):
        w = torch.zeros(sequences, h, tokens, device="cuda")
        ws.fill_(0x7F)
        return f.fp8_block_attn_weights(q, cu, new, cache, table, lens, w, decay=0.0, workspace=ws, fault=fault)
    _runs_out(call)


@pytest.mark.parametrize("cu", [[0, 200, 50, 100], [100, 200, 50, 100], [0, 1000, 150, 200], [0, 130, 20, 200]])
def test_starts_that_decrease(cu):
    """A sequence's weights do not depend on what a bad one does to the starts behind it: whose rows lie behind those of all earlier
    sequences (of those that are sound by themselves) get their weights, the others keep what was there."""
    c = Case([300, 260, 400], [200, 0, 0], 16, 4, 64, seed=20)
    c.cu, rows = cu, [(cu[b], cu[b + 1] - cu[b]) for b in range(3)]
    got = c.run(0.0)
    assert int(c.fault) == f.FAULT_QLEN
    end = 0
    for b, (r, n) in enumerate(rows):
        sound = 0 < n <= 200 and r + n <= 200 and n <= c.ctx[b]
        if sound and r >= end:
            want = longcontext.softmax_weights(c.q[r:r + n].float().numpy().astype(np.float64), c.k, c.k_scale, c.table[b:b + 1], c.ctx[b:b + 1], [0, n])[0]
            assert np.linalg.norm(got[b, :, :c.ctx[b]] - want) <= 2.0 ** -16 * np.linalg.norm(want), f"sequence {b}"
        else:
            assert np.array_equal(got[b], c.before[b].astype(np.float64)), f"sequence {b}"
        end = max(end, r + n) if sound else end


@pytest.mark.parametrize("cu,max_q", [([0, 3, 1, 2], 3)])
def test_starts_that_decrease_few_rows(cu, max_q):
    c = Case([300, 260, 400], [3, 0, 0], 16, 4, 64, seed=21)
    c.cu = cu
    got = c.run(0.0)
    assert int(c.fault) == f.FAULT_QLEN
    want = longcontext.softmax_weights(c.q[:3].float().numpy().astype(np.float64), c.k, c.k_scale, c.table[:1], c.ctx[:1], [0, 3])[0]
    assert np.linalg.norm(got[0, :, :300] - want) <= 2.0 ** -16 * np.linalg.norm(want)
    assert np.array_equal(got[1], c.before[1].astype(np.float64))


@pytest.mark.parametrize("new", [[1, 1], [40, 20]])
def test_weights_of_no_tokens(new):
    """weights_len 0: every context is clamped to 0, and a query without keys is skipped."""
    c = Case([100, 60], new, 4, 2, 64, seed=22)
    c.before = c.before[:, :, :0]
    c.run(1.0)
    assert int(c.fault) == f.FAULT_CONTEXT | f.FAULT_QLEN
