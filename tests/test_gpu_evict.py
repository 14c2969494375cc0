"""kv_block_evict on the GPU against the oracle: indices, codes, scales and moved weights bit for bit (the selection is by
comparisons, the codes by fixed roundings: nothing is left to tolerance)."""
import numpy as np
import pytest
import torch

from oracle import longcontext

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, ctx, budget, sink, recent, h, d, seed=0, weights=None, wide=0, any_scale=False):
        rng = np.random.default_rng(seed)
        self.ctx, self.budget, self.sink, self.recent = ctx, budget, sink, recent
        keep = [min(t, budget) for t in ctx]
        n = [(t + 15) // 16 for t in ctx + keep]
        nb = sum(n) + 3
        perm, at, rows = rng.permutation(nb).astype(np.int32), 0, []
        for m in n:
            rows.append(perm[at:at + m])
            at += m
        width, room = max(1, max(n[:len(ctx)])) + wide, max(1, max(n[len(ctx):])) + wide
        self.table, self.new_table = np.full((len(ctx), width), -1, np.int32), np.full((len(ctx), room), -1, np.int32)
        for b in range(len(ctx)):
            self.table[b, :n[b]] = rows[b]
            self.new_table[b, :n[len(ctx) + b]] = rows[len(ctx) + b]
        self.pools = [rng.integers(0, 256, (nb, h, 16, d)).astype(np.uint8) for _ in range(2)]      # NaN codes among them
        self.scales = [(rng.uniform(0.001, 3.0, (nb, h)) if any_scale else 2.0 ** rng.integers(-12, 4, (nb, h))).astype(np.float32)
                       for _ in range(2)]
        L = width * 16
        w = rng.standard_normal((len(ctx), h, L)) if weights is None else weights(rng, (len(ctx), h, L))
        self.weights = np.asarray(w, np.float32)
        self.new_len = room * 16

    def run(self, **kw):
        self.cache = f.BlockCache(*(torch.from_numpy(p.copy()).cuda() for p in self.pools),
                                  *(torch.from_numpy(s.copy()).cuda() for s in self.scales))
        self.moved = torch.full((*self.weights.shape[:2], self.new_len), -3.0, device="cuda")
        self.fault = torch.zeros(1, dtype=torch.int32, device="cuda")
        return f.kv_block_evict(self.cache, torch.from_numpy(self.table).cuda(), torch.tensor(self.ctx, dtype=torch.int32).cuda(),
                                torch.from_numpy(self.weights).cuda(), self.budget, torch.from_numpy(self.new_table).cuda(),
                                sink=self.sink, recent=self.recent, new_weights=self.moved, fault=self.fault, **kw)

    def check(self):
        lens, kept = self.run()
        assert int(self.fault) == 0
        want, want_lens = longcontext.evict(self.pools, self.scales, self.table, self.ctx, self.weights, self.budget, self.new_table,
                                            self.sink, self.recent)
        assert np.array_equal(lens.cpu().numpy(), want_lens)
        assert np.array_equal(kept.cpu().numpy(), want)
        for got, pool, scale, name in ((self.cache.k_cache, self.pools[0], self.scales[0], "k"), (self.cache.v_cache, self.pools[1], self.scales[1], "v")):
            assert np.array_equal((self.cache.k_scale if name == "k" else self.cache.v_scale).cpu().numpy(), scale), name
            got = got.cpu().numpy()
            nan = (pool & 0x7F) == 0x7F                                   # a kept NaN is a NaN
            assert np.array_equal(np.where(nan, 0x7F, got & np.where(nan, 0x7F, 0xFF)), np.where(nan, 0x7F, pool)), name
        moved = self.moved.cpu().numpy()
        for b, n in enumerate(want_lens):
            for g in range(moved.shape[1]):
                assert np.array_equal(moved[b, g, :n], self.weights[b, g][want[b, g, :n]], equal_nan=True)
                assert np.all(moved[b, g, n:] == -3.0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,budget,sink,recent,h", [
    ([0, 1, 15, 16, 17, 33, 300], 16, 0, 0, 3), ([1, 2, 40], 1, 0, 0, 1), ([40, 41], 7, 3, 4, 2), ([100, 5, 64], 64, 4, 10, 2),
    ([1000], 999, 1, 1, 1), ([2500, 2048, 31], 300, 4, 64, 2), ([64] * 40, 33, 0, 33, 1),
])
def test_evict(d, ctx, budget, sink, recent, h):
    Case(ctx, budget, sink, recent, h, d, seed=len(ctx) + budget).check()


@pytest.mark.parametrize("ctx,budget,h", [([5000, 12345], 1000, 1), ([40001], 20000, 2), ([30000, 100, 8193], 8192, 3), ([90001, 66000], 30000, 1)])
def test_evict_clusters(ctx, budget, h):
    Case(ctx, budget, 4, 100, h, 64, seed=budget, wide=3).check()


def test_evict_more_keys_than_shared_memory_holds():
    """400,001 tokens of one head: eight CTAs hold 40,960 keys each, the walk goes over global memory."""
    Case([400001], 700, 4, 100, 1, 64, seed=9).check()


def _ties(rng, shape):
    return rng.integers(0, 3, shape)


def _same(rng, shape):
    return np.zeros(shape)


def _special(rng, shape):
    return rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, 1.0], np.float32), shape)


def _close(rng, shape):
    return 1.0 + rng.integers(0, 700, shape) * 2.0 ** -23         # differ in the last digit of the search only


@pytest.mark.parametrize("weights", [_ties, _same, _special, _close])
@pytest.mark.parametrize("ctx,budget", [([100, 4097], 50), ([20000], 4001), ([80003], 5001)])
def test_evict_equal_and_special_weights(weights, ctx, budget):
    Case(ctx, budget, 2, 5, 2, 64, seed=budget, weights=weights).check()


def test_evict_any_scales():
    Case([300, 170], 100, 0, 10, 2, 128, seed=4, any_scale=True).check()


def test_evict_shared_sources_and_without_weights_to_move():
    """Two sequences read the same blocks; new_weights None."""
    c = Case([100, 100], 40, 2, 8, 2, 64, seed=6)
    c.table[1] = c.table[0]
    c.check()
    cache = c.cache
    lens, kept = f.kv_block_evict(cache, torch.from_numpy(c.table).cuda(), torch.tensor([100, 100], dtype=torch.int32).cuda(),
                                  torch.from_numpy(c.weights).cuda(), 40, torch.from_numpy(c.new_table).cuda(), 2, 8)
    assert lens.tolist() == [40, 40] and int(kept.min()) == 0


def test_evict_bad_blocks_and_contexts_are_reported():
    c = Case([60, 60, 60], 20, 0, 0, 1, 64, seed=8)
    c.table[0, 1] = 10 ** 6                     # read as block 0
    c.new_table[1, 0] = -1                      # skipped
    c.ctx = [60, 60, 16 * c.table.shape[1] + 1]  # clamped to the table
    before = [p.copy() for p in c.pools]
    c.run()
    assert int(c.fault) == f.FAULT_BLOCK_ID | f.FAULT_CONTEXT
    assert np.array_equal(c.cache.k_cache.cpu().numpy()[c.table[1]], before[0][c.table[1]])
    c.ctx = [60, -1, 60]
    lens, kept = c.run()
    assert lens.tolist() == [20, 0, 20] and int(kept[1].max()) == -1 and int(c.fault) & f.FAULT_CONTEXT


def test_evict_captured_and_replayed_with_other_contents():
    c = Case([500, 90], 64, 4, 16, 2, 64, seed=11)
    lens, kept = c.run()
    torch.cuda.synchronize()
    cache, tab, new = c.cache, torch.from_numpy(c.table).cuda(), torch.from_numpy(c.new_table).cuda()
    ctx, w = torch.tensor(c.ctx, dtype=torch.int32).cuda(), torch.from_numpy(c.weights).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.kv_block_evict(cache, tab, ctx, w, 64, new, 4, 16, new_lens=lens, kept=kept)
    w.copy_(w.flip(2))
    ctx.copy_(torch.tensor([400, 70]))
    g.replay()
    torch.cuda.synchronize()
    for b, t in enumerate((400, 70)):
        for h in range(2):
            want = longcontext.kept_tokens(w[b, h].cpu().numpy(), t, 64, 4, 16)
            assert np.array_equal(kept[b, h, :want.size].cpu().numpy(), want)


def test_evict_on_another_stream():
    c = Case([3000], 128, 4, 16, 2, 128, seed=12)
    s = torch.cuda.Stream()
    c.run()
    s.wait_stream(torch.cuda.current_stream())
    lens, kept = f.kv_block_evict(c.cache, torch.from_numpy(c.table).cuda(), torch.tensor(c.ctx, dtype=torch.int32).cuda(),
                                  torch.from_numpy(c.weights).cuda(), 128, torch.from_numpy(c.new_table).cuda(), 4, 16, stream=s)
    s.synchronize()
    want = longcontext.kept_tokens(c.weights[0, 1], 3000, 128, 4, 16)
    assert np.array_equal(kept[0, 1].cpu().numpy(), want)


def test_evict_without_weights_keeps_nothing():
    """weights_len 0: every context is clamped to 0."""
    c = Case([60, 40], 20, 0, 0, 2, 64, seed=13)
    c.weights, c.new_table = c.weights[:, :, :0], c.new_table[:, :0]
    lens, kept = c.run()
    assert int(c.fault) == f.FAULT_CONTEXT
    assert lens.tolist() == [0, 0] and bool((kept == -1).all())
    assert np.array_equal(c.cache.k_cache.cpu().numpy(), c.pools[0]) and np.array_equal(c.cache.v_scale.cpu().numpy(), c.scales[1])


def _counting(tokens, columns):
    """One sequence of one head over a pool of two blocks, which its whole table names in turn."""
    pool = torch.arange(16, dtype=torch.uint8, device="cuda")[None, None, :, None].expand(8, 1, 16, 64).contiguous()
    cache = f.BlockCache(pool.clone(), pool.clone(), torch.ones(8, 1, device="cuda"), torch.ones(8, 1, device="cuda"))
    table = (torch.arange(columns, device="cuda") % 2).to(torch.int32)[None]
    return cache, table, torch.tensor([tokens], dtype=torch.int32, device="cuda")


def _tokens(cache, block):
    """What the block's tokens hold (a kept value moves to a new scale)."""
    return (cache.k_cache[block, 0, :, 0].view(torch.float8_e4m3fn).float() * cache.k_scale[block, 0]).tolist()


def test_evict_the_largest_budget():
    """A budget without a limit, whose last entries' indices a step of all threads carries beyond 32 bits."""
    cache, table, ctx = _counting(40, 3)
    new = torch.tensor([[2, 3, 4]], dtype=torch.int32, device="cuda")
    lens, kept = f.kv_block_evict(cache, table, ctx, torch.zeros(1, 1, 48, device="cuda"), 2 ** 31 - 1, new)
    assert lens.tolist() == [40] and kept.shape[2] == 2 ** 31 - 1
    assert kept[0, 0, :40].tolist() == list(range(40))
    assert all(int(x.max()) == -1 == int(x.min()) for x in kept[0, 0, 40:].split(1 << 28))
    assert _tokens(cache, 2) == _tokens(cache, 0) == _tokens(cache, 3) and _tokens(cache, 4)[:8] == _tokens(cache, 0)[:8]


def test_evict_the_longest_context():
    """As many tokens as a table can name, most of them of equal weight."""
    columns = (1 << 27) - 64
    tokens = 16 * columns
    cache, table, ctx = _counting(tokens, columns)
    weights = torch.zeros(1, 1, tokens, device="cuda")
    weights[0, 0, [5, 2 ** 30 + 7, tokens - 1]] = torch.tensor([1.0, 3.0, 2.0], device="cuda")
    lens, kept = f.kv_block_evict(cache, table, ctx, weights, 16, torch.tensor([[2]], dtype=torch.int32, device="cuda"))
    assert lens.tolist() == [16] and kept[0, 0].tolist() == [*range(14), 2 ** 30 + 7, tokens - 1]
    assert _tokens(cache, 2) == [_tokens(cache, 0)[x % 16] for x in kept[0, 0].tolist()]


def test_evict_results_beside_its_input():
    """Lengths and weights right behind the input's in one allocation."""
    pool, sc = torch.zeros(9, 1, 16, 64, dtype=torch.uint8, device="cuda"), torch.ones(9, 1, device="cuda")
    lens, w = torch.tensor([40, 40, 0, 0], dtype=torch.int32, device="cuda"), torch.arange(2 * 48 + 2 * 20, device="cuda").float()
    tab = torch.tensor([[0, 1, 2], [1, 2, 0]], dtype=torch.int32, device="cuda")
    new = torch.tensor([[3, 4], [5, 6]], dtype=torch.int32, device="cuda")
    moved = w[96:].view(2, 1, 20)
    got, kept = f.kv_block_evict(f.BlockCache(pool, pool, sc, sc), tab, lens[:2], w[:96].view(2, 1, 48), 20, new, new_weights=moved, new_lens=lens[2:])
    assert lens.tolist() == [40, 40, 20, 20] and kept[1, 0].tolist() == list(range(20, 40))
    assert moved[1, 0].tolist() == list(range(48 + 20, 48 + 40))
    with pytest.raises(f.FkvError):
        f.kv_block_evict(f.BlockCache(pool, pool, sc, sc), tab, lens[:2], w[:96].view(2, 1, 48), 20, new, new_lens=lens[:2])
