"""Rotary positions of several axes, and positions given to the block append, on the GPU against the oracle: codes,
scales and bf16 values bit for bit (the rotation's float32 roundings are fixed, so nothing is left to tolerance)."""
import numpy as np
import pytest
import torch

from oracle import blockcache, e4m3, e5m2

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu


def _bf16(rng, *shape, scale=2.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def _same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.int16), b.cpu().contiguous().view(torch.int16))


def _fused(rng, n, hq, h, d):
    w = _bf16(rng, n, (hq + 2 * h) * d).cuda()
    return (w[:, :hq * d].view(n, hq, d), w[:, hq * d:(hq + h) * d].view(n, h, d), w[:, (hq + h) * d:].view(n, h, d))


def _rows(table, pos, axes):
    """The oracle's table rows [n][rot]: pair i's entry at the position of its axis."""
    t, half = table.cpu().numpy(), len(axes)
    cols = np.arange(half)
    at = np.asarray(pos)[np.asarray(axes)].T                     # [n][half]
    return np.concatenate((t[at, cols], t[at, half + cols]), 1)


def _round_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def _axes(rng, rot, count, kind):
    half = rot // 2
    if kind == "runs":
        cut = np.sort(rng.choice(np.arange(1, half), count - 1, replace=False))
        return f.Rope.sections(*np.diff(np.concatenate(([0], cut, [half]))).tolist())
    if kind == "turns":
        return [i % count for i in range(half)]
    return rng.integers(0, count, half).tolist()


@pytest.mark.parametrize("pool", ["e4m3", "e5m2", "bf16"])
@pytest.mark.parametrize("n,hq,h,d,rot,interleaved,gran,count,kind", [
    (1, 4, 1, 64, 64, False, 0, 3, "runs"), (7, 8, 2, 128, 128, False, 1, 3, "turns"), (33, 3, 3, 128, 96, True, 1, 2, "any"),
    (5, 16, 1, 256, 64, False, 0, 4, "any"), (9, 64, 8, 128, 16, True, 0, 4, "turns"), (21, 40, 8, 256, 256, True, 1, 3, "runs"),
    (600, 1, 1, 64, 48, False, 1, 1, "any"), (3001, 4, 2, 64, 64, False, 1, 3, "turns"),
])
def test_rope_cache_axes_bit_exact(pool, n, hq, h, d, rot, interleaved, gran, count, kind):
    rng = np.random.default_rng(n + d + rot)
    q, k, v = _fused(rng, n, hq, h, d)
    table = f.Rope.table(500, rot)
    axes = _axes(rng, rot, count, kind)
    pos = rng.integers(0, 500, (count, n))
    nb = n // 16 + 4
    slots = rng.permutation(nb * 16)[:n]
    slots[n // 2] = -1 if n > 1 else slots[0]  # a padding token
    bf = pool == "bf16"
    cache = f.LayerCache(*(torch.from_numpy(rng.integers(0, 256, (nb, h, 16, d * (2 if bf else 1))).astype(np.uint8)).cuda()
                           for _ in range(2)), f.KV_E5M2 if pool == "e5m2" else f.KV_E4M3)
    if bf:
        cache.k_cache, cache.v_cache = cache.k_cache.view(torch.bfloat16), cache.v_cache.view(torch.bfloat16)
    before = cache.k_cache.clone(), cache.v_cache.clone()
    ks, vs = (torch.from_numpy(rng.uniform(0.003, 0.05, h if gran else 1).astype(np.float32)) for _ in range(2))
    q_out = torch.full((n, hq, d), -7.0, dtype=torch.bfloat16, device="cuda")
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.zeros(count, n + 5, dtype=torch.int64, device="cuda")      # rows of a wider tensor
    wide[:, 3:n + 3] = torch.from_numpy(pos)
    f.kv_rope_cache(q, k, v, wide[:, 3:n + 3], torch.from_numpy(slots).cuda(), f.Rope(table, interleaved, axes), cache,
                    None if bf else ks.cuda(), None if bf else vs.cuda(), gran=gran, skip_layer_mask=[1] if bf else None,
                    q_out=q_out, fault=fault)
    assert int(fault) == 0
    rows, live = _rows(table, pos, axes), slots >= 0
    ref = _round_bf16(blockcache.turn(_f64(q), rows, interleaved))
    assert _same(q_out[live], ref[live]) and bool((q_out[~torch.from_numpy(live)] == -7.0).all())
    codec = {"e4m3": e4m3, "e5m2": e5m2}.get(pool)
    for x, got, old, sc in ((blockcache.turn(_f64(k), rows, interleaved), cache.k_cache, before[0], ks),
                            (_f64(v), cache.v_cache, before[1], vs)):
        want = old.cpu()
        y = _round_bf16(x[live]) if bf else torch.from_numpy(codec.quantize(x[live], sc.numpy().reshape(-1, 1)))
        want[slots[live] // 16, :, slots[live] % 16] = y
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


def test_rope_cache_axes_positions_outside_the_table():
    """One axis outside is enough: the token is skipped whole and reported."""
    rng = np.random.default_rng(1)
    q, k, v = _fused(rng, 5, 2, 1, 64)
    pos = torch.tensor([[0, 49, 3, 3, 3], [1, 1, 50, 1, 1], [2, 2, 2, -1, 1 << 40]]).cuda()
    rope = f.Rope(f.Rope.table(50, 64), axes=f.Rope.sections(10, 12, 10))
    cache = f.LayerCache.empty(1, 1, 64)
    cache.k_cache.fill_(9), cache.v_cache.fill_(9)
    s, fault = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((5, 2, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    f.kv_rope_cache(q, k, v, pos, torch.arange(5).cuda(), rope, cache, s, s, q_out=out, fault=fault)
    assert int(fault) == f.FAULT_POSITION
    assert bool((out[2:] == -7.0).all()) and bool((out[:2] != -7.0).any())
    assert bool((cache.k_cache[0, 0, 2:] == 9).all()) and bool((cache.v_cache[0, 0, 2:] == 9).all())


class Appended:
    """Sequences of `ctx` tokens, the last `new` of them appended by the library and by the oracle."""

    def __init__(self, rng, ctx, new, h, d):
        n = [(t + 15) // 16 for t in ctx]
        self.nb = sum(n) + 2
        perm, at = rng.permutation(self.nb).astype(np.int32), 0
        self.table = np.full((len(ctx), max(1, *n)), -1, np.int32)
        for b, m in enumerate(n):
            self.table[b, :m] = perm[at:at + m]
            at += m
        self.ctx, self.new, self.cu = ctx, new, np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        self.pools = [(rng.integers(0, 255, (self.nb, h, 16, d)) & 0x7B).astype(np.uint8) for _ in range(2)]
        self.scales = [(2.0 ** rng.integers(-9, -3, (self.nb, h))).astype(np.float32) for _ in range(2)]

    def cache(self):
        return f.BlockCache(*(torch.from_numpy(p.copy()).cuda() for p in self.pools),
                            *(torch.from_numpy(s.copy()).cuda() for s in self.scales))

    def args(self):
        return torch.from_numpy(self.cu).cuda(), max(self.new), torch.from_numpy(self.table).cuda(), torch.tensor(self.ctx, dtype=torch.int32).cuda()

    def want(self, k, v):
        for x, pool, scale in ((k, self.pools[0], self.scales[0]), (v, self.pools[1], self.scales[1])):
            for b, (t, n) in enumerate(zip(self.ctx, self.new)):
                blockcache.append(x[self.cu[b]:self.cu[b + 1]], t - n, self.table[b], pool, scale)


@pytest.mark.parametrize("d,hq,h,rot,interleaved,count,kind", [
    (64, 4, 2, 64, False, 3, "runs"), (128, 8, 2, 128, False, 3, "turns"), (128, 6, 3, 96, True, 4, "any"), (256, 2, 1, 64, True, 2, "any"),
    (128, 2, 2, 128, False, 0, ""), (256, 4, 2, 256, False, 3, "runs"),
])
def test_block_cache_positions_bit_exact(d, hq, h, rot, interleaved, count, kind):
    rng = np.random.default_rng(d + rot + count)
    a = Appended(rng, [40, 1, 16, 700, 33, 5], [1, 1, 16, 123, 0, 4], h, d)
    n = int(a.cu[-1])
    q, k, v = _fused(rng, n, hq, h, d)
    table = f.Rope.table(100, rot)                       # shorter than the sequences: places do not count
    axes = _axes(rng, rot, count, kind) if count else None
    pos = rng.integers(0, 100, (max(count, 1), n))
    rows = _rows(table, pos, axes or [0] * (rot // 2))
    cache, (cu, mx, tab, ctx) = a.cache(), a.args()
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = torch.from_numpy(pos if count else pos[0]).cuda()
    out = f.kv_block_cache(k, v, cu, mx, cache, tab, ctx, rope=f.Rope(table, interleaved, axes), q=q, positions=p, fault=fault)
    assert int(fault) == 0
    assert _same(out, _round_bf16(blockcache.turn(_f64(q), rows, interleaved)))
    a.want(blockcache.turn(_f64(k), rows, interleaved), _f64(v))
    for got, want in zip((cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale), a.pools + a.scales):
        assert np.array_equal(got.cpu().numpy(), want)


def test_block_cache_positions_equal_places_and_are_clamped():
    rng = np.random.default_rng(7)
    a = Appended(rng, [50, 21], [30, 21], 2, 128)
    q, k, v = _fused(rng, 51, 4, 2, 128)
    rope = f.Rope(f.Rope.table(64, 128))
    cu, mx, tab, ctx = a.args()
    places = torch.cat((torch.arange(20, 50), torch.arange(21))).cuda()
    one, two = a.cache(), a.cache()
    x = f.kv_block_cache(k, v, cu, mx, one, tab, ctx, rope=rope, q=q)
    y = f.kv_block_cache(k, v, cu, mx, two, tab, ctx, rope=rope, q=q, positions=places)
    assert _same(x, y) and all(torch.equal(getattr(one, m), getattr(two, m)) for m in ("k_cache", "v_cache", "k_scale", "v_scale"))
    # outside the table: the nearer end, reported
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    far = places.clone()
    far[0], far[1] = -5, 1 << 40
    near = places.clone()
    near[0], near[1] = 0, 63
    x = f.kv_block_cache(k, v, cu, mx, a.cache(), tab, ctx, rope=rope, q=q, positions=far, fault=fault)
    y = f.kv_block_cache(k, v, cu, mx, a.cache(), tab, ctx, rope=rope, q=q, positions=near)
    assert int(fault) == f.FAULT_POSITION and _same(x, y)


def test_axes_captured_and_replayed_with_other_positions():
    rng = np.random.default_rng(3)
    a = Appended(rng, [100], [9], 1, 64)
    q, k, v = _fused(rng, 9, 2, 1, 64)
    rope = f.Rope(f.Rope.table(200, 64), axes=f.Rope.sections(12, 10, 10))
    cu, mx, tab, ctx = a.args()
    pos = torch.from_numpy(rng.integers(0, 200, (3, 9))).cuda()
    other = torch.from_numpy(rng.integers(0, 200, (3, 9))).cuda()
    cache, out = a.cache(), torch.empty_like(q.contiguous())
    f.kv_block_cache(k, v, cu, mx, cache, tab, ctx, rope=rope, q=q, q_out=out, positions=pos)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.kv_block_cache(k, v, cu, mx, cache, tab, ctx, rope=rope, q=q, q_out=out, positions=pos)
    pos.copy_(other)
    g.replay()
    assert _same(out, _round_bf16(blockcache.turn(_f64(q), _rows(rope.cos_sin, other.cpu().numpy(), rope.axes), False)))
