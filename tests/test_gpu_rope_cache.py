"""kv_rope_cache and kv_block_cache on the GPU against the oracle: codes, scales and bf16 values
bit for bit (the rotation's float32 roundings are fixed, so nothing is left to tolerance)."""
import numpy as np
import pytest
import torch

from oracle import blockcache, e4m3, e5m2

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.detach().cpu().float().numpy().astype(np.float64)


def _round_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def _same(a, b):
    """Two bf16 tensors bit for bit (NaN included)."""
    return torch.equal(a.cpu().contiguous().view(torch.int16), b.cpu().contiguous().view(torch.int16))


def _fused(rng, n, hq, h, d, dev="cuda"):
    """q, k, v as slices of one projection's output."""
    w = _bf16(rng, n, (hq + 2 * h) * d, scale=2.0).to(dev)
    return (w[:, :hq * d].view(n, hq, d), w[:, hq * d:(hq + h) * d].view(n, h, d), w[:, (hq + h) * d:].view(n, h, d))


@pytest.mark.parametrize("pool", ["e4m3", "e5m2", "bf16"])
@pytest.mark.parametrize("n,hq,h,d,rot,interleaved,gran", [
    (1, 4, 1, 64, 64, False, 0), (7, 8, 2, 128, 128, False, 1), (33, 3, 3, 128, 96, True, 1), (5, 16, 1, 256, 64, False, 0),
    (9, 64, 8, 128, 16, True, 0), (21, 40, 8, 256, 256, True, 1), (2, 1, 1, 64, 32, False, 1), (600, 1, 1, 64, 48, False, 1),
])
def test_rope_cache_bit_exact(pool, n, hq, h, d, rot, interleaved, gran):
    rng = np.random.default_rng(n + d + rot)
    q, k, v = _fused(rng, n, hq, h, d)
    table = f.Rope.table(500, rot)
    pos = rng.integers(0, 500, n)
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
    got = f.kv_rope_cache(q, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), f.Rope(table, interleaved),
                          cache, None if bf else ks.cuda(), None if bf else vs.cuda(), gran=gran,
                          skip_layer_mask=[1] if bf else None, q_out=q_out, fault=fault)
    assert got is q_out and int(fault) == 0
    rows = table.cpu().numpy()[pos]
    live = slots >= 0
    ref = _round_bf16(blockcache.turn(_f64(q), rows, interleaved))
    assert _same(q_out[live], ref[live]) and bool((q_out[~torch.from_numpy(live)] == -7.0).all())
    codec = {"e4m3": e4m3, "e5m2": e5m2}.get(pool)
    for x, got, old, sc in ((blockcache.turn(_f64(k), rows, interleaved), cache.k_cache, before[0], ks),
                            (_f64(v), cache.v_cache, before[1], vs)):
        want = old.cpu()
        for t in np.flatnonzero(live):
            y = _round_bf16(x[t]) if bf else torch.from_numpy(codec.quantize(x[t], sc.numpy().reshape(-1, 1)))
            want[slots[t] // 16, :, slots[t] % 16] = y
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


def test_rope_cache_in_place_without_queries_and_faults():
    rng = np.random.default_rng(5)
    n, hq, h, d = 6, 4, 2, 128
    q, k, v = _fused(rng, n, hq, h, d)
    rope = f.Rope(f.Rope.table(50, 128))
    pos = torch.tensor([0, 49, 50, -1, 3, 7]).cuda()         # two outside the table
    slots = torch.tensor([5, 0, 9, 10, 16 * 3, 1]).cuda()    # slot 48 beyond 3 blocks
    s = torch.full((1,), 0.02, device="cuda")
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = f.LayerCache.empty(3, h, d)
    cache.k_cache.fill_(9), cache.v_cache.fill_(9)
    ref_q = q.clone()
    f.kv_rope_cache(q, k, v, pos, slots, rope, cache, s, s, q_out=q, fault=fault)
    assert int(fault) == f.FAULT_POSITION | f.FAULT_SLOT
    done = [0, 1, 5]
    turned = _round_bf16(blockcache.turn(_f64(ref_q), rope.cos_sin.cpu().numpy()[pos.clamp(0, 49).cpu()], False))
    for t in range(n):
        assert _same(q[t], turned[t] if t in done else ref_q[t])
    touched = torch.zeros(48, dtype=torch.bool)
    touched[[5, 0, 1]] = True
    left = cache.k_cache.transpose(1, 2).reshape(48, -1).cpu()[~touched]
    assert bool((left == 9).all())
    other = f.LayerCache.empty(3, h, d)
    other.k_cache.fill_(9), other.v_cache.fill_(9)
    assert f.kv_rope_cache(None, k, v, pos, slots, rope, other, s, s) is None
    assert torch.equal(other.k_cache, cache.k_cache) and torch.equal(other.v_cache, cache.v_cache)
    with pytest.raises(ValueError, match="not consecutive"):
        f.kv_rope_cache(None, k.flip(2).transpose(1, 2).contiguous().transpose(1, 2), v, pos, slots, rope, cache, s, s)
    with pytest.raises(f.FkvError):
        f.kv_rope_cache(None, k, v, pos, slots, f.Rope(torch.zeros(50, 24, device="cuda")), cache, s, s)


def test_rope_cache_non_finite_and_extreme_values():
    """Infinities saturate, NaN stays NaN, and a product that overflows float32 counts as infinite."""
    h, d = 1, 64
    k = torch.zeros(1, h, d, dtype=torch.bfloat16)
    k[0, 0, :6] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.38e38, -3.38e38, 1e-38])
    k[0, 0, 32:38] = torch.tensor([1.0, 2.0, 3.0, -3.38e38, 3.38e38, 0.0])
    rope = f.Rope(torch.tensor([[0.6] * 32 + [0.8] * 32], device="cuda"))
    s = torch.ones(1, device="cuda")
    for bf in (False, True):
        cache = f.LayerCache.empty(1, h, d, bf16=bf)
        one = torch.zeros(1, dtype=torch.int64, device="cuda")
        f.kv_rope_cache(None, k.cuda(), k.cuda(), one, one, rope, cache, s, s, skip_layer_mask=[1] if bf else None)
        with np.errstate(all="ignore"):
            y = blockcache.turn(_f64(k), rope.cos_sin.cpu().numpy(), False)
        if bf:
            got, ref = _f64(cache.k_cache[0, 0, 0]), _f64(_round_bf16(y[0, 0]))
        else:
            got, ref = e4m3.decode(cache.k_cache[0, 0, 0].cpu().numpy()), e4m3.decode(e4m3.quantize(y[0, 0], np.float32(1)))
        assert np.array_equal(got, ref, equal_nan=True)


# ------------------------------------------------------------------ kv_block_cache

def _paged(rng, ctx, extra=3):
    n = [(t + 15) // 16 for t in ctx]
    perm = rng.permutation(sum(n) + extra).astype(np.int32)
    table, at = np.full((len(ctx), max(1, *n)), -1, np.int32), 0
    for b, m in enumerate(n):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, sum(n) + extra


def _pools(rng, nb, h, d):
    c = f.BlockCache.empty(nb, h, d)
    for t in (c.k_cache, c.v_cache):
        t.copy_(torch.from_numpy(rng.integers(0, 256, t.shape).astype(np.uint8)))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.from_numpy((2.0 ** rng.integers(-9, 3, t.shape)).astype(np.float32)))
    return c


def _snapshot(c):
    return [t.cpu().numpy().copy() for t in (c.k_cache, c.v_cache, c.k_scale, c.v_scale)]


def _oracle_append(state, k, v, new, ctx, table, rows, interleaved):
    kp, vp, ks, vs = state
    at = 0
    for b, (m, t) in enumerate(zip(new, ctx)):
        x = _f64(k)[at:at + m]
        if rows is not None and m:
            x = blockcache.turn(x, rows[t - m:t], interleaved)
        blockcache.append(x, t - m, table[b], kp, ks)
        blockcache.append(_f64(v)[at:at + m], t - m, table[b], vp, vs)
        at += m
    return state


@pytest.mark.parametrize("new,ctx,hq,h,d,rot,interleaved", [
    ([1], [1], 4, 1, 64, 64, False), ([1, 1, 1], [16, 17, 300], 8, 2, 128, 128, False),
    ([0, 5, 31, 48], [9, 5, 40, 50], 6, 3, 128, 32, True), ([130, 1, 17], [143, 33, 17], 8, 1, 256, 256, True),
    ([15, 16, 2], [31, 47, 18], 0, 4, 64, 48, False), ([40], [71], 0, 2, 256, 0, False), ([3, 0, 700], [3, 0, 1000], 64, 8, 64, 64, True),
])
def test_block_cache_bit_exact(new, ctx, hq, h, d, rot, interleaved):
    rng = np.random.default_rng(sum(ctx) + d)
    n = sum(new)
    q, k, v = _fused(rng, n, hq, h, d) if hq else (None, *_fused(rng, n, 1, h, d)[1:])
    # tokens of differing size, so that scales grow in continued blocks
    size = torch.from_numpy((2.0 ** rng.integers(-8, 9, n)).astype(np.float32)).to(torch.bfloat16).cuda()
    k.mul_(size[:, None, None]), v.mul_(size.flip(0)[:, None, None])
    table, nb = _paged(rng, ctx)
    cache = _pools(rng, nb, h, d)
    before = _snapshot(cache)
    rope = f.Rope(f.Rope.table(1000, rot), interleaved) if rot else None
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device="cuda")
    out = f.kv_block_cache(k, v, cu, max(new), cache, torch.from_numpy(table).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                           rope=rope, q=q, fault=fault)
    assert int(fault) == 0
    rows = rope.cos_sin.cpu().numpy() if rope else None
    want = _oracle_append([x.copy() for x in before], k, v, new, ctx, table, rows, interleaved)
    for got, ref in zip(_snapshot(cache), want):
        assert np.array_equal(got, ref)
    if hq:
        pos = np.concatenate([np.arange(t - m, t) for m, t in zip(new, ctx)])
        assert _same(out, _round_bf16(blockcache.turn(_f64(q), rows[pos], interleaved)))


def test_block_cache_token_by_token_and_at_once():
    """Appending in pieces ends with the scales of appending at once; codes differ only where a
    growing scale pushed earlier codes below their subnormal step, by half of it per growth."""
    rng = np.random.default_rng(8)
    h, d, T = 2, 128, 37
    k, v = _bf16(rng, T, h, d).cuda(), _bf16(rng, T, h, d).cuda()
    k.mul_(torch.from_numpy((2.0 ** rng.integers(-4, 5, T)).astype(np.float32)).to(torch.bfloat16).cuda()[:, None, None])
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    once, steps = _pools(rng, 3, h, d), _pools(rng, 3, h, d)

    def put(cache, a, b):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        f.kv_block_cache(k[a:b], v[a:b], cu, b - a, cache, table, torch.tensor([b], dtype=torch.int32, device="cuda"))
    put(once, 0, T)
    for t in range(T):
        put(steps, t, t + 1)
    assert torch.equal(once.k_scale, steps.k_scale) and torch.equal(once.v_scale, steps.v_scale)
    for g in range(h):
        a, b = (blockcache.sequence(c.k_cache.cpu().numpy(), c.k_scale.cpu().numpy(), [2, 0, 1], T, g) for c in (once, steps))
        s = np.repeat(once.k_scale[[2, 0, 1], g].cpu().numpy(), 16)[:T, None]
        assert np.all(np.abs(a - b) <= 9 * s * 2.0 ** -9)


def test_block_cache_odd_old_scales_and_non_finite_tokens():
    """An old scale that is no normal positive number counts as 0; one that is no power of two
    still scales by one float32 ratio; infinities saturate and do not set the scale."""
    rng = np.random.default_rng(9)
    h, d = 1, 64
    for old in (float("nan"), float("inf"), -1.0, 0.0, 1e-40, 3.0, 0.7):
        cache = _pools(rng, 1, h, d)
        cache.k_scale.fill_(old), cache.v_scale.fill_(old)
        k = _bf16(rng, 2, h, d, scale=1000.0)
        k[0, 0, 0], k[0, 0, 1], k[1, 0, 2] = float("inf"), float("nan"), -float("inf")
        before = _snapshot(cache)
        f.kv_block_cache(k.cuda(), k.cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda(), 2, cache,
                         torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([9], dtype=torch.int32).cuda())
        want = _oracle_append(before, k, k, [2], [9], np.zeros((1, 1), int), None, False)
        for got, ref in zip(_snapshot(cache), want):
            assert np.array_equal(got, ref, equal_nan=True), old


def test_block_cache_faults_leave_the_pools():
    rng = np.random.default_rng(10)
    h, d = 2, 64
    k = _bf16(rng, 8, h, d).cuda()
    cache = _pools(rng, 4, h, d)
    before = _snapshot(cache)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.tensor([[1, 4], [0, 3]], dtype=torch.int32, device="cuda")
    for cu, ctx, tab, rope, bit in [
        (i32(0, 4, 8), i32(33, -1), table, None, f.FAULT_CONTEXT),           # beyond the table, negative
        (i32(0, 4, 8), i32(3, 2), table, None, f.FAULT_QLEN),                # more new tokens than context
        (i32(0, 5, 3), i32(2, 2), table, None, f.FAULT_QLEN),                # decreasing
        (i32(2, 9, 10), i32(9, 9), table, None, f.FAULT_QLEN),               # rows beyond the tokens
        (i32(0, 4, 8), i32(9, 9), table, f.Rope(f.Rope.table(8, 64)), f.FAULT_POSITION),
        (i32(0, 4, 4), i32(20, 0), table, None, f.FAULT_BLOCK_ID),           # block 4 of 4
        (i32(0, 4, 4), i32(20, 0), -table, None, f.FAULT_BLOCK_ID),
    ]:
        fault = torch.zeros(1, dtype=torch.int32, device="cuda")
        f.kv_block_cache(k, k, cu, 8 if bit != f.FAULT_QLEN else 6, cache, tab, ctx, rope=rope, fault=fault)
        assert int(fault) == bit
        for got, ref in zip(_snapshot(cache), before):
            assert np.array_equal(got, ref)


def test_writes_past_four_gigabytes():
    """Blocks whose bytes lie behind 2^32 in the pools."""
    rng = np.random.default_rng(11)
    h, d, nb = 8, 128, (1 << 32) // (8 * 16 * 128) + 5
    k, v = _bf16(rng, 20, h, d).cuda(), _bf16(rng, 20, h, d).cuda()
    ids = [nb - 1, nb - 3]
    big = f.BlockCache.empty(nb, h, d)
    small = f.BlockCache.empty(2, h, d)
    cu, ctx = torch.tensor([0, 20], dtype=torch.int32, device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda")
    for c, t in ((big, ids), (small, [1, 0])):
        f.kv_block_cache(k, v, cu, 20, c, torch.tensor([t], dtype=torch.int32, device="cuda"), ctx)
    for a, b in ((big.k_cache, small.k_cache), (big.v_cache, small.v_cache), (big.k_scale, small.k_scale)):
        assert torch.equal(a[ids[0]], b[1]) and (a.dim() == 2 and torch.equal(a[ids[1]], b[0]) or torch.equal(a[ids[1], :, :4], b[0, :, :4]))
    rope, s = f.Rope(f.Rope.table(32, 128)), torch.full((1,), 0.01, device="cuda")
    pos = torch.arange(20, device="cuda")
    lc, ls = f.LayerCache(big.k_cache, big.v_cache), f.LayerCache(small.k_cache, small.v_cache)
    f.kv_rope_cache(None, k, v, pos, torch.where(pos < 16, ids[0] * 16 + pos, ids[1] * 16 + pos - 16), rope, lc, s, s)
    f.kv_rope_cache(None, k, v, pos, torch.where(pos < 16, 16 + pos, pos - 16), rope, ls, s, s)
    assert torch.equal(big.k_cache[ids[0]], small.k_cache[1]) and torch.equal(big.v_cache[ids[1], :, :4], small.v_cache[0, :, :4])


def test_writes_follow_one_another():
    """Calls in a row, each of which reads what the one before wrote: queries turned in place, and a block that grows
    token by token, against the same calls with a wait after each."""
    rng = np.random.default_rng(12)
    n, h, d = 700, 4, 128
    rope = f.Rope(f.Rope.table(900, d))
    pos = torch.arange(n, device="cuda")
    k, q0 = _bf16(rng, n, h, d).cuda(), _bf16(rng, n, 2 * h, d).cuda()
    growing = _bf16(rng, 48, h, d).cuda() * torch.logspace(-3, 2, 48, device="cuda", dtype=torch.bfloat16)[:, None, None]
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    ctx = [torch.tensor([t + 1], dtype=torch.int32, device="cuda") for t in range(48)]
    results = []
    for wait in (True, False):
        q, cache, blocks = q0.clone(), f.LayerCache.empty(n // 16 + 1, h, d), f.BlockCache.empty(3, h, d)
        one = torch.ones(1, device="cuda")
        for t in range(48):
            f.kv_rope_cache(q, k, k, pos, pos, rope, cache, one, one, q_out=q)
            if wait:
                torch.cuda.synchronize()
            f.kv_block_cache(growing[t:t + 1], q[t:t + 1, :h], cu, 1, blocks, table, ctx[t], rope=rope)
            if wait:
                torch.cuda.synchronize()
        results.append((q, cache.k_cache.view(-1, h, 16, d)[:n // 16], blocks.k_cache, blocks.v_cache, blocks.k_scale, blocks.v_scale))
    for x, y in zip(*results):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_writes_captured_and_on_another_stream():
    rng = np.random.default_rng(12)
    h, hq, d = 2, 4, 128
    q, k, v = _fused(rng, 3, hq, h, d)
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda")
    cu, ctx = torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([1, 5, 9], dtype=torch.int32, device="cuda")
    rope = f.Rope(f.Rope.table(16, 128))
    want = _pools(rng, 3, h, d)
    got = f.BlockCache(*(t.clone() for t in (want.k_cache, want.v_cache, want.k_scale, want.v_scale)))
    ref = f.kv_block_cache(k, v, cu, 1, want, table, ctx, rope=rope, q=q)
    out = torch.empty_like(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        f.kv_block_cache(k, v, cu, 1, got, table, ctx, rope=rope, q=q, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert _same(out, ref) and torch.equal(got.k_cache, want.k_cache) and torch.equal(got.v_scale, want.v_scale)


def test_block_cache_continues_a_block_of_zero_or_subnormal_scale():
    """Tokens of a block whose scale is 0 (or below 2^-126) are worth code * scale before and after the block takes
    a larger scale, down to half of that scale's subnormal step 2^-9; in the oracle's bytes."""
    rng = np.random.default_rng(21)
    h, d = 2, 64
    for old in (0.0, 2.0 ** -130, 2.0 ** -149, 1.5 * 2.0 ** -128):
        for size in (1.0, 2.0 ** -123):
            cache = _pools(rng, 2, h, d)
            for p in (cache.k_cache, cache.v_cache):
                p.copy_(torch.where((p & 0x7F) == 0x7F, 0x7E, p))
            cache.k_scale.fill_(old), cache.v_scale.fill_(old)
            k = _bf16(rng, 3, h, d, scale=size)
            before = _snapshot(cache)
            f.kv_block_cache(k.cuda(), k.cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda(), 3, cache,
                             torch.ones(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([11], dtype=torch.int32).cuda())
            after = _snapshot(cache)
            for a, b, s0, s1 in ((before[0], after[0], before[2], after[2]), (before[1], after[1], before[3], after[3])):
                was, now = (e4m3.decode(x[1, :, :8]) * s[1].astype(np.float64)[:, None, None] for x, s in ((a, s0), (b, s1)))
                assert np.all(np.abs(now - was) <= 2.0 ** -4 * np.abs(was) + 2.0 ** -10 * s1[1].astype(np.float64)[:, None, None]), old
                assert np.array_equal(a[0], b[0]) and np.array_equal(a[1, :, 11:], b[1, :, 11:])
            want = _oracle_append(before, k, k, [3], [11], np.ones((1, 1), int), None, False)
            for got, ref in zip(after, want):
                assert np.array_equal(got, ref), old
