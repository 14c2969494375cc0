"""The oracle of attention weights and eviction, pinned by hand-worked cases and by plain loops."""
import math

import numpy as np
import pytest

from oracle import blockcache, e4m3, longcontext


def _cache(rng, nb, h, d):
    pool = rng.integers(0, 127, (nb, h, 16, d)).astype(np.uint8)
    return pool & 0x5F, (2.0 ** rng.integers(-9, -5, (nb, h))).astype(np.float32)


def test_weights_of_one_query_by_loops_and_sums():
    rng = np.random.default_rng(0)
    pool, scale = _cache(rng, 4, 2, 64)
    q = rng.standard_normal((3, 4, 64))
    table, ctx, cu = [[2, 0], [1, 3]], [20, 17], [0, 1, 3]
    got = longcontext.softmax_weights(q, pool, scale, table, ctx, cu)
    for b in range(2):
        n = cu[b + 1] - cu[b]
        assert np.allclose(got[b].sum(1), 2 * n)                      # two heads per group, each row sums to one
        for g in range(2):
            want = [0.0] * ctx[b]
            for r in range(cu[b], cu[b + 1]):
                last = ctx[b] - n + (r - cu[b])
                for h in (2 * g, 2 * g + 1):
                    s = []
                    for j in range(last + 1):
                        blk = table[b][j // 16]
                        k = e4m3.decode(pool[blk, g, j % 16]) * float(scale[blk, g])
                        s.append(sum(a * c for a, c in zip(q[r, h], k)) / 8)
                    m = max(s)
                    z = sum(math.exp(x - m) for x in s)
                    for j, x in enumerate(s):
                        want[j] += math.exp(x - m) / z
            assert np.allclose(got[b][g], want, rtol=1e-10, atol=1e-14)


def test_weights_times_values_are_the_attention():
    rng = np.random.default_rng(1)
    pool, scale = _cache(rng, 3, 1, 64)
    vals, vs = _cache(rng, 3, 1, 64)
    q = rng.standard_normal((1, 1, 64))
    w = longcontext.softmax_weights(q, pool, scale, [[1, 2, 0]], [41], [0, 1])[0][0]
    o = blockcache.attend(q, pool, vals, scale, vs, [[1, 2, 0]], [41])
    assert np.allclose(w @ blockcache.sequence(vals, vs, [1, 2, 0], 41, 0), o[0, 0])


def test_accumulate():
    before = np.array([[1.0, 2.0, 4.0, np.nan, 7.0]])
    new = np.array([[0.5, 0.25, 0.125, 0.0625]])
    assert np.array_equal(longcontext.accumulate(before, new, 1, 0.5)[0], [1.0, 1.25, 2.125, 0.0625, 7.0])
    assert np.array_equal(longcontext.accumulate(before * np.nan, new, 2, 0.0)[0, :4], new[0])


@pytest.mark.parametrize("w,T,budget,sink,recent,want", [
    ([5, 1, 9, 3], 4, 2, 0, 0, [0, 2]), ([5, 5, 5, 5], 4, 2, 0, 0, [0, 1]), ([5, 5, 5, 5], 4, 2, 0, 1, [0, 3]),
    ([0, 0, 9, 0], 4, 1, 1, 0, [0]), ([1, 2, 3], 3, 3, 0, 0, [0, 1, 2]), ([1, 2, 3, 9], 3, 5, 0, 0, [0, 1, 2]),
    ([math.nan, -math.inf, 1, 0], 4, 3, 0, 0, [1, 2, 3]), ([math.nan, 2, math.nan, 1], 4, 3, 0, 0, [0, 1, 3]),
    ([math.inf, 3, 3, -0.0, 0.0], 5, 4, 0, 0, [0, 1, 2, 3]), ([0, 0, 7, 0, 0, 0], 6, 4, 1, 2, [0, 2, 4, 5]),
])
def test_kept_tokens(w, T, budget, sink, recent, want):
    assert longcontext.kept_tokens(np.array(w, np.float32), T, budget, sink, recent).tolist() == want


def test_evict_keeps_values_and_finds_scales():
    """A block whose kept tokens are small takes a smaller scale, and every kept value that is not below its subnormal
    step is what it was."""
    rng = np.random.default_rng(2)
    pools, scales = zip(*(_cache(rng, 8, 2, 64) for _ in range(2)))
    pools, scales = list(pools), list(scales)
    before = [blockcache.sequence(p, s, [3, 1, 5], 40, g) for p, s in zip(pools, scales) for g in range(2)]
    w = rng.random((1, 2, 48)).astype(np.float32)
    kept, lens = longcontext.evict(pools, scales, [[3, 1, 5]], [40], w, 20, [[0, 2]], 2, 3)
    assert lens.tolist() == [20] and kept.shape == (1, 2, 20)
    for g in range(2):
        ids = kept[0, g]
        assert ids[:2].tolist() == [0, 1] and ids[-3:].tolist() == [37, 38, 39] and np.all(np.diff(ids) > 0)
        for kind in range(2):
            now = blockcache.sequence(pools[kind], scales[kind], [0, 2], 20, g)
            was = before[2 * kind + g][ids]
            step = np.repeat(scales[kind][[0, 2], g].astype(float), 16)[:20, None] * 2.0 ** -9
            assert np.all(np.abs(now - was) <= step / 2)
            top = [np.abs(was[:16]).max(), np.abs(was[16:]).max()]
            assert all(m <= 448 * s and m > 224 * s for m, s in zip(top, scales[kind][[0, 2], g]))
