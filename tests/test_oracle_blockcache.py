"""Pins of the oracle's rotary embedding and block-scaled cache (CPU only)."""
import math

import numpy as np
import pytest
import torch

from oracle import blockcache, e4m3


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    ang = rng.uniform(-9, 9, (5, 16))
    y = blockcache.turn(x, np.concatenate((np.cos(ang), np.sin(ang)), 1), interleaved, f32=False)
    i = np.arange(16)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 16)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang)[:, None]
    assert np.allclose(y[..., a], z.real, atol=1e-14) and np.allclose(y[..., b], z.imag, atol=1e-14)
    assert np.array_equal(y[..., 32:], x[..., 32:])


def test_turn_in_float32_matches_elementwise_torch():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((7, 2, 32)).astype(np.float32)).to(torch.bfloat16).float()
    cs = torch.from_numpy(rng.uniform(-1, 1, (7, 32)).astype(np.float32))
    c, s = cs[:, None, :16], cs[:, None, 16:]
    ref = torch.cat((x[..., :16] * c - x[..., 16:] * s, x[..., 16:] * c + x[..., :16] * s), -1)
    assert np.array_equal(blockcache.turn(x.numpy(), cs.numpy(), False), ref.double().numpy())


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (np.nextafter(np.float32(448), np.float32(500)), 2.0), (1.0, 2.0 ** -8),
                                        (0.875, 2.0 ** -9), (0.0, 2.0 ** -126), (1e-40, 2.0 ** -126),
                                        (3.3895314e38, 2.0 ** 120)])
def test_scale_is_the_smallest_power_of_two(amax, scale):
    assert blockcache.scale_for([0.0, -float(amax), np.inf, np.nan]) == scale


def test_append_in_pieces_keeps_every_token_within_half_a_step():
    """Tokens whose size grows: earlier codes are brought to the block's growing scale.  Codes scaled
    by powers of two lose nothing but subnormals, so that every element stays within half a step of
    its own e4m3 grid plus one subnormal step of the block's final scale for each growth."""
    rng = np.random.default_rng(2)
    n, H, D = 40, 2, 8
    x = rng.standard_normal((n, H, D)) * (2.0 ** np.linspace(-6, 3, n))[:, None, None]
    x = x.astype(np.float32).astype(np.float64)
    pool = rng.integers(0, 256, (4, H, 16, D)).astype(np.uint8)
    scale = np.full((4, H), 77.0, np.float32)
    ids, at = [2, 0, 3], 0
    before = pool[1].copy()
    for m in (1, 1, 9, 0, 13, 2, 14):
        blockcache.append(x[at:at + m], at, ids, pool, scale)
        at += m
    assert at == n and np.array_equal(pool[1], before) and np.all(scale[1] == 77.0)
    for g in range(H):
        y = blockcache.sequence(pool, scale, ids, n, g)
        s = np.repeat(scale[ids, g].astype(np.float64), 16)[:n, None]
        assert np.all(np.abs(y - x[:, g]) <= 2.0 ** -4 * np.abs(x[:, g]) + 16 * s * 2.0 ** -10)
    # the last block holds tokens 32 .. 39: slots behind them keep their bytes
    assert np.all(np.log2(scale[ids]) % 1 == 0)


def test_append_fresh_block_forgets_and_continued_block_keeps():
    pool = np.zeros((1, 1, 16, 8), np.uint8)
    scale = np.full((1, 1), 1024.0, np.float32)
    blockcache.append(np.ones((3, 1, 8)), 0, [0], pool, scale)
    assert scale[0, 0] == 2.0 ** -8                       # 1 <= 448 * 2^-8
    blockcache.append(np.full((1, 1, 8), 0.01), 3, [0], pool, scale)
    assert scale[0, 0] == 2.0 ** -8                       # kept: smaller tokens do not shrink it
    blockcache.append(np.full((1, 1, 8), 100.0), 4, [0], pool, scale)
    assert scale[0, 0] == 2.0 ** -2
    assert np.all(e4m3.decode(pool[0, 0, :3]) * scale[0, 0] == 1.0)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0)])
def test_attend_is_torch_softmax(causal, window):
    rng = np.random.default_rng(3)
    H, G, D, ctx, new = 2, 2, 64, [37, 0, 16], [9, 0, 16]
    kp, vp = (rng.integers(0, 0x78, (8, H, 16, D)).astype(np.uint8) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-5, 0, (8, H)).astype(np.float32) for _ in range(2))
    table = np.array([[5, 1, 7], [-1, -1, -1], [2, -1, -1]])
    cu = np.concatenate(([0], np.cumsum(new)))
    q = rng.standard_normal((25, H * G, D)) * 0.1
    got = blockcache.attend(q, kp, vp, ks, vs, table, ctx, cu, causal=causal, window=window)
    for b in (0, 2):
        T, n = ctx[b], new[b]
        for h in range(H * G):
            K, V = (torch.from_numpy(blockcache.sequence(p, s, table[b], T, h // G)) for p, s in ((kp, ks), (vp, vs)))
            w = torch.from_numpy(q[cu[b]:cu[b + 1], h]) @ K.T / math.sqrt(D)
            pos, key = torch.arange(T - n, T)[:, None], torch.arange(T)
            if causal:
                w[key > pos] = -math.inf
            if window:
                w[key <= pos - window] = -math.inf
            assert np.allclose(got[cu[b]:cu[b + 1], h], (torch.softmax(w, 1) @ V).numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("old", [0.0, 2.0 ** -130, 2.0 ** -149, 1.5 * 2.0 ** -128])
def test_append_continues_a_block_of_zero_or_subnormal_scale(old):
    """A value is code * scale whatever the scale >= 0: kept tokens are worth what they were, down to half of the
    subnormal step 2^-9 of the block's new scale."""
    for x in (1.0, 2.0 ** -125):
        pool = np.full((1, 1, 16, 8), 0x7E, np.uint8)
        pool[0, 0, 1] = 0xB8
        scale = np.full((1, 1), old, np.float32)
        before = e4m3.decode(pool[0, 0, :3]) * float(scale[0, 0])
        blockcache.append(np.full((1, 1, 8), x), 3, [0], pool, scale)
        assert scale[0, 0] == blockcache.scale_for([x])
        after = e4m3.decode(pool[0, 0, :3]) * float(scale[0, 0])
        assert np.all(np.abs(after - before) <= 2.0 ** -4 * np.abs(before) + float(scale[0, 0]) * 2.0 ** -10)
