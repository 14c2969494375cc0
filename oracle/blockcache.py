"""The rotary position embedding and the block-scaled FP8 cache, in float64.

Rotation: pair i = (a, b) of a head's first rot_dim elements, elements i and i + rot_dim / 2 or
(interleaved) 2 i and 2 i + 1, becomes (a cos - b sin, b cos + a sin).  What is stored rounds the
products and the sum to float32 one by one; ``turn(..., f32=True)`` restates that, so that codes
compare exactly.

Block-scaled cache: e4m3 pools [num_blocks][H_kv][16][D] whose every (block, KV head) has one
power-of-two scale for K and one for V, found when tokens are appended.  Attention over it is
the plain softmax of the dequantised keys and values; nothing else is rounded.
"""
from __future__ import annotations

import math

import numpy as np

from . import e4m3
from .e4m3 import fl32


def turn(x, rows, interleaved, f32=True):
    """x float64 [n][heads][D] turned by the table rows [n][rot_dim] (float32 values)."""
    r = fl32 if f32 else (lambda y: y)
    x = np.array(x, np.float64)
    rows = np.asarray(rows, np.float64)
    half = rows.shape[1] // 2
    c, s = rows[:, None, :half], rows[:, None, half:]
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., ia], x[..., ib]
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., ia] = r(r(a * c) - r(b * s))
        y[..., ib] = r(r(b * c) + r(a * s))
    return y


def scale_for(values):
    """The smallest power of two s >= 2^-126 with the largest finite magnitude <= 448 s."""
    v = np.abs(np.asarray(values, np.float64))
    v = v[np.isfinite(v)]
    amax = float(v.max()) if v.size else 0.0
    k = -126
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def append(x, start, ids, pool, scale):
    """Append x [n][H][D] (values before quantisation) of one sequence whose first token has position
    ``start`` and whose page i is pool block ids[i]; pool uint8 [nb][H][16][D] and scale float32
    [nb][H] are changed in place."""
    n, H, _ = x.shape
    for page in range(start // 16, (start + n + 15) // 16 if n else 0):
        lo, hi = max(start, 16 * page), min(start + n, 16 * page + 16)
        kept, blk = lo - 16 * page, int(ids[page])
        for h in range(H):
            y = x[lo - start:hi - start, h]
            s = scale_for(y)
            if kept:
                old = float(scale[blk, h])
                if math.isfinite(old) and old >= 0.0:
                    if old >= s:
                        s = old
                    else:
                        codes = pool[blk, h, :kept]
                        codes[:] = e4m3.encode(fl32(e4m3.decode(codes) * fl32(old / s)))
            scale[blk, h] = s
            pool[blk, h, kept:hi - 16 * page] = e4m3.quantize(y, np.float32(s))


def sequence(pool, scale, ids, T, g):
    """Dequantised rows [T][D] of KV head g of a sequence."""
    ids = np.asarray(ids[:(T + 15) // 16], np.int64)
    rows = e4m3.decode(pool[ids, g]) * np.asarray(scale, np.float64)[ids, g][:, None, None]
    return rows.reshape(-1, pool.shape[3])[:T]


def attend(q, k_pool, v_pool, k_scale, v_scale, table, ctx, cu=None, softmax_scale=0.0, causal=True, window=0):
    """softmax(q K^T) V in float64, q [rows][Hq][D]; cu None: decode, row b of sequence b."""
    rows, Hq, D = q.shape
    H = k_pool.shape[1]
    tau = softmax_scale if softmax_scale > 0 else 1.0 / math.sqrt(D)
    out = np.zeros((rows, Hq, D))
    for b, T in enumerate(ctx):
        r0, r1 = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
        if T == 0 or r1 == r0:
            continue
        pos = np.arange(T - (r1 - r0), T)[:, None]
        key = np.arange(T)[None, :]
        seen = (key <= pos) if causal else np.ones((r1 - r0, T), bool)
        if window:
            seen &= key > pos - window
        for g in range(H):
            K = sequence(k_pool, k_scale, table[b], T, g)
            V = sequence(v_pool, v_scale, table[b], T, g)
            used = seen.any(0)
            K, V = np.where(used[:, None], K, 0.0), np.where(used[:, None], V, 0.0)
            for h in range(g * (Hq // H), (g + 1) * (Hq // H)):
                s = np.where(seen, (q[r0:r1, h] @ K.T) * tau, -np.inf)
                p = np.exp(s - s.max(1, keepdims=True))
                out[r0:r1, h] = (p @ V) / p.sum(1, keepdims=True)
    return out


def p_bound(q, k_pool, v_pool, k_scale, v_scale, table, ctx, cu=None, **kw):
    """sum_j p_j |v_j| / l per output element: what a relative error of each p scales."""
    return attend(q, k_pool, v_pool & 0x7F, k_scale, v_scale, table, ctx, cu, **kw)
