"""Attention weights of cached keys and eviction by them, in float64.

Weights: w[g, j] = decay * before[g, j] + sum over the chunk's queries and the heads of group g of the
softmax weight of key j; keys that came with the chunk have no before.
Eviction: per KV head the first ``sink`` and last ``recent`` tokens and the heaviest others, ``budget`` in all, in
their order; what is kept is stored as an append of its dequantised values to empty blocks.
"""
from __future__ import annotations

import math

import numpy as np

from . import blockcache, e4m3
from .e4m3 import fl32


def softmax_weights(q, k_pool, k_scale, table, ctx, cu, softmax_scale=0.0):
    """Per sequence [H][T]: what the keys receive from rows cu[b] .. cu[b + 1] - 1 of q [rows][Hq][D], the last tokens of
    each sequence."""
    Hq, D = q.shape[1:]
    H = k_pool.shape[1]
    tau = softmax_scale if softmax_scale > 0 else 1.0 / math.sqrt(D)
    out = []
    for b, T in enumerate(ctx):
        w = np.zeros((H, T))
        rows = q[cu[b]:cu[b + 1]]
        n = rows.shape[0]
        if n and T:
            seen = np.arange(T)[None, :] <= np.arange(T - n, T)[:, None]
            for g in range(H):
                K = blockcache.sequence(k_pool, k_scale, table[b], T, g)
                for h in range(g * (Hq // H), (g + 1) * (Hq // H)):
                    s = np.where(seen, rows[:, h] @ K.T * tau, -np.inf)
                    p = np.exp(s - s.max(1, keepdims=True))
                    w[g] += (p / p.sum(1, keepdims=True)).sum(0)
        out.append(w)
    return out


def accumulate(before, new, n, decay):
    """before float [H][>= T] with the weights `new` [H][T] of a chunk of n tokens taken in."""
    out = np.array(before, np.float64)
    T = new.shape[1]
    old = T - n
    out[:, :T] = new
    if decay != 0.0:
        out[:, :old] += decay * np.asarray(before, np.float64)[:, :old]
    return out


def kept_tokens(weights, T, budget, sink, recent):
    """Ascending indices of the tokens of one KV head that stay; weights [>= T] float32."""
    if T <= budget:
        return np.arange(T)
    def before(i):                      # the order in which tokens are taken
        sure = i < sink or i >= T - recent
        w = float(weights[i])
        return (0 if sure else 1, 0.0 if sure else (math.inf if w != w else -w), 0 if sure else (1 if w != w else 0), i)
    return np.array(sorted(sorted(range(T), key=before)[:budget]))


def evict(pools, scales, table, ctx, weights, budget, new_table, sink, recent):
    """kept [B][H][budget] and new lengths; pools and scales (K, V) are changed in place in new_table's blocks."""
    B, H = len(ctx), pools[0].shape[1]
    kept = np.full((B, H, budget), -1, np.int32)
    source = [(p.copy(), s.copy()) for p, s in zip(pools, scales)]
    lens = np.array([min(t, budget) for t in ctx], np.int32)
    for b, T in enumerate(ctx):
        for h in range(H):
            ids = kept_tokens(weights[b, h], T, budget, sink, recent)
            kept[b, h, :ids.size] = ids
            for (old, old_scale), pool, scale in zip(source, pools, scales):
                blk = np.asarray(table[b])[ids // 16]
                with np.errstate(invalid="ignore", over="ignore"):
                    x = fl32(e4m3.decode(old[blk, h, ids % 16]) * old_scale[blk, h].astype(np.float64)[:, None])
                for page in range((ids.size + 15) // 16):
                    y = x[16 * page:16 * page + 16]
                    s = blockcache.scale_for(y)
                    dst = new_table[b][page]
                    scale[dst, h] = s
                    pool[dst, h, :y.shape[0]] = e4m3.quantize(y, np.float32(s))
    return kept, lens
