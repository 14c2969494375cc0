"""Long prompts kept in a budget, as a program runs it: prompts appended at positions of three axes, attended, their keys
weighed and thinned out, tokens decoded behind them at their own positions while the weights go on, eager and as a
replayed graph on another stream, and many answers sampled from one thinned prompt.  After every stage the pools are the
oracle's bit for bit, and outputs within the tolerances of the operators' own tests:
attention (2^-8 + 2^-10) sum_j p_j |v_j| + 2^-10 max |v| + 2^-8 |o|, weights within 2^-16 in relative L2 distance."""
import numpy as np
import pytest
import torch

from helpers import rel_l2
from oracle import blockcache, longcontext

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu

HQ, H, D, ROWS = 8, 2, 128, 9000


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


class Session:
    """The pools on the GPU and as the oracle has them, and blocks handed out in a shuffled order."""

    def __init__(self, rng, num_blocks, pairs):
        self.rng, self.free = rng, list(rng.permutation(num_blocks))
        self.pools = [(rng.integers(0, 256, (num_blocks, H, 16, D)) & 0x7B).astype(np.uint8) for _ in range(2)]
        self.scales = [np.ones((num_blocks, H), np.float32) for _ in range(2)]
        self.cache = f.BlockCache(*(torch.from_numpy(p.copy()).cuda() for p in self.pools), *(torch.from_numpy(s.copy()).cuda() for s in self.scales))
        self.rope = f.Rope(f.Rope.table(ROWS, D), axes=f.Rope.sections(*pairs))

    def table(self, lens, width):
        t = np.full((len(lens), width), -1, np.int32)
        for b, n in enumerate(lens):
            for i in range((n + 15) // 16):
                t[b, i] = self.free.pop()
        return t

    def append(self, q, k, v, cu, table, ctx, positions):
        """The oracle's append; the turned queries, rounded as the library rounds them."""
        rows = self.rope.cos_sin.cpu().numpy()
        half = D // 2
        axes = np.asarray([int(a) for a in self.rope.axes])
        at = positions[axes]                                # [half][n]: the table row of each pair
        pairs = np.arange(half)[:, None]
        turned = np.concatenate((rows[at, pairs], rows[at, pairs + half])).T
        k64, v64 = blockcache.turn(_f64(k), turned, False), _f64(v)
        for b, t in enumerate(ctx):
            lo, hi = cu[b], cu[b + 1]
            for x, pool, scale in ((k64, self.pools[0], self.scales[0]), (v64, self.pools[1], self.scales[1])):
                blockcache.append(x[lo:hi], t - (hi - lo), table[b], pool, scale)
        return torch.from_numpy(blockcache.turn(_f64(q), turned, False).astype(np.float32)).to(torch.bfloat16)

    def same(self):
        c = self.cache
        for got, want in zip((c.k_cache, c.v_cache, c.k_scale, c.v_scale), self.pools + self.scales):
            assert np.array_equal(got.cpu().numpy(), want)

    def attended(self, got, q, table, ctx, cu=None):
        a = (_f64(q), self.pools[0], self.pools[1], self.scales[0], self.scales[1], table, ctx, cu)
        o, mag = blockcache.attend(*a), blockcache.p_bound(*a)
        top = np.zeros((o.shape[0], 1, 1))
        for b, t in enumerate(ctx):
            lo, hi = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
            top[lo:hi] = max(np.abs(blockcache.sequence(self.pools[1], self.scales[1], table[b], t, g)).max() for g in range(H))
        assert np.all(np.abs(_f64(got) - o) <= (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -10 * top + 2.0 ** -8 * np.abs(o))

    def weighed(self, got, before, q, table, ctx, cu, decay):
        new = longcontext.softmax_weights(_f64(q), self.pools[0], self.scales[0], table, ctx, cu)
        for b, t in enumerate(ctx):
            want = longcontext.accumulate(before[b], new[b], cu[b + 1] - cu[b], decay)[:, :t]
            assert rel_l2(got[b, :, :t].cpu().numpy().astype(np.float64), want) <= 2.0 ** -16


def test_long_prompts_in_a_budget():
    rng = np.random.default_rng(1)
    s = Session(rng, 800, (24, 20, 20))
    lens, budget, room = [2600, 77, 330], 2048, 2048 + 64
    table, cu = s.table(lens, 170), np.concatenate(([0], np.cumsum(lens)))
    n = int(cu[-1])
    q, k, v = _bf16(rng, n, HQ, D), _bf16(rng, n, H, D), _bf16(rng, n, H, D)
    # text moves all axes alike, an image's patches stand in rows and columns: positions fall behind the places
    positions = np.stack([np.concatenate([np.minimum(np.arange(t), 40 + np.arange(t) // (1 + a)) for t in lens]) for a in range(3)])
    d_table, d_ctx, d_cu, fault = _i32(table), _i32(lens), _i32(cu), _i32([0])
    turned = f.kv_block_cache(k, v, d_cu, max(lens), s.cache, d_table, d_ctx, rope=s.rope, q=q,
                              positions=torch.from_numpy(positions).cuda(), fault=fault)
    want = s.append(q, k, v, cu, table, lens, positions)
    assert torch.equal(turned.cpu(), want)
    s.same()
    out = f.fp8_block_prefill_attn(turned, d_cu, max(lens), s.cache, d_table, d_ctx, fault=fault)
    few = [0, 40, 77, 107]                   # of each prompt's rows the oracle takes the last ones
    rows = np.concatenate([np.arange(cu[b + 1] - (few[b + 1] - few[b]), cu[b + 1]) for b in range(3)])
    s.attended(out[rows], turned[rows], table, lens, few)
    # the weights of the prompts' last queries, into a buffer that holds anything
    last = turned[rows].contiguous()
    weights = torch.full((3, H, 170 * 16), 7.0, device="cuda")
    f.fp8_block_attn_weights(last, _i32(few), 40, s.cache, d_table, d_ctx, weights, decay=0.0, fault=fault)
    s.weighed(weights, np.zeros((3, H, 170 * 16)), last, table, lens, few, 0.0)
    # thinned out to the budget: sinks, recent tokens, the heaviest others
    kept_lens = [min(t, budget) for t in lens]
    new_table = s.table([t + 64 for t in kept_lens], room // 16)
    moved = torch.zeros(3, H, room, device="cuda")
    new_lens, kept = f.kv_block_evict(s.cache, d_table, d_ctx, weights, budget, _i32(new_table), sink=4, recent=64, new_weights=moved, fault=fault)
    want_kept, want_lens = longcontext.evict(s.pools, s.scales, table, lens, weights.cpu().numpy(), budget, new_table, 4, 64)
    assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(new_lens.cpu().numpy(), want_lens)
    s.same()
    # decoding behind what is left, at the tokens' own positions
    b3 = _i32([0, 1, 2, 3])
    d_table = _i32(new_table)
    ws, wws = f.block_decode_workspace(3, HQ, s.cache), f.attn_weights_workspace(3, 3, 1, HQ, s.cache, room // 16)
    place = torch.from_numpy(np.stack([[int(positions[a, cu[b + 1] - 1]) for b in range(3)] for a in range(3)])).cuda()
    q1, k1, v1 = _bf16(rng, 3, HQ, D), _bf16(rng, 3, H, D), _bf16(rng, 3, H, D)
    turned1, out1 = torch.empty_like(q1), torch.empty_like(q1)

    def step():
        new_lens.add_(1)
        place.add_(1)
        f.kv_block_cache(k1, v1, b3, 1, s.cache, d_table, new_lens, rope=s.rope, q=q1, q_out=turned1, positions=place, fault=fault)
        f.fp8_block_decode_attn(turned1, s.cache, d_table, new_lens, out=out1, workspace=ws, fault=fault)
        f.fp8_block_attn_weights(turned1, b3, 1, s.cache, d_table, new_lens, moved, decay=1.0, workspace=wws, fault=fault)

    def run(do, ctx):
        before = moved.cpu().numpy()
        for x in (q1, k1, v1):
            x.copy_(_bf16(rng, *x.shape))
        torch.cuda.synchronize()
        do()
        torch.cuda.synchronize()
        want = s.append(q1, k1, v1, [0, 1, 2, 3], new_table, ctx, place.cpu().numpy())
        assert torch.equal(turned1.cpu(), want) and int(fault) == 0
        s.same()
        s.attended(out1, turned1, new_table, ctx)
        s.weighed(moved, before, turned1, new_table, ctx, [0, 1, 2, 3], 1.0)
    ctx = list(want_lens)
    for _ in range(3):
        ctx = [t + 1 for t in ctx]
        run(step, ctx)
    side = torch.cuda.Stream()
    keep = [x.clone() for x in (new_lens, place, moved, *(getattr(s.cache, m) for m in ("k_cache", "v_cache", "k_scale", "v_scale")))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for x, y in zip((new_lens, place, moved, *(getattr(s.cache, m) for m in ("k_cache", "v_cache", "k_scale", "v_scale"))), keep):
        assert torch.equal(x, y), "capturing runs nothing"

    def replay():
        with torch.cuda.stream(side):
            graph.replay()
    for _ in range(14):                      # over a block's border
        ctx = [t + 1 for t in ctx]
        run(replay, ctx)
    # a second eviction, by weights that the decoding has added to, within what is left
    third = s.table([500] * 3, 512 // 16)
    again = torch.zeros(3, H, 512, device="cuda")
    lens2, kept2 = f.kv_block_evict(s.cache, d_table, new_lens, moved, 500, _i32(third), sink=4, recent=20, new_weights=again, fault=fault)
    want_kept, want_lens = longcontext.evict(s.pools, s.scales, new_table, ctx, moved.cpu().numpy(), 500, third, 4, 20)
    assert np.array_equal(kept2.cpu().numpy(), want_kept) and np.array_equal(lens2.cpu().numpy(), want_lens)
    s.same()
    assert int(fault) == 0


def test_many_answers_from_one_thinned_prompt():
    rng = np.random.default_rng(2)
    s = Session(rng, 700, (22, 22, 20))
    n, budget, answers = 2500, 2040, 100        # (2,040 x 99 tokens of 512 bytes saved: the decode shares them)
    table = s.table([n], 157)
    q, k, v = _bf16(rng, n, HQ, D), _bf16(rng, n, H, D), _bf16(rng, n, H, D)
    positions = np.stack([np.arange(n), np.arange(n) // 2, np.arange(n) // 3])
    fault = _i32([0])
    turned = f.kv_block_cache(k, v, _i32([0, n]), n, s.cache, _i32(table), _i32([n]), rope=s.rope, q=q, positions=torch.from_numpy(positions).cuda(),
                              fault=fault)
    s.append(q, k, v, [0, n], table, [n], positions)
    weights = torch.zeros(1, H, 157 * 16, device="cuda")
    f.fp8_block_attn_weights(turned[-32:].contiguous(), _i32([0, 32]), 32, s.cache, _i32(table), _i32([n]), weights, decay=0.0, fault=fault)
    kept_table = s.table([budget], 128)
    f.kv_block_evict(s.cache, _i32(table), _i32([n]), weights, budget, _i32(kept_table), sink=4, recent=128, fault=fault)
    longcontext.evict(s.pools, s.scales, table, [n], weights.cpu().numpy(), budget, kept_table, 4, 128)
    s.same()
    # the whole blocks are everyone's, the last, half-full one is copied for each
    full = budget // 16
    forks = np.full((answers, full + 3), -1, np.int32)
    forks[:, :full] = kept_table[0, :full]
    for b in range(answers):
        forks[b, full] = s.free.pop()
        forks[b, full + 1] = s.free.pop()
    src, dst = int(kept_table[0, full]), torch.from_numpy(forks[:, full].astype(np.int64)).cuda()
    for x, y in zip((s.cache.k_cache, s.cache.v_cache, s.cache.k_scale, s.cache.v_scale), s.pools + s.scales):
        x[dst] = x[src].clone()
        y[forks[:, full]] = y[src]
    ctx, place = [budget] * answers, torch.from_numpy(np.repeat(positions[:, -1:], answers, 1)).cuda()
    cu = np.arange(answers + 1)
    # (an append requantises the block that it goes on in, each answer's its own way: the whole blocks are what is shared)
    starts, shared, d_forks = _i32([0, answers]), _i32([full * 16]), _i32(forks)
    ws = f.block_shared_workspace(answers, HQ, s.cache, 1)
    for i in range(10):                          # each answer its own tokens, over a block's border
        ctx = [t + 1 for t in ctx]
        place.add_(1)
        q1, k1, v1 = _bf16(rng, answers, HQ, D), _bf16(rng, answers, H, D), _bf16(rng, answers, H, D)
        turned1 = f.kv_block_cache(k1, v1, _i32(cu), 1, s.cache, d_forks, _i32(ctx), rope=s.rope, q=q1, positions=place, fault=fault)
        want = s.append(q1, k1, v1, cu, forks, ctx, place.cpu().numpy())
        assert torch.equal(turned1.cpu(), want)
        out = f.fp8_block_shared_decode_attn(turned1, s.cache, d_forks, _i32(ctx), starts, shared, workspace=ws, fault=fault)
        if i in (0, 9):
            s.same()
            s.attended(out, turned1, forks, ctx)
    assert int(fault) == 0
    alone = f.fp8_block_decode_attn(turned1, s.cache, d_forks, _i32(ctx), fault=fault)
    s.attended(alone, turned1, forks, ctx)
    assert not torch.equal(out, alone), "the shared part is attended by itself"


def test_calls_right_behind_one_another():
    """Kernels start while those before them end: the calls of a program, each fed by the one before, give the bits that they give
    with the GPU idle in between."""
    rng = np.random.default_rng(3)
    lens, members, budget = [3000, 700, 1500], 100, 2000
    blocks = [(t + 15) // 16 for t in lens]
    nb = sum(blocks) + (members + 2) * 4 + 3 * 125
    ids = rng.permutation(nb).astype(np.int32)
    table = np.full((3, max(blocks)), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = ids[at:at + n]
        at += n
    new_table = ids[at:at + 3 * 125].reshape(3, 125)
    at += 3 * 125
    forks = np.full((members, 125 + 2), -1, np.int32)     # 100 sequences behind what the first one keeps, two blocks each of their own
    forks[:, :125] = new_table[0]
    forks[:, 125:] = ids[at:at + 2 * members].reshape(members, 2)
    n = sum(lens)
    cu = np.concatenate(([0], np.cumsum(lens)))
    pools = [torch.from_numpy((rng.integers(0, 256, (nb, H, 16, D)) & 0x7B).astype(np.uint8)).cuda() for _ in range(2)]
    scales = [torch.full((nb, H), 2.0 ** -9, device="cuda") for _ in range(2)]
    q, k, v = _bf16(rng, n, HQ, D), _bf16(rng, n, H, D), _bf16(rng, n, H, D)
    q1, k1, v1 = _bf16(rng, members, HQ, D), _bf16(rng, members, H, D), _bf16(rng, members, H, D)
    rope = f.Rope(f.Rope.table(ROWS, D), axes=f.Rope.sections(24, 20, 20))
    pos, pos1 = (torch.from_numpy(rng.integers(0, ROWS, (3, m))).cuda() for m in (n, members))
    d = dict(cu=_i32(cu), table=_i32(table), lens=_i32(lens), new_table=_i32(new_table), forks=_i32(forks), starts=_i32([0, members]),
             shared=_i32([budget]), cu1=_i32(np.arange(members + 1)))
    last = torch.cat([torch.arange(e - 40, e) for e in cu[1:]]).cuda()

    def run(wait):
        cache = f.BlockCache(*(x.clone() for x in pools + scales))
        weights, moved = (torch.zeros(3, H, m * 16, device="cuda") for m in (table.shape[1], 125))
        per_fork = torch.zeros(members, H, 127 * 16, device="cuda")
        fault = _i32([0])
        ws = (f.block_shared_workspace(members, HQ, cache, 1), f.attn_weights_workspace(3, 120, 40, HQ, cache, table.shape[1]),
              f.block_decode_workspace(members, HQ, cache), f.attn_weights_workspace(members, members, 1, HQ, cache, forks.shape[1]))
        turned1, out1, out2 = (torch.empty_like(q1) for _ in range(3))
        fork_lens = torch.full((members,), budget, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        turned = f.kv_block_cache(k, v, d["cu"], max(lens), cache, d["table"], d["lens"], rope=rope, q=q, positions=pos, fault=fault)
        wait()
        out = f.fp8_block_prefill_attn(turned, d["cu"], max(lens), cache, d["table"], d["lens"], fault=fault)
        wait()
        f.fp8_block_attn_weights(turned, d["cu"], max(lens), cache, d["table"], d["lens"], weights, decay=0.0, fault=fault)
        wait()
        f.fp8_block_attn_weights(turned[last], _i32([0, 40, 80, 120]), 40, cache, d["table"], d["lens"], weights, decay=0.5, workspace=ws[1], fault=fault)
        wait()
        new_lens, kept = f.kv_block_evict(cache, d["table"], d["lens"], weights, budget, d["new_table"], sink=4, recent=64, new_weights=moved, fault=fault)
        wait()
        for _ in range(3):
            fork_lens += 1
            f.kv_block_cache(k1, v1, d["cu1"], 1, cache, d["forks"], fork_lens, rope=rope, q=q1, q_out=turned1, positions=pos1, fault=fault)
            wait()
            f.fp8_block_shared_decode_attn(turned1, cache, d["forks"], fork_lens, d["starts"], d["shared"], out=out1, workspace=ws[0], fault=fault)
            wait()
            f.fp8_block_attn_weights(out1, d["cu1"], 1, cache, d["forks"], fork_lens, per_fork, workspace=ws[3], fault=fault)
            wait()
            f.fp8_block_decode_attn(out1, cache, d["forks"], fork_lens, out=out2, workspace=ws[2], fault=fault)
            wait()
            f.fp8_block_shared_decode_attn(out2, cache, d["forks"], fork_lens, d["starts"], d["shared"], out=out1, workspace=ws[0], fault=fault)
            wait()
        torch.cuda.synchronize()
        assert int(fault) == 0
        return [out, weights, moved, new_lens, kept, out1, out2, per_fork, cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale]
    want = run(torch.cuda.synchronize)
    assert all(bool(x.float().isfinite().all()) for x in want[:8])
    for _ in range(8):
        for x, y in zip(run(lambda: None), want):
            assert torch.equal(x, y)


def test_blocks_behind_four_gigabytes():
    """The same contents in a small pool and at the end of one of 4.5 GB: the same bits of every call."""
    rng = np.random.default_rng(4)
    lens, budget, nb, far = [2300, 40, 700], 600, 400, 1_100_000
    ids, at = rng.permutation(nb).astype(np.int32), 0
    table, new_table = np.full((3, 150), -1, np.int32), np.full((3, 40), -1, np.int32)
    for b, t in enumerate(lens):
        n, m = (t + 15) // 16, (min(t, budget) + 15) // 16
        table[b, :n], new_table[b, :m] = ids[at:at + n], ids[at + n:at + n + m]
        at += n + m
    members = 90                              # of one group behind the first sequence's first 2,288 tokens
    forks = np.tile(table[0, :144], (members, 1))
    n, cu = sum(lens), np.concatenate(([0], np.cumsum(lens)))
    pools = [torch.from_numpy((rng.integers(0, 256, (nb, H, 16, D)) & 0x7B).astype(np.uint8)).cuda() for _ in range(2)]
    q, k, v, q1 = _bf16(rng, n, HQ, D), _bf16(rng, n, H, D), _bf16(rng, n, H, D), _bf16(rng, members, HQ, D)
    rope = f.Rope(f.Rope.table(ROWS, D), axes=f.Rope.sections(24, 20, 20))
    pos = torch.from_numpy(rng.integers(0, ROWS, (3, n))).cuda()

    def run(blocks):
        off = blocks - nb
        cache = f.BlockCache(*(torch.zeros(blocks, H, 16, D, dtype=torch.uint8, device="cuda") for _ in range(2)),
                             *(torch.ones(blocks, H, device="cuda") for _ in range(2)))
        for x, y in zip((cache.k_cache, cache.v_cache), pools):
            x[off:] = y
        t, nt, fk = (_i32(np.where(x < 0, x, x + off)) for x in (table, new_table, forks))
        fault, weights, ctx, moved = _i32([0]), torch.zeros(3, H, 2400, device="cuda"), _i32(lens), torch.zeros(3, H, 640, device="cuda")
        turned = f.kv_block_cache(k, v, _i32(cu), max(lens), cache, t, ctx, rope=rope, q=q, positions=pos, fault=fault)
        f.fp8_block_attn_weights(turned, _i32(cu), max(lens), cache, t, ctx, weights, decay=0.0, fault=fault)
        f.fp8_block_attn_weights(turned[:3].contiguous(), _i32([0, 1, 2, 3]), 1, cache, t, ctx, weights, fault=fault)
        out = f.fp8_block_shared_decode_attn(q1, cache, fk, _i32([2300] * members), _i32([0, members]), _i32([2288]), fault=fault)
        kept = f.kv_block_evict(cache, t, ctx, weights, budget, nt, sink=4, recent=64, new_weights=moved, fault=fault)
        assert int(fault) == 0
        return [turned, weights, out, moved, *kept, *(x[off:].clone() for x in (cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale))]
    for x, y in zip(run(nb), run(far)):
        assert torch.equal(x, y)
