"""fp8_block_decode_attn and fp8_block_prefill_attn on the GPU against the float64 softmax.

Tolerance of an output element o, derived before the first run.  With p_j the softmax weights,
P = sum_j p_j |v_j| and V the largest |v_j| of the sequence:
  * P enters the product with at most 2^-8 relative error each: 2^-8 P;
  * the scores are FP32 sums of exact products: a relative error of each weight below 2^-10 for the
    sizes here (|q| |k| tau < 32, 512 terms of 2^-24): 2^-10 P;
  * weights below a tile's largest by more than 2^18 may round to zero or by a fixed step of
    2^-18.8 of it, in at most 256 keys of a tile: 2^-10 V (in practice far less);
  * the bf16 rounding of the output: 2^-8 |o|.
The relative L2 distance is held to 2^-7, the two half steps of 2^-8 together: a kernel that rounded
P or q to e4m3 (2^-4) would fail it."""
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
    """A seeded block-scaled cache with queries: finite codes inside the sequences, any byte (NaN codes
    too) behind them and in blocks that no sequence owns."""

    def __init__(self, ctx, hq, h, d, new=None, seed=0, spread=3, q_size=1.0, extra=2):
        rng = np.random.default_rng(seed)
        n = [(t + 15) // 16 for t in ctx]
        nb = sum(n) + extra
        perm = rng.permutation(nb).astype(np.int32)
        self.table, at = np.full((len(ctx), max(1, *n)), -1, np.int32), 0
        self.pools, self.scales = [], []
        for _ in range(2):
            x = rng.standard_normal((nb, h, 16, d))
            s = 2.0 ** rng.integers(-spread, spread + 1, (nb, h)) * 2.0 ** -7   # codes of size ~128
            self.pools.append(torch.from_numpy((x * 128).astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
            self.scales.append(s.astype(np.float32))
        for b, m in enumerate(n):
            self.table[b, :m] = perm[at:at + m]
            at += m
        for p in self.pools:
            p[perm[at:]] = 0x7F
            for b, t in enumerate(ctx):
                if t % 16:
                    p[self.table[b, t // 16], :, t % 16:] = rng.choice([0x7F, 0xFF, 0x7E, 3], p[0, :, t % 16:].shape)
        self.ctx, self.cu = list(ctx), None if new is None else np.concatenate(([0], np.cumsum(new)))
        rows = len(ctx) if new is None else int(self.cu[-1])
        self.max_new = None if new is None else max(new)
        self.q = torch.from_numpy((rng.standard_normal((rows, hq, d)) * q_size).astype(np.float32)).to(torch.bfloat16)

    def cache(self):
        return f.BlockCache(*(torch.from_numpy(p).cuda() for p in self.pools), *(torch.from_numpy(s).cuda() for s in self.scales))

    def exact(self, **kw):
        a = (self.pools[0], self.pools[1], self.scales[0], self.scales[1], self.table, self.ctx, self.cu)
        q = self.q.float().numpy().astype(np.float64)
        o = blockcache.attend(q, *a, **kw)
        mag = blockcache.p_bound(q, *a, **kw)
        top = np.zeros(q.shape[0])
        for b, t in enumerate(self.ctx):
            r = slice(b, b + 1) if self.cu is None else slice(self.cu[b], self.cu[b + 1])
            if t:
                top[r] = max(np.abs(blockcache.sequence(self.pools[1], self.scales[1], self.table[b], t, g)).max()
                             for g in range(self.pools[1].shape[1]))
        return o, (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -10 * top[:, None, None] + 2.0 ** -8 * np.abs(o)

    def decode(self, **kw):
        fault = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = f.fp8_block_decode_attn(self.q.cuda(), self.cache(), _i32(self.table), _i32(self.ctx), fault=fault, **kw)
        assert int(fault) == 0
        return out

    def prefill(self, **kw):
        fault = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = f.fp8_block_prefill_attn(self.q.cuda(), _i32(self.cu), self.max_new, self.cache(), _i32(self.table), _i32(self.ctx),
                                       fault=fault, **kw)
        assert int(fault) == 0
        return out


def _check(got, exact, what=""):
    o, tol = exact
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), what
    err = np.abs(got - o)
    i = np.unravel_index(int(np.argmax(err - tol)), err.shape)
    assert np.all(err <= tol), f"{what}: {err[i]:.3e} above {tol[i]:.3e} at {i}"
    if np.any(o):
        assert rel_l2(got, o) <= 2.0 ** -7, f"{what}: rel_l2 {rel_l2(got, o):.2e}"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
def test_decode_groups_and_lengths(d, g):
    if g * d > 2048:
        pytest.skip("group and head_dim beyond the decode's limit")
    c = Case([0, 1, 15, 16, 17, 127, 128, 129, 300, 700], 3 * g, 3, d, seed=d + g)
    _check(c.decode(), c.exact())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 17, 33, 128, 500])
def test_decode_windows(d, window):
    c = Case([0, 1, 16, 31, 129, 640, 777], 8, 2, d, seed=window)
    _check(c.decode(window=window), c.exact(window=window))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,hq,h", [([2100, 40, 0], 8, 1), ([0, 0, 7, 0], 4, 4), ([9000], 2, 2),
                                      ([33, 500, 0, 16, 128, 1000, 64] * 11, 8, 8), ([20] * 300, 2, 1), ([5000] + [1] * 70, 3, 3)])
def test_decode_ranges_over_sequences(d, ctx, hq, h):
    """Contexts whose tiles are dealt out over the CTAs: units in many pieces, in one, several units (and
    sequences without keys between them) in one CTA's range."""
    c = Case(ctx, hq, h, d, seed=len(ctx))
    _check(c.decode(softmax_scale=0.2), c.exact(softmax_scale=0.2))


def test_decode_range_of_many_short_units():
    """More units than resident CTAs, each of a tile or two: every CTA walks several pieces."""
    rng = np.random.default_rng(4)
    ctx = [int(x) for x in rng.integers(0, 260, 230)]
    c = Case(ctx, 12, 6, 64, seed=7)
    _check(c.decode(), c.exact())


def test_decode_of_very_many_sequences():
    """More (sequence, KV head) pairs than the workspace's least number of counters, after a call with a smaller batch
    over the same workspace."""
    rng = np.random.default_rng(9)
    c = Case([int(x) for x in rng.integers(0, 24, 9000)] + [6000], 4, 2, 64, seed=9)
    small = Case([300, 6000], 4, 2, 64, seed=1)
    ws = f.block_decode_workspace(len(c.ctx), 4, c.cache())
    _check(c.decode(workspace=ws), c.exact())
    _check(small.decode(workspace=ws), small.exact())


@pytest.mark.parametrize("d,hq,h", [(64, 96, 96), (128, 160, 40), (256, 72, 9)])
def test_attention_of_many_heads(d, hq, h):
    dec = Case([70, 300, 1], hq, h, d, seed=d)
    _check(dec.decode(), dec.exact())
    pre = Case([70, 300, 1], hq, h, d, new=[7, 2, 1], seed=d)
    _check(pre.prefill(), pre.exact())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_workspace_serves_other_batches(d):
    """A batch that shrinks and grows again, and other heads, over one workspace that is never cleared."""
    cases = [Case([700] * 90, 8, 2, d, seed=1), Case([4000, 10], 8, 2, d, seed=2), Case([2500], 2, 2, 64, seed=3)]
    fresh = [c.decode() for c in cases]
    ws = f.block_decode_workspace(90, 8, cases[0].cache())
    for i in (0, 1, 0, 2, 1, 2, 0):
        assert torch.equal(cases[i].decode(workspace=ws), fresh[i]), i


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_on_another_stream_makes_its_tensors_there(raw):
    """The workspace and the output that a call makes belong to the stream it is given, also while the
    current stream is busy and free memory holds other bytes."""
    c = Case([3000, 40], 8, 2, 128, seed=5)
    p = Case([300, 40], 8, 2, 128, new=[20, 3], seed=6)
    ref, pref = c.decode(), p.prefill()
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx))
    pargs = (p.q.cuda(), _i32(p.cu), p.max_new, p.cache(), _i32(p.table), _i32(p.ctx))
    dirty = f.block_decode_workspace(2, 8, args[1]).fill_(255)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    del dirty
    torch.cuda._sleep(100_000_000)
    given = s.cuda_stream if raw else s
    out = f.fp8_block_decode_attn(*args, fault=fault, stream=given)
    pout = f.fp8_block_prefill_attn(*pargs, fault=fault, stream=given)
    with torch.cuda.stream(s):
        got, pgot, bits = out.cpu(), pout.cpu(), fault.cpu()
    assert int(bits) == 0
    assert torch.equal(got, ref.cpu()) and torch.equal(pgot, pref.cpu())


def test_decode_replays_with_other_contexts():
    """A captured launch with other context lengths than it was captured with."""
    full = [700, 300, 1100]
    c = Case(full, 8, 2, 128, seed=13)
    q, cache, table = c.q.cuda(), c.cache(), _i32(c.table)
    ctx, out = _i32([1, 1, 1]), torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    ws = f.block_decode_workspace(3, 8, cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.fp8_block_decode_attn(q, cache, table, ctx, out=out, workspace=ws)
    for lens in (full, [0, 300, 17], [700, 0, 0], [5, 6, 1100], [0, 0, 0], full):
        c.ctx = lens
        ctx.copy_(_i32(lens))
        graph.replay()
        _check(out, c.exact())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_scales_far_apart(d):
    """Block scales over 2^-12 .. 2^12, zero scales among them, and the largest query that a bf16
    softmax meets."""
    c = Case([333, 90], 4, 1, d, seed=d, spread=6, q_size=0.25)
    c.scales[0][c.table[0, 3]] = 0.0
    c.scales[1][c.table[0, 5]] = 0.0
    c.scales[1][c.table[1, :6]] = 0.0           # a sequence whose values are all zero
    _check(c.decode(), c.exact())


def test_decode_one_dominant_key():
    """A key whose weight is nearly one returns its value row, whatever the scales around it."""
    for d in (64, 128, 256):
        c = Case([1000], 8, 1, d, seed=d, spread=0)
        blk, slot = c.table[0, 700 // 16], 700 % 16
        k = (c.q[0, :1].float() / c.q[0, :1].float().norm()).numpy()
        c.q[0] = torch.from_numpy(k * 40.0).to(torch.bfloat16)
        c.pools[0][blk, 0, slot] = torch.from_numpy(k[0] * 400).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        c.scales[0][blk] = 2.0 ** -4
        o = c.decode(softmax_scale=1.0).float().cpu().numpy()
        v = blockcache.sequence(c.pools[1], c.scales[1], c.table[0], 1000, 0)[700]
        assert np.all(np.abs(o - v) <= 2.0 ** -7 * np.abs(v) + 1e-6)


def test_decode_many_weights_far_below_the_first():
    """One key of weight about 1/2 and 20,000 that share the other half: weights far below the running
    maximum must not be lost."""
    T, d = 20000, 128
    c = Case([T], 4, 1, d, seed=3, spread=0)
    c.pools[0][:] = 0
    c.q[:] = 0
    c.q[0, :, 0] = 1.0
    c.pools[0][c.table[0, 0], 0, 5, 0] = 0x7E      # 448 / 16 = 28 ... times the softmax scale below
    c.scales[0][:] = 2.0 ** -4
    sm = float(np.log(T)) / 28.0
    _check(c.decode(softmax_scale=sm), c.exact(softmax_scale=sm))


def test_decode_long_context():
    """131,072 keys against float64 on the GPU."""
    T, hq, h, d = 131072, 8, 1, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    nb = T // 16
    codes = [(torch.randn(nb, h, 16, d, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-9, -5, (nb, h), generator=g, device="cuda").float()) for _ in range(2)]
    q = torch.randn(1, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)[None]
    out = f.fp8_block_decode_attn(q, f.BlockCache(codes[0].view(torch.uint8), codes[1].view(torch.uint8), *scales), table, _i32([T]))
    k, v = (c[table[0].long(), 0].double().mul(s[table[0].long(), 0].double()[:, None, None]).flatten(0, 1) for c, s in zip(codes, scales))
    ref = torch.softmax(q[0].double() @ k.T / d ** 0.5, 1) @ v
    assert rel_l2(out[0].double().cpu().numpy(), ref.cpu().numpy()) <= 2.0 ** -7


def test_decode_reuses_its_workspace_and_two_streams_with_their_own():
    c = Case([900, 77, 1300], 8, 2, 128, seed=21)
    q, cache, table, ctx = c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx)
    ws = [f.block_decode_workspace(3, 8, cache) for _ in range(2)]
    first = f.fp8_block_decode_attn(q, cache, table, ctx, workspace=ws[0])
    torch.cuda.synchronize()
    outs = []
    for i, s in enumerate((torch.cuda.Stream(), torch.cuda.Stream())):
        with torch.cuda.stream(s):
            for _ in range(5):
                outs.append(f.fp8_block_decode_attn(q, cache, table, ctx, workspace=ws[i]))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)
    assert int(ws[0][:4 * 3 * 2].sum()) == 0


def test_decode_bad_block_ids_and_contexts_are_reported():
    c = Case([100, 40], 4, 1, 128, seed=2)
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = c.table.copy()
    bad[0, 2] = c.pools[0].shape[0]
    bad[1, 0] = -1
    f.fp8_block_decode_attn(c.q.cuda(), c.cache(), _i32(bad), _i32(c.ctx), fault=fault)
    assert int(fault) == f.FAULT_BLOCK_ID
    fault.zero_()
    c2 = Case([112, 0], 4, 1, 128, seed=2)
    out = f.fp8_block_decode_attn(c2.q.cuda(), c2.cache(), _i32(c2.table), _i32([10 ** 9, -3]), fault=fault)
    assert int(fault) == f.FAULT_CONTEXT
    o, tol = c2.exact()
    assert np.all(np.abs(out.float().cpu().numpy() - o) <= tol)   # clamped to 112 and 0 keys


# ------------------------------------------------------------------ prefill

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g", [1, 3, 8])
def test_prefill_ragged_causal(d, g):
    new = [1, 2, 0, 17, 128, 129, 260]
    c = Case([1, 300, 9, 17, 128, 400, 700], 2 * g, 2, d, new=new, seed=d + g)
    _check(c.prefill(), c.exact())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 5, 64, 129, 300])
def test_prefill_windows(d, window):
    c = Case([600, 40, 257], 4, 2, d, new=[333, 40, 1], seed=window + d)
    _check(c.prefill(window=window), c.exact(window=window))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_all_keys_and_more_queries_than_keys(d):
    c = Case([5, 0, 333, 129], 4, 1, d, new=[140, 3, 20, 129], seed=d)
    _check(c.prefill(causal=False, softmax_scale=0.11), c.exact(causal=False, softmax_scale=0.11))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_scales_far_apart(d):
    c = Case([500], 4, 1, d, new=[200], seed=d, spread=6, q_size=0.25)
    c.scales[0][c.table[0, 3]] = 0.0
    c.scales[1][c.table[0, 5]] = 0.0
    c.scales[1][c.table[0, 16:24]] = 0.0        # a whole tile of zero values
    _check(c.prefill(), c.exact())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,new,hq,h,kw", [
    ([2050], [9], 8, 2, {}), ([1300, 5000, 70], [1, 4, 70], 4, 1, {}), ([3000], [20], 3, 1, dict(window=700)),
    ([700, 2600], [7, 130], 2, 2, dict(causal=False)), ([4097, 129], [1, 2], 16, 1, dict(softmax_scale=0.3)),
])
def test_prefill_few_rows_over_long_contexts(d, ctx, new, hq, h, kw):
    """Key tiles shared by the CTAs of a cluster, some of which may have none."""
    c = Case(ctx, hq, h, d, new=new, seed=d + sum(new))
    _check(c.prefill(**kw), c.exact(**kw))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_and_blocks_of_zeros(d):
    """Query rows of zeros (and tiny ones) over blocks of zero keys, whose scale the append sets to 2^-126, and
    blocks of scale zero: the keys they see weigh alike, the masked ones nothing."""
    for new in (None, [200, 77, 1]):
        for window in (0, 40):
            c = Case([500, 77, 130], 4, 2, d, new=new, seed=d)
            c.q[:, 1] = 0
            c.q[::3] = 0
            c.q[1::5] *= 2.0 ** -120
            zero = c.table[0, 1:31:2]
            c.pools[0][zero] = 0
            c.scales[0][zero] = 2.0 ** -126
            c.scales[0][c.table[0, 2:31:4]] = 0.0
            c.pools[0][c.table[2]] = np.where(c.pools[0][c.table[2]] & 0x7F == 0x7F, 0x7F, 0)
            c.scales[0][c.table[2]] = 2.0 ** -126
            _check(c.decode(window=window) if new is None else c.prefill(window=window), c.exact(window=window), (new, window))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_subnormal_value_scales(d):
    """Scales on both sides of the smallest normal number (outputs are normal bf16 numbers, whose step at
    2^-126 is within the tolerance's 2^-10 V)."""
    for new in (None, [200, 77]):
        c = Case([500, 77], 4, 2, d, new=new, seed=d)
        c.scales[1] = (c.scales[1].astype(np.float64) * 2.0 ** -119).astype(np.float32)
        c.scales[1][c.table[1]] = 2.0 ** -128
        _check(c.decode() if new is None else c.prefill(), c.exact(), new)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("batch,h", [(1, 2), (2, 8), (5, 4), (3, 8), (7, 4), (5, 8), (9, 7)])
def test_prefill_clusters_of_any_size(d, batch, h):
    """Few rows on 2 to 63 CTAs: clusters of 8 down to 2, also of sizes that are no power of two, over key tiles
    that do not divide among them."""
    ctx = [2000 - 37 * b for b in range(batch)]
    c = Case(ctx, 2 * h, h, d, new=[3 + b for b in range(batch)], seed=d + batch)
    _check(c.prefill(), c.exact())


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_last_wave_in_clusters(d):
    """More CTAs than SMs over a long context, in clusters of two; one sequence of few queries among them."""
    c = Case([8230, 8300], 32, 4, d, new=[317, 5], seed=d)
    _check(c.prefill(), c.exact())


def test_lengths_bounded_by_the_largest_integer():
    """max_q_len may be any upper bound."""
    c = Case([300, 40], 4, 2, 128, new=[20, 3], seed=6)
    ref = c.prefill()
    c.max_new = 2 ** 31 - 1
    assert torch.equal(c.prefill(), ref)
    k = torch.randn(23, 2, 128, device="cuda").to(torch.bfloat16)
    pools = []
    for most in (20, 2 ** 31 - 1):
        cache = c.cache()
        f.kv_block_cache(k, k, _i32(c.cu), most, cache, _i32(c.table), _i32(c.ctx))
        pools.append(cache)
    assert torch.equal(pools[0].k_cache, pools[1].k_cache) and torch.equal(pools[0].v_scale, pools[1].v_scale)


@pytest.mark.parametrize("hq", [130, 200])
def test_prefill_groups_beyond_128_heads(hq):
    c = Case([40, 300], hq, 1, 64, new=[3, 2], seed=hq)
    _check(c.prefill(), c.exact())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows_over_evicted_blocks(d):
    """What lies before the window is gone: blocks taken out of the table, their slots in the window's
    first block overwritten with NaN codes."""
    ctx, new, w = [900, 140], [3, 20], 100
    c = Case(ctx, 4, 2, d, new=new, seed=d)
    exact = c.exact(window=w)
    dec = Case(ctx, 4, 2, d, seed=d)
    dec_exact = dec.exact(window=w)
    for case, first in ((c, [t - n + 1 - w for t, n in zip(ctx, new)]), (dec, [t - w for t in ctx])):
        for b, lo in enumerate(first):
            for p in case.pools:
                p[case.table[b, lo // 16], :, :lo % 16] = 0x7F
            case.table[b, :lo // 16] = -1
    _check(c.prefill(window=w), exact)
    _check(dec.decode(window=w), dec_exact)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_query_rows_that_are_not_finite_give_nan_and_leave_the_others(d, bad):
    for new, ctx in ((None, [300, 5000]), ([5, 2], [300, 5000])):
        c = Case(ctx, 4, 2, d, new=new, seed=d)
        ref = c.decode() if new is None else c.prefill()
        c.q[1, 2, 7] = bad
        out = c.decode() if new is None else c.prefill()
        assert bool(torch.isnan(out[1, 2]).all())
        out[1, 2] = ref[1, 2]
        assert torch.equal(out, ref)


def test_first_calls_inside_a_capture():
    """A process whose first call of each entry point is a captured one."""
    code = """
import torch, fp8_kv_cache_quant_gb300 as f
f.load_binding()
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
k = torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16)
q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
c = f.BlockCache.empty(4, 2, 64)
tab, ctx, cu = i32(1, 2).view(1, 2), i32(3), i32(0, 3)
rope = f.Rope(f.Rope.table(40, 64))
lc, s = f.LayerCache.empty(4, 2, 64), torch.ones(1, device="cuda")
pos = torch.arange(3, device="cuda")
ws = f.block_decode_workspace(1, 4, c)
outs = [torch.empty_like(q) for _ in range(3)]
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    f.kv_rope_cache(None, k, k, pos, pos, rope, lc, s, s)
    f.kv_block_cache(k, k, cu, 3, c, tab, ctx, rope=rope, q=q, q_out=outs[0])
    f.fp8_block_prefill_attn(outs[0], cu, 3, c, tab, ctx, out=outs[1])
    f.fp8_block_decode_attn(outs[0][2:], c, tab, ctx, out=outs[2][:1], workspace=ws)
g.replay()
torch.cuda.synchronize()
assert torch.isfinite(outs[1]).all() and (outs[1][2] - outs[2][0]).float().abs().max() <= 2.0 ** -6 * outs[1][2].float().abs().max()
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_captured_behind_copies_fills_and_joined_streams():
    """One graph in which the calls follow a copy, a fill, kernels of torch and a second stream, replayed with other
    inputs, against the same calls made eagerly."""
    d, hq, h = 128, 8, 2
    rng = np.random.default_rng(3)
    rope = f.Rope(f.Rope.table(300, d))
    table, cu = _i32([[1, 3], [0, 2]]), _i32([0, 5, 25])
    ctx, pos = _i32([5, 20]), torch.arange(25, device="cuda")
    one = torch.ones(1, device="cuda")

    def draw():
        return torch.from_numpy(rng.standard_normal((25, hq + 2 * h, d)).astype(np.float32)).to(torch.bfloat16).cuda()

    x, source = draw(), draw()
    side = torch.cuda.Stream()
    slots, blocks, more = f.LayerCache.empty(2, h, d), f.BlockCache.empty(4, h, d), f.BlockCache.empty(4, h, d)

    def calls():
        x.copy_(source)
        slots.k_cache.zero_()
        q1 = f.kv_rope_cache(x[:, :hq], x[:, hq:hq + h], x[:, hq + h:], pos, pos, rope, slots, one, one)
        more.k_scale.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = x + x
            q2 = f.kv_block_cache(y[:, hq:hq + h], y[:, hq + h:], cu, 20, more, table, ctx, rope=rope, q=y[:, :hq])
            o2 = f.fp8_block_decode_attn(q2[3:5], more, table, ctx)
        q3 = f.kv_block_cache(x[:, hq:hq + h], x[:, hq + h:], cu, 20, blocks, table, ctx, rope=rope, q=x[:, :hq])
        o3 = f.fp8_block_prefill_attn(q3, cu, 20, blocks, table, ctx)
        torch.cuda.current_stream().wait_stream(side)
        o4 = f.fp8_block_decode_attn(q3[:2], more, table, ctx)
        return [q1, q2, o2, q3, o3, o4, slots.k_cache[:1], more.k_scale, blocks.v_scale]

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls()
    for _ in range(3):
        source.copy_(draw())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        want = calls()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), i


def test_prefill_leaves_other_rows_and_reports_bad_sequences():
    c = Case([40, 50, 60], 4, 2, 128, new=[10, 20, 30], seed=4)
    q = torch.cat((c.q, c.q[:7])).cuda()
    out = torch.full_like(q, -3.0)
    args = (c.cache(), _i32(c.table))
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    f.fp8_block_prefill_attn(q, _i32(c.cu), 30, *args, _i32(c.ctx), out=out, fault=fault)
    assert int(fault) == 0 and bool((out[60:] == -3.0).all())
    _check(out[:60], c.exact())
    for cu, mx, ctx, bit in [([0, 10, 30, 60], 29, c.ctx, f.FAULT_QLEN), ([0, 10, 30, 68], 40, c.ctx, f.FAULT_QLEN),
                             ([0, 10, 5, 35], 30, c.ctx, f.FAULT_QLEN), ([0, 10, 30, 60], 30, [40, 50, 29], f.FAULT_QLEN),
                             ([0, 10, 30, 60], 30, [40, 50, 65], f.FAULT_CONTEXT)]:
        fault.zero_()
        f.fp8_block_prefill_attn(q, _i32(cu), mx, *args, _i32(ctx), out=out, fault=fault)
        assert int(fault) == bit
    fault.zero_()
    f.fp8_block_prefill_attn(q, _i32(c.cu), 30, args[0], _i32(np.where(c.table >= 0, c.table + 10 ** 6, -1)), _i32(c.ctx), out=out, fault=fault)
    assert int(fault) == f.FAULT_BLOCK_ID


def test_attention_past_four_gigabytes():
    h, d = 8, 128
    nb = (1 << 32) // (h * 16 * d) + 40
    c = Case([500], 8, h, d, new=[30], seed=6)
    small = c.cache()
    big = f.BlockCache.empty(nb, h, d)
    m = small.k_cache.shape[0]
    for a, b in ((big.k_cache, small.k_cache), (big.v_cache, small.v_cache), (big.k_scale, small.k_scale), (big.v_scale, small.v_scale)):
        a[nb - m:] = b
    far = _i32(np.where(c.table >= 0, c.table + nb - m, -1))
    q = c.q.cuda()
    assert torch.equal(f.fp8_block_prefill_attn(q, _i32(c.cu), 30, big, far, _i32(c.ctx)),
                       f.fp8_block_prefill_attn(q, _i32(c.cu), 30, small, _i32(c.table), _i32(c.ctx)))
    assert torch.equal(f.fp8_block_decode_attn(q[:1], big, far, _i32(c.ctx)), f.fp8_block_decode_attn(q[:1], small, _i32(c.table), _i32(c.ctx)))


def test_attention_refusals():
    c = Case([40], 4, 2, 128, new=[4], seed=1)
    q, cache, table, ctx, cu = c.q.cuda(), c.cache(), _i32(c.table), _i32(c.ctx), _i32(c.cu)
    for bad in (q.float(), q.transpose(0, 1).contiguous().transpose(0, 1), q[..., :64]):
        with pytest.raises(ValueError):
            f.fp8_block_prefill_attn(bad, cu, 4, cache, table, ctx)
    with pytest.raises(ValueError):
        f.fp8_block_decode_attn(q, cache, table, ctx)                       # 4 rows for one sequence
    with pytest.raises(ValueError):
        f.fp8_block_decode_attn(q[:1], f.BlockCache(cache.k_cache, cache.v_cache, cache.k_scale[:1], cache.v_scale), table, ctx)
    with pytest.raises(f.FkvError):
        f.fp8_block_prefill_attn(q, cu, 4, cache, table, ctx, causal=False, window=3)


# ------------------------------------------------------------------ the operators together

@pytest.mark.parametrize("d,hq,h,style", [(128, 8, 2, False), (64, 8, 1, True), (256, 4, 1, False)])
def test_serving_run(d, hq, h, style):
    """Two sequences: a prompt in two chunks, then single tokens captured in one graph per step (append and
    decode), against float64 attention over the codes that the appends left, and the rotated keys within
    half a step of their codes."""
    rng = np.random.default_rng(d)
    lens, rope = [45, 150], f.Rope(f.Rope.table(400, d), style)
    rows = rope.cos_sin.cpu().numpy()
    nb = 40
    cache = f.BlockCache.empty(nb, h, d)
    table = rng.permutation(nb)[:2 * 12].reshape(2, 12).astype(np.int32)
    tab, ctx = _i32(table), [0, 0]
    keys = [np.zeros((0, h, d)), np.zeros((0, h, d))]

    def draw(n):
        w = torch.from_numpy(rng.standard_normal((n, (hq + 2 * h) * d)).astype(np.float32)).to(torch.bfloat16).cuda()
        return w[:, :hq * d].view(n, hq, d), w[:, hq * d:(hq + h) * d].view(n, h, d), w[:, (hq + h) * d:].view(n, h, d)

    def check(out, q, new):
        cu = np.concatenate(([0], np.cumsum(new)))
        a = [t.cpu().numpy() for t in (cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale)]
        ref = blockcache.attend(q.float().cpu().numpy().astype(np.float64), *a, table, ctx, cu)
        assert rel_l2(out.float().cpu().numpy(), ref) <= 2.0 ** -7

    def remember(k, new):
        at = 0
        for b, m in enumerate(new):
            x = k[at:at + m].float().cpu().numpy().astype(np.float64)
            keys[b] = np.concatenate((keys[b], blockcache.turn(x, rows[ctx[b] - m:ctx[b]], style)))
            at += m

    for new in ([30, 99], [15, 51]):
        q, k, v = draw(sum(new))
        ctx = [c + m for c, m in zip(ctx, new)]
        cu = _i32(np.concatenate(([0], np.cumsum(new))))
        turned = f.kv_block_cache(k, v, cu, max(new), cache, tab, _i32(ctx), rope=rope, q=q)
        out = f.fp8_block_prefill_attn(turned, cu, max(new), cache, tab, _i32(ctx))
        remember(k, new)
        check(out, turned, new)
    assert ctx == lens
    # one graph, replayed with new inputs
    q, k, v = (t.clone() for t in draw(2))
    dctx, cu = _i32([1, 1]), _i32([0, 1, 2])
    ws = f.block_decode_workspace(2, hq, cache)
    turned, out = torch.empty(2, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(2, hq, d, dtype=torch.bfloat16, device="cuda")
    spare = f.BlockCache(*(t.clone() for t in (cache.k_cache, cache.v_cache, cache.k_scale, cache.v_scale)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.kv_block_cache(k, v, cu, 1, cache, tab, dctx, rope=rope, q=q, q_out=turned)
        f.fp8_block_decode_attn(turned, cache, tab, dctx, out=out, workspace=ws)
    assert torch.equal(spare.k_cache, cache.k_cache)
    for _ in range(20):
        nq, nk, nv = draw(2)
        ctx = [c + 1 for c in ctx]
        q.copy_(nq), k.copy_(nk), v.copy_(nv), dctx.copy_(_i32(ctx))
        graph.replay()
        remember(nk, [1, 1])
        check(out, turned, [1, 1])
    for b in range(2):
        for g in range(h):
            got = blockcache.sequence(cache.k_cache.cpu().numpy(), cache.k_scale.cpu().numpy(), table[b], ctx[b], g)
            s = np.repeat(cache.k_scale.cpu().numpy()[table[b], g], 16)[:ctx[b], None]
            assert np.all(np.abs(got - keys[b][:, g]) <= 2.0 ** -4 * np.abs(keys[b][:, g]) + 4 * s * 2.0 ** -10)


def test_decode_of_very_many_sequences_after_smaller_calls():
    """A batch of more (sequence, KV head) pairs than the workspace's counters, after calls of fewer over the same
    workspace, whose scratch they have left in it: none of it is where the large batch counts."""
    rng = np.random.default_rng(19)
    big = Case([int(x) for x in rng.integers(0, 24, 9000)] + [60000], 4, 2, 64, seed=9)
    exact = big.exact()
    ws = f.block_decode_workspace(len(big.ctx), 4, big.cache())
    for small in (Case([300, 6000], 4, 2, 64, seed=1), Case([9000] * 3, 16, 2, 256, seed=2), Case([700] * 90, 8, 2, 128, seed=3)):
        _check(small.decode(workspace=ws), small.exact())
        _check(big.decode(workspace=ws), exact)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,new,hq,h,kw", [
    ([200, 190, 180], [4, 3, 4], 8, 2, {}), ([300, 2000, 16], [2, 9, 1], 8, 2, {}), ([2000, 300], [5, 1], 4, 1, dict(window=150)),
    ([700, 8300, 0, 3], [700, 40, 0, 3], 32, 4, {}), ([833], [833], 32, 4, {}), ([9000, 700], [300, 700], 32, 4, dict(window=8500)),
    ([500, 9000], [400, 300], 32, 4, dict(causal=False)), ([2048] + [500] * 20, [600] + [1] * 20, 8, 2, {}),
])
def test_prefill_with_tables_wider_than_the_contexts(d, ctx, new, hq, h, kw):
    """Tables as wide as a model's longest context: the plan, made from that width, must serve short contexts too
    (query tiles that share their keys in clusters, some sequences of a batch and others not)."""
    c = Case(ctx, hq, h, d, new=new, seed=d + len(ctx))
    c.table = np.concatenate((c.table, np.full((len(ctx), 8192 - c.table.shape[1]), -1, np.int32)), 1)
    exact = c.exact(**kw)
    _check(c.prefill(**kw), exact)
