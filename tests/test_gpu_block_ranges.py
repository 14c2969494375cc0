"""Block-scaled attention where the scales of a tile, or the elements of a query, lie far apart, against the
float64 softmax, row by row.

Tolerance, derived before the first run.  P enters with a relative error of at most 2^-8 wherever it is
not below 2^-17 of its tile's largest p * v_scale, and the output is rounded to bf16 (2^-9): a row whose weight
lies in keys of one V scale is within 2^-8 + 2^-9 < 2^-7 of its own norm.  An output below 2^-126 is rounded to a multiple
of 2^-133, bf16's subnormal step: half of it, 2^-134, for each of the d elements adds sqrt(d) 2^-134 to the norm."""
import numpy as np
import pytest
import torch

from oracle import blockcache
from test_gpu_block_attn import Case

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu


def _rows(got, ref, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), what
    err, norm = np.linalg.norm(got - ref, axis=-1), np.linalg.norm(ref, axis=-1)
    over = err - 2.0 ** -7 * norm - np.sqrt(ref.shape[-1]) * 2.0 ** -134
    i = np.unravel_index(int(np.argmax(over)), err.shape)
    assert over[i] <= 0, f"{what}: row {i} is off by {err[i]:.2e}, of a norm of {norm[i]:.2e}"


def _drawn_to(c, blocks, gap):
    """Make every query of the (one-sequence) case prefer the keys of its pages `blocks` by `gap` nats (softmax scale 1)."""
    c.q.mul_(0.02)
    c.q[..., 0] = gap / 4.0
    c.scales[0][:] = 2.0 ** -7
    c.pools[0][..., 0] = 0
    c.pools[0][c.table[0, blocks], ..., 0] = 0x78              # 256, at the scale 2^-6: 4
    c.scales[0][c.table[0, blocks]] = 2.0 ** -6


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("far", [10, 12, 14, 16, 20, 40, 70, 95])
def test_weight_in_blocks_of_small_value_scales(d, far):
    """The keys that carry the weight have V scales 2^-far of their neighbours' in the same tile."""
    for new, causal in ((None, True), ([40], True), ([3], True), ([40], False)):
        c = Case([500], 8, 1, d, new=new, seed=d + far, spread=0)
        small = [2, 5, 13, 21]
        _drawn_to(c, small, 0.75 * far + 10.0)                 # the others' weights: 2^-8 below what their scales are above
        c.scales[1][:] = 2.0 ** (far - 20)
        c.scales[1][c.table[0, small]] = 2.0 ** -20
        kw = {} if new is None else dict(causal=causal)
        ref = c.exact(softmax_scale=1.0, **kw)[0]
        _rows(c.decode(softmax_scale=1.0) if new is None else c.prefill(softmax_scale=1.0, **kw), ref, (new, causal))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("top", [2.0 ** -120, 2.0 ** -7, 2.0 ** 70, 2.0 ** 110])
def test_weight_in_blocks_of_zero_value_scale(d, top):
    """Keys of scale zero, and of one 2^120 below the others', carry about half of the weight, and all but 2^-14
    of it: the rest of the sequence makes the output.  (A whole tile, or two, of them among the others.)"""
    for new in (None, [40], [2]):
        for gap in (0.0, 14.0 * np.log(2.0)):
            c = Case([900], 4, 1, d, new=new, seed=d, spread=0)
            zero = [1, 6, 17, 30, *range(32, 48)]
            _drawn_to(c, zero, gap)
            c.scales[1][:] = top
            c.scales[1][c.table[0, zero]] = 0.0
            c.scales[1][c.table[0, [6, 40]]] = top * 2.0 ** -120
            _rows(c.decode(softmax_scale=1.0) if new is None else c.prefill(softmax_scale=1.0), c.exact(softmax_scale=1.0)[0], new)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_value_scales_that_grow_along_the_sequence(d):
    """A whole prompt, and its last tokens, whose every block has a V scale 2^4 above the one before: each row's own
    last block makes its output."""
    for new in ([300], [37]):
        c = Case([300], 4, 2, d, new=new, seed=d, spread=0)
        c.scales[1][c.table[0]] = 2.0 ** (4.0 * np.arange(len(c.table[0])) - 40.0)[:, None]
        _rows(c.prefill(), c.exact()[0], new)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,new,window", [(300, 300, 0), (2000, 40, 0), (2000, 70, 500), (9000, 20, 0)])
def test_rows_do_not_depend_on_later_values(d, ctx, new, window):
    """V scales of the chunk's later blocks 2^20 higher: the rows before them keep their bytes."""
    c = Case([ctx], 4, 1, d, new=[new], seed=d)
    ref = c.prefill(window=window)
    first = (ctx - new) // 16 + 1                              # the first page whose tokens are all of the chunk
    for page in (first, first + 1):
        changed = Case([ctx], 4, 1, d, new=[new], seed=d)
        changed.scales[1][changed.table[0, page:]] *= 2.0 ** 20
        rows = page * 16 - (ctx - new)
        if rows >= new:
            continue
        out = changed.prefill(window=window)
        assert torch.equal(out[:rows], ref[:rows]) and not torch.equal(out[rows:], ref[rows:])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("top", [2.0 ** 127, 3e38, 2.0 ** 100, 2.0 ** -100, 2.0 ** -126])
def test_value_scales_at_the_ends_of_float32(d, top):
    """Scales near the largest float32 and at the smallest the append writes (codes of at most 1, so that the values are
    finite)."""
    for new in (None, [30], [300]):
        c = Case([300], 4, 1, d, new=new, seed=d, spread=0, q_size=0.3)
        c.scales[1][:] = np.float32(top)
        c.scales[1][c.table[0, ::3]] = np.float32(top / 8)
        live = c.pools[1][c.table[0]]
        c.pools[1][c.table[0]] = np.where((live & 0x7F) > 0x38, (live & 0x80) | 0x38, live)
        _rows(c.decode() if new is None else c.prefill(), c.exact()[0], new)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("first,then", [(2.0 ** -126, 2.0 ** 120), (2.0 ** 120, 2.0 ** -126), (2.0 ** -126, 2.0 ** 127), (2.0 ** -60, 2.0 ** 70)])
def test_tiles_of_tiny_and_of_huge_value_scales(d, first, then):
    """Whole tiles of scales at one end of float32, with zeros among them, before tiles at the other: every key's
    weight counts, whatever its value is worth (codes of at most 1)."""
    for new in (None, [300], [7]):
        c = Case([900], 4, 1, d, new=new, seed=d, spread=0, q_size=0.3)
        live = c.pools[1][c.table[0]]
        c.pools[1][c.table[0]] = np.where((live & 0x7F) > 0x38, (live & 0x80) | 0x38, live)
        for page, blk in enumerate(c.table[0]):
            c.scales[1][blk] = np.float32(0.0 if page % 16 == 3 else first if page < 16 or 32 <= page < 48 else then)
        _rows(c.decode() if new is None else c.prefill(), c.exact()[0], new)


# ------------------------------------------------------------------ queries

def _terms(x):
    """The worst distance of a bf16 element from its two e4m3 terms when the leading one is truncated to 3 fraction
    bits and each is then rounded by itself (x scaled so that the row's largest element is 128)."""
    lead = (x.view(torch.int32) & -(1 << 20)).view(torch.float32)
    e4 = lambda y: y.to(torch.float8_e4m3fn).float()  # noqa: E731
    return e4(lead) + e4(x - lead) - x


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_with_an_outlier_channel(d):
    """One element 2^13 times the others, whose keys are zero there: the scores are made by the small ones alone.  With
    its row's largest element brought to above 224, the remainder of a leading term is off by at most 2^-10, half a
    step of e4m3's subnormals.  With |k| = 1 in d - 1 channels the scores are then off by at most
    s = tau (d - 1) |q|max 2^-10 / 224, and the output by (e^2s - 1) sum p |v|, besides the rounding of P (2^-8) and
    of the output (2^-9)."""
    small = torch.arange(0x3C00, 0x3D80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()   # 2^-7 .. 2^-4
    worst = float(small[int(_terms(small).abs().argmax())])
    assert abs(_terms(torch.tensor([worst])).item()) > 2.0 ** -9.6
    for new in (None, [5], [200]):
        c = Case([300], 4, 1, d, new=new, seed=d, spread=0)
        c.q[:] = worst / 128.0
        c.q[..., 3] = 1.0
        sign = np.random.default_rng(d).integers(0, 2, c.pools[0].shape[:3])[..., None]
        c.pools[0] = np.broadcast_to(np.where(sign, 0x38, 0xB8), c.pools[0].shape).astype(np.uint8).copy()
        c.pools[1] = c.pools[0].copy()                          # values +-1, along the scores
        c.pools[0][..., 3] = 0
        c.scales[0][:], c.scales[1][:] = 1.0, 1.0
        tau = 2.0 ** 12 / d
        ref, mag = c.exact(softmax_scale=tau)[0], blockcache.p_bound(
            c.q.float().numpy().astype(np.float64), c.pools[0], c.pools[1], c.scales[0], c.scales[1], c.table, c.ctx, c.cu, softmax_scale=tau)
        s = tau * (d - 1) * 2.0 ** -10 / 224.0
        out = (c.decode(softmax_scale=tau) if new is None else c.prefill(softmax_scale=tau)).float().cpu().numpy().astype(np.float64)
        tol = (np.expm1(2.0 * s) + 2.0 ** -8) * mag + 2.0 ** -9 * np.abs(ref)
        assert np.all(np.abs(out - ref) <= tol), (new, float((np.abs(out - ref) / tol).max()))
