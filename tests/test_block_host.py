"""The rotary cache writes and the block-scaled cache on the host (no GPU needed): arguments that
are refused before anything is enqueued, by the C entry points and by the binding."""
import os

import pytest
import torch

f = pytest.importorskip("fp8_kv_cache_quant_gb300")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(f.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return f.load_library()


P = 1 << 20  # an aligned address that no refused call reads


def _layer(**kw):
    a = dict(k=P, v=P, nb=4, bs=16, H=2, D=128, fmt=0)
    a.update(kw)
    return f._LayerCache(a["k"], a["v"], a["nb"], a["bs"], a["H"], a["D"], a["fmt"])


def _block(**kw):
    a = dict(k=P, v=P, ks=P, vs=P, nb=4, bs=16, H=2, D=128)
    a.update(kw)
    return f._BlockCache(a["k"], a["v"], a["ks"], a["vs"], a["nb"], a["bs"], a["H"], a["D"])


def _rope(**kw):
    a = dict(t=P, n=100, rot=128, il=0)
    a.update(kw)
    return f._Rope(a["t"], a["n"], a["rot"], a["il"])


def _rope_cache(lib, **kw):
    a = dict(q=P, qs=1024, qo=2 * P, qos=1024, hq=8, k=P, ks=256, v=P, vs=256, pos=P, slot=P, n=4, rope=_rope(),
             cache=_layer(), ksc=P, vsc=P, gran=0, layer=0, mask=None, nl=0)
    a.update(kw)
    return lib.kv_rope_cache(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(hq=-1), dict(hq=0), dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(pos=None),
    dict(slot=None), dict(ksc=None), dict(vsc=None), dict(gran=2), dict(qs=1016), dict(qos=1020), dict(ks=255), dict(vs=252),
    dict(k=P + 8), dict(v=P + 2), dict(q=P + 8), dict(qo=P + 8), dict(qo=P, qos=2048), dict(pos=P + 4), dict(slot=P + 4),
    dict(rope=_rope(t=None)), dict(rope=_rope(t=P + 8)), dict(rope=_rope(n=0)), dict(rope=_rope(rot=0)),
    dict(rope=_rope(rot=144)), dict(rope=_rope(rot=-16)), dict(cache=_layer(nb=0)), dict(cache=_layer(H=0)),
    dict(cache=_layer(fmt=2)), dict(cache=_layer(k=None)), dict(cache=_layer(v=P + 8)), dict(cache=_layer(bs=0)), dict(layer=1, mask=P, nl=1),
])
def test_rope_cache_invalid(lib, kw):
    assert _rope_cache(lib, **kw) == f.INVALID_ARG


@pytest.mark.parametrize("kw", [dict(cache=_layer(bs=8)), dict(cache=_layer(D=96)), dict(rope=_rope(rot=24))])
def test_rope_cache_unsupported(lib, kw):
    assert _rope_cache(lib, **kw) == f.UNSUPPORTED


def test_empty_calls_do_nothing(lib):
    assert _rope_cache(lib, n=0) == f.OK
    assert _block_cache(lib, n=0) == f.OK and _block_cache(lib, b=0) == f.OK and _block_cache(lib, mq=0) == f.OK
    assert _decode(lib, b=0) == f.OK
    assert _prefill(lib, tq=0) == f.OK and _prefill(lib, b=0) == f.OK and _prefill(lib, mq=0) == f.OK


def _block_cache(lib, **kw):
    a = dict(q=P, qs=1024, qo=2 * P, qos=1024, hq=8, k=P, ks=256, v=P, vs=256, n=4, cu=P, b=2, mq=3, rope=_rope(),
             cache=_block(), table=P, mb=9, ctx=P)
    a.update(kw)
    return lib.kv_block_cache(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(b=-1), dict(mq=-1), dict(mb=0), dict(hq=0), dict(q=None), dict(qo=None), dict(k=None), dict(v=None),
    dict(cu=None), dict(table=None), dict(ctx=None), dict(cu=P + 2), dict(table=P + 1), dict(ctx=P + 2), dict(ks=248),
    dict(vs=260), dict(k=P + 4), dict(qs=1000), dict(qo=P, qos=1032), dict(rope=_rope(t=None)),
    dict(rope=_rope(t=None, rot=0)),  # queries without a rotation
    dict(q=None, qo=None, hq=0, rope=_rope(t=None)), dict(rope=_rope(rot=256)), dict(cache=_block(k=None)),
    dict(cache=_block(ks=None)), dict(cache=_block(vs=P + 2)), dict(cache=_block(v=P + 8)), dict(cache=_block(nb=0)),
    dict(cache=_block(H=-1)), dict(cache=_block(bs=-16)),
])
def test_block_cache_invalid(lib, kw):
    assert _block_cache(lib, **kw) == f.INVALID_ARG


@pytest.mark.parametrize("kw", [dict(cache=_block(bs=32)), dict(cache=_block(D=80)), dict(b=65536), dict(rope=_rope(rot=8))])
def test_block_cache_unsupported(lib, kw):
    assert _block_cache(lib, **kw) == f.UNSUPPORTED


def _decode(lib, **kw):
    a = dict(q=P, b=2, hq=8, cache=_block(), table=P, mb=9, ctx=P, sm=0.0, win=0, out=P, ws=P, wsb=1 << 30, ns=0)
    a.update(kw)
    return lib.fp8_block_decode_attn(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(b=-1), dict(hq=0), dict(hq=7), dict(mb=0), dict(win=-1), dict(ns=-1), dict(sm=-1.0), dict(sm=float("inf")),
    dict(sm=float("nan")), dict(q=None), dict(out=None), dict(table=None), dict(ctx=None), dict(ws=None), dict(wsb=64),
    dict(ws=P + 128), dict(q=P + 8), dict(out=P + 8), dict(cache=_block(vs=None)), dict(cache=_block(nb=-4)),
])
def test_block_decode_invalid(lib, kw):
    assert _decode(lib, **kw) == f.INVALID_ARG


@pytest.mark.parametrize("kw", [dict(hq=6), dict(hq=64), dict(hq=32, cache=_block(D=256)), dict(cache=_block(D=32)), dict(cache=_block(bs=1)),
                                dict(b=65536)])
def test_block_decode_unsupported(lib, kw):
    assert _decode(lib, **kw) == f.UNSUPPORTED


def test_block_decode_takes_the_decode_workspace(lib):
    n = f.fp8_decode_attn_workspace_size(2, 8, 2, 128, 9)
    assert n > 0 and _decode(lib, wsb=n - 1) == f.INVALID_ARG


def _prefill(lib, **kw):
    a = dict(q=P, cu=P, tq=10, b=2, hq=8, mq=7, cache=_block(), table=P, mb=9, ctx=P, sm=0.0, causal=1, win=0, out=P)
    a.update(kw)
    return lib.fp8_block_prefill_attn(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(tq=-1), dict(b=-1), dict(hq=0), dict(hq=9), dict(mq=-1), dict(mb=0), dict(win=-1), dict(sm=-0.5), dict(q=None),
    dict(cu=None), dict(table=None), dict(ctx=None), dict(out=None), dict(q=P + 4), dict(out=P + 4), dict(cu=P + 1),
    dict(cache=_block(k=P + 4)), dict(cache=_block(ks=None)),
])
def test_block_prefill_invalid(lib, kw):
    assert _prefill(lib, **kw) == f.INVALID_ARG


@pytest.mark.parametrize("kw", [dict(win=3, causal=0), dict(cache=_block(D=48)), dict(b=65536), dict(hq=65536 * 2)])
def test_block_prefill_unsupported(lib, kw):
    assert _prefill(lib, **kw) == f.UNSUPPORTED


# ------------------------------------------------------------------ the binding's own checks

def test_binding_refuses_cpu_tensors():
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    cache = f.BlockCache.empty(2, 1, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(1, 1, dtype=torch.int32)
    rope = f.Rope(f.Rope.table(4, 64, device="cpu"))
    with pytest.raises(ValueError, match="CUDA"):
        f.kv_block_cache(k, k, i, 1, cache, table, i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        f.kv_rope_cache(None, k, k, i.long(), i.long(), rope, f.LayerCache.empty(2, 1, 64, device="cpu"))
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_block_decode_attn(k[:1], cache, table, i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        f.fp8_block_prefill_attn(k, i, 1, cache, table, i[:1])


def test_binding_row_strides():
    dev = torch.device("cpu")
    wide = torch.zeros(5, 3 * 128, dtype=torch.bfloat16)
    assert f._rows("f", dev, "k", wide[:, 128:256].view(5, 2, 64), 5, 2, 64) == 384
    assert f._rows("f", dev, "k", wide[:1, :128].view(1, 2, 64), 1, 2, 64) >= 128
    assert f._rows("f", dev, "k", wide[:0, :128].view(0, 2, 64), 0, 2, 64) == 128
    for bad in (wide[:, ::2].unflatten(1, (3, 64))[:, :2], wide.view(5, 6, 64)[:, ::3], wide.float()[:, :128].view(5, 2, 64),
                wide[:, :128].view(5, 2, 64)[:4]):
        with pytest.raises(ValueError):
            f._rows("f", dev, "k", bad, 5, 2, 64)


def test_binding_tensor_checks():
    dev = torch.device("cpu")
    t = torch.zeros(4, 6, dtype=torch.int32)
    f._check_tensors("f", dev, ("t", t, torch.int32, (4, 6)), ("u", None, torch.int32, (1,)))
    for bad in (t.long(), t[:3], t.T, torch.zeros(4, 12, dtype=torch.int32)[:, ::2], t[0]):
        with pytest.raises(ValueError, match="f: t is"):
            f._check_tensors("f", dev, ("t", bad, torch.int32, (4, 6)))


def test_rope_table():
    t = f.Rope.table(7, 32, base=10000.0, device="cpu")
    assert t.shape == (7, 32) and t.dtype is torch.float32
    assert torch.equal(t[0], torch.cat((torch.ones(16), torch.zeros(16))))
    assert abs(float(t[3, 1]) - torch.cos(torch.tensor(3.0 * 10000.0 ** (-2 / 32), dtype=torch.float64)).item()) < 2 ** -24
    r = f.Rope(t, interleaved=True).c()
    assert (r.max_positions, r.rot_dim, r.interleaved) == (7, 32, 1)
