"""What the operators for long and shared contexts refuse on the host (no GPU needed): the C entry points before
anything is enqueued, and the binding."""
import ctypes
import dataclasses
import os

import numpy as np
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


_PAIRS = (ctypes.c_uint8 * 64)(*([0] * 32 + [2] * 32))


def _pos(**kw):
    a = dict(pos=P, stride=64, n=3, pair=ctypes.addressof(_PAIRS))
    a.update(kw)
    return f._Axes(a["pos"], a["stride"], a["n"], a["pair"])


BAD_AXES = [dict(n=0), dict(n=5), dict(n=2), dict(stride=-1), dict(pos=None), dict(pos=P + 4)]


def _rope_axes(lib, **kw):
    a = dict(q=P, qs=1024, qo=2 * P, qos=1024, hq=8, k=P, ks=256, v=P, vs=256, axes=_pos(), slot=P, n=4, rope=_rope(),
             cache=_layer(), ksc=P, vsc=P, gran=0, layer=0, mask=None, nl=0)
    a.update(kw)
    return lib.kv_rope_cache_axes(*a.values(), None, None)


def _block_axes(lib, **kw):
    a = dict(q=P, qs=1024, qo=2 * P, qos=1024, hq=8, k=P, ks=256, v=P, vs=256, n=4, axes=_pos(), cu=P, b=2, mq=4, rope=_rope(),
             cache=_block(), tab=P, mb=4, ctx=P)
    a.update(kw)
    return lib.kv_block_cache_axes(*a.values(), None, None)


@pytest.mark.parametrize("kw", BAD_AXES)
def test_axes_invalid(lib, kw):
    assert _rope_axes(lib, axes=_pos(**kw)) == f.INVALID_ARG
    assert _block_axes(lib, axes=_pos(**kw)) == f.INVALID_ARG


def test_axes_other_refusals_and_empty_calls(lib):
    assert _rope_axes(lib, slot=None) == f.INVALID_ARG and _rope_axes(lib, rope=_rope(rot=24)) == f.UNSUPPORTED
    assert _block_axes(lib, rope=_rope(t=None, rot=0)) == f.INVALID_ARG      # positions without a rotation
    assert _block_axes(lib, q=None, qo=None, hq=0, rope=_rope(t=None, rot=0)) == f.INVALID_ARG
    assert _block_axes(lib, cache=_block(D=96)) == f.UNSUPPORTED
    assert _rope_axes(lib, n=0) == f.OK and _block_axes(lib, n=0) == f.OK and _block_axes(lib, b=0) == f.OK


def test_rope_axes_of_the_binding():
    t = torch.zeros(9, 64)
    assert f.Rope(t).pair_args == (None, 0)
    assert f.Rope.sections(2, 0, 3) == [0, 0, 2, 2, 2]
    r = f.Rope(t, axes=f.Rope.sections(12, 10, 10))
    assert r.pair_args[1] == 32 and r.pair_axis.dtype == np.uint8
    for bad in ([0] * 31, [0] * 33, [4] + [0] * 31, [-1] + [0] * 31, [0.5] * 32, [[0] * 32]):
        with pytest.raises(ValueError, match="axes names"):
            f.Rope(t, axes=bad)


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_compiled_binding_checks_of_axes(lib):
    b = f.load_binding()
    i64, t = torch.zeros(5, dtype=torch.int64), torch.zeros(9, 64)
    pool, s = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(1)
    rope = f.Rope(t, axes=f.Rope.sections(12, 10, 10))
    pos = torch.zeros(3, 5, dtype=torch.int64)
    i32 = torch.zeros(3, dtype=torch.int32)
    one = dict(q=_bf(5, 4, 64), k=_bf(5, 2, 64), v=_bf(5, 2, 64), pos=pos, slots=i64, cs=t, il=0, ax=rope.pair_args[0], n=rope.pair_args[1],
               kc=pool, vc=pool, fmt=0, ks=s, vs=s, gran=0, layer=0, mask=None, nl=0, skip=0, qo=None, fault=None)
    two = dict(k=_bf(5, 2, 64), v=_bf(5, 2, 64), cu=i32, mx=3, kc=pool, vc=pool, ks=torch.ones(3, 2), vs=torch.ones(3, 2),
               tab=torch.zeros(2, 4, dtype=torch.int32), ctx=i32[:2], cs=t, il=0, ax=rope.pair_args[0], n=rope.pair_args[1], pos=pos, q=None,
               qo=None, fault=None)
    for fn, a in ((b.kv_rope_cache_axes, one), (b.kv_block_cache_axes, two)):
        for match, change in [
            ("positions is Long", dict(pos=i64)), (r"wanted Long \[axes, 5\]", dict(pos=pos[:, :4])), ("positions is Int", dict(pos=pos.int())),
            ("consecutive rows", dict(pos=torch.zeros(5, 3, dtype=torch.int64).T)), ("its table has 32", dict(n=31)), ("not a tensor", dict(pos=None)),
        ]:
            with pytest.raises(ValueError, match=match):
                fn(0, *dict(a, **change).values())
    with pytest.raises(ValueError, match="without a rope"):
        b.kv_block_cache_axes(0, *dict(two, cs=None, ax=None, n=0, pos=i64).values())
    with pytest.raises(ValueError, match="takes positions"):
        f.kv_block_cache(two["k"], two["v"], i32, 3, f.BlockCache(pool, pool, two["ks"], two["vs"]), two["tab"], two["ctx"], rope=rope)


# ------------------------------------------------------------------ eviction

def _evict(lib, **kw):
    a = dict(cache=_block(), tab=P, b=2, mb=8, ctx=P, w=P, wl=128, budget=32, sink=4, recent=8, nt=P, nmb=2, nl=P, kept=P, nw=P, nwl=32)
    a.update(kw)
    return lib.kv_block_evict(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(b=-1), dict(mb=0), dict(wl=-1), dict(nmb=-1), dict(nwl=-1), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=25),
    dict(recent=33), dict(recent=2 ** 31 - 1, sink=2 ** 31 - 1), dict(nmb=1), dict(nwl=31), dict(tab=None), dict(ctx=None), dict(w=None),
    dict(nt=None), dict(nl=None), dict(kept=None), dict(tab=P + 2), dict(w=P + 1), dict(nw=P + 2), dict(kept=P + 3),
    dict(cache=_block(k=None)), dict(cache=_block(vs=P + 2)), dict(cache=_block(nb=0)), dict(cache=_block(H=0)), dict(cache=_block(bs=0)),
])
def test_evict_invalid(lib, kw):
    assert _evict(lib, **kw) == f.INVALID_ARG


def test_evict_unsupported_and_empty(lib):
    assert _evict(lib, cache=_block(D=96)) == f.UNSUPPORTED and _evict(lib, cache=_block(bs=32)) == f.UNSUPPORTED
    assert _evict(lib, b=65536) == f.UNSUPPORTED and _evict(lib, mb=1 << 27) == f.UNSUPPORTED
    assert _evict(lib, b=65535, cache=_block(H=8192)) == f.UNSUPPORTED
    assert _evict(lib, b=0) == f.OK and _evict(lib, b=0, nw=None, nwl=0) == f.OK


def test_compiled_binding_checks_of_evict(lib):
    b = f.load_binding()
    pool, sc, i32 = torch.zeros(9, 2, 16, 64, dtype=torch.uint8), torch.ones(9, 2), torch.zeros(2, dtype=torch.int32)
    tab = torch.zeros(2, 4, dtype=torch.int32)
    a = dict(kc=pool, vc=pool, ks=sc, vs=sc, tab=tab, ctx=i32, w=torch.zeros(2, 2, 64), budget=20, sink=0, recent=0, nt=tab[:, :2].contiguous(),
             nw=torch.zeros(2, 2, 32), nl=i32, kept=torch.zeros(2, 2, 20, dtype=torch.int32), fault=None)
    for match, change in [
        ("k_cache is", dict(kc=pool[0])), ("v_scale", dict(vs=sc.T.contiguous())), ("block_table", dict(tab=tab[0])), ("context_lens", dict(ctx=i32[:1])),
        ("weights is Double", dict(w=torch.zeros(2, 2, 64).double())), (r"weights is .* \[2, 3, 64\]", dict(w=torch.zeros(2, 3, 64))),
        ("weights is .*not contiguous", dict(w=torch.zeros(2, 64, 2).transpose(1, 2))), ("weights is", dict(w=torch.zeros(4, 64))),
        ("new_table", dict(nt=tab[:1])), ("new_table", dict(nt=tab[0])), ("new_weights", dict(nw=torch.zeros(1, 2, 32))), ("new_weights", dict(nw=torch.zeros(32))),
        ("new_lens", dict(nl=i32.long())), ("kept", dict(kept=torch.zeros(2, 2, 19, dtype=torch.int32))), ("kept", dict(budget=-1)),
        ("fault", dict(fault=i32)), ("32 bits", dict(sink=1 << 40)), ("not a tensor", dict(nl=None)),
    ]:
        with pytest.raises(ValueError, match=match):
            b.kv_block_evict(0, *dict(a, **change).values())
    with pytest.raises(ValueError, match="not on a CUDA device"):
        f.kv_block_evict(f.BlockCache(pool, pool, sc, sc), tab, i32, a["w"], 20, tab)


# ------------------------------------------------------------------ attention weights

def _weights(lib, **kw):
    a = dict(q=P, cu=P, tq=8, b=2, hq=8, mq=4, cache=_block(), tab=P, mb=8, ctx=P, sm=0.0, decay=1.0, w=P, wl=128, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.fp8_block_attn_weights(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(tq=-1), dict(b=-1), dict(hq=0), dict(hq=7), dict(mq=-1), dict(mb=0), dict(wl=-1), dict(sm=-1.0), dict(sm=float("inf")),
    dict(sm=float("nan")), dict(decay=float("nan")), dict(decay=float("inf")), dict(q=None), dict(cu=None), dict(tab=None), dict(ctx=None),
    dict(w=None), dict(ws=None), dict(q=P + 8), dict(cu=P + 2), dict(tab=P + 2), dict(ctx=P + 1), dict(w=P + 2), dict(ws=P + 128), dict(wsb=16),
    dict(cache=_block(k=None)), dict(cache=_block(ks=None)), dict(cache=_block(nb=0)), dict(cache=_block(H=0)), dict(cache=_block(bs=0)),
])
def test_weights_invalid(lib, kw):
    assert _weights(lib, **kw) == f.INVALID_ARG


def test_weights_unsupported_empty_and_sizes(lib):
    assert _weights(lib, cache=_block(D=96)) == f.UNSUPPORTED and _weights(lib, cache=_block(bs=32)) == f.UNSUPPORTED
    assert _weights(lib, b=65536) == f.UNSUPPORTED and _weights(lib, mb=1 << 27) == f.UNSUPPORTED
    assert _weights(lib, tq=1 << 29, hq=6) == f.UNSUPPORTED
    assert _weights(lib, tq=0) == f.OK and _weights(lib, b=0) == f.OK and _weights(lib, mq=0) == f.OK
    size = f.fp8_block_attn_weights_workspace_size
    assert size(2, 8, 4, 8, 2, 128, 8) > 0 and size(2, 8, 99, 8, 2, 128, 8) == size(2, 8, 8, 8, 2, 128, 8)
    for bad in ((0, 8, 4, 8, 2, 128, 8), (2, 0, 4, 8, 2, 128, 8), (2, 8, 0, 8, 2, 128, 8), (2, 8, 4, 7, 2, 128, 8), (2, 8, 4, 8, 2, 96, 8),
                (2, 8, 4, 8, 2, 128, 0), (2, 8, 4, 8, 2, 128, 1 << 27)):
        assert size(*bad) == 0


def test_compiled_binding_checks_of_weights(lib):
    b = f.load_binding()
    pool, sc, i32 = torch.zeros(9, 2, 16, 64, dtype=torch.uint8), torch.ones(9, 2), torch.zeros(3, dtype=torch.int32)
    tab = torch.zeros(2, 4, dtype=torch.int32)
    a = dict(q=_bf(5, 4, 64), cu=i32, mx=3, kc=pool, vc=pool, ks=sc, vs=sc, tab=tab, ctx=i32[:2], w=torch.zeros(2, 2, 64), sm=0.0, decay=1.0,
             ws=torch.zeros(1 << 16, dtype=torch.uint8), fault=None)
    for match, change in [
        ("q is Half", dict(q=_bf(5, 4, 64).half())), ("q is", dict(q=_bf(5, 256))), ("q is .*not contiguous", dict(q=_bf(4, 5, 64).transpose(0, 1))),
        ("cu_seqlens_q", dict(cu=i32[:2])), ("k_cache", dict(q=_bf(5, 4, 128))), ("block_table", dict(tab=tab.long())), ("context_lens", dict(ctx=i32)),
        ("weights is", dict(w=torch.zeros(2, 64))), ("weights is", dict(w=torch.zeros(2, 4, 64))), ("weights is Half", dict(w=torch.zeros(2, 2, 64).half())),
        ("weights is .*not contiguous", dict(w=torch.zeros(2, 64, 2).transpose(1, 2))), ("workspace", dict(ws=torch.zeros(8, 8)[:, ::2])), ("fault", dict(fault=i32)),
    ]:
        with pytest.raises(ValueError, match=match):
            b.fp8_block_attn_weights(0, *dict(a, **change).values())
    with pytest.raises(ValueError, match="not on a CUDA device"):
        f.fp8_block_attn_weights(a["q"], i32, 3, f.BlockCache(pool, pool, sc, sc), tab, i32[:2], a["w"])


# ------------------------------------------------------------------ shared decode

def _shared(lib, **kw):
    a = dict(q=P, b=4, hq=8, cache=_block(), tab=P, mb=8, ctx=P, gs=P, sl=P, ng=2, sm=0.0, win=0, out=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.fp8_block_shared_decode_attn(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(b=-1), dict(hq=0), dict(hq=7), dict(mb=0), dict(ng=-1), dict(sm=-1.0), dict(sm=float("nan")), dict(win=-1), dict(q=None), dict(tab=None),
    dict(ctx=None), dict(gs=None), dict(sl=None), dict(gs=P + 2), dict(sl=P + 1), dict(out=None), dict(out=P + 8), dict(ws=None), dict(ws=P + 128),
    dict(wsb=1 << 16), dict(cache=_block(k=None)), dict(cache=_block(vs=None)), dict(cache=_block(nb=0)), dict(cache=_block(bs=0)),
])
def test_shared_invalid(lib, kw):
    assert _shared(lib, **kw) == f.INVALID_ARG


def test_shared_unsupported_empty_and_sizes(lib):
    assert _shared(lib, cache=_block(D=96)) == f.UNSUPPORTED and _shared(lib, hq=6) == f.UNSUPPORTED and _shared(lib, b=65536) == f.UNSUPPORTED
    assert _shared(lib, b=0) == f.OK and _shared(lib, b=0, ng=0, gs=None, sl=None) == f.OK
    size = f.fp8_block_shared_decode_attn_workspace_size
    assert size(4, 8, 2, 128, 2) >= f.fp8_block_decode_attn_workspace_size(4, 8, 2, 128) > 0
    assert size(4, 8, 2, 128, -1) == 0 and size(0, 8, 2, 128, 1) == 0 and size(4, 7, 2, 128, 1) == 0 and size(4, 8, 2, 96, 1) == 0


def test_compiled_binding_checks_of_shared(lib):
    b = f.load_binding()
    pool, sc, i32 = torch.zeros(9, 2, 16, 64, dtype=torch.uint8), torch.ones(9, 2), torch.zeros(3, dtype=torch.int32)
    tab = torch.zeros(3, 4, dtype=torch.int32)
    a = dict(q=_bf(3, 4, 64), kc=pool, vc=pool, ks=sc, vs=sc, tab=tab, ctx=i32, gs=i32, sl=i32[:2], sm=0.0, win=0, out=None,
             ws=torch.zeros(1 << 16, dtype=torch.uint8), fault=None)
    for match, change in [
        ("q is Half", dict(q=_bf(3, 4, 64).half())), ("q is BFloat16", dict(q=_bf(2, 4, 64))), ("k_cache", dict(q=_bf(3, 4, 128))), ("block_table", dict(tab=tab[0])),
        ("context_lens", dict(ctx=i32[:2])), ("group_starts", dict(gs=i32[:2])), ("group_starts is Long", dict(gs=i32.long())), ("shared_lens", dict(sl=tab)),
        ("shared_lens is Long", dict(sl=i32[:2].long())), ("out is", dict(out=_bf(3, 4, 32))), ("workspace", dict(ws=torch.zeros(8, 8)[:, ::2])), ("fault", dict(fault=i32)),
    ]:
        with pytest.raises(ValueError, match=match):
            b.fp8_block_shared_decode_attn(0, *dict(a, **change).values())
    with pytest.raises(ValueError, match="not on a CUDA device"):
        f.fp8_block_shared_decode_attn(a["q"], f.BlockCache(pool, pool, sc, sc), tab, i32, i32, i32[:2])


def test_no_weights_at_all(lib):
    """Null where there are none: refused for another reason only."""
    assert _weights(lib, w=None, wl=0, ws=None) == f.INVALID_ARG and _weights(lib, w=None, wl=0, b=0) == f.OK
    assert _weights(lib, w=None, wl=1) == f.INVALID_ARG
    assert _evict(lib, w=None, wl=1) == f.INVALID_ARG and _evict(lib, nt=None, nmb=1, wl=16) == f.INVALID_ARG


def test_copies_of_a_rope_with_axes():
    """The library reads a copy's axes from the copy's own memory, also in another process and behind the original."""
    import copy
    import pickle
    axes = f.Rope.sections(12, 10, 10)
    r = f.Rope(torch.zeros(9, 64), axes=axes)
    for make in (copy.deepcopy, copy.copy, lambda x: pickle.loads(pickle.dumps(x)), lambda x: dataclasses.replace(x, interleaved=True)):
        c = make(f.Rope(r.cos_sin, axes=axes))      # (the original is gone)
        at, n = c.pair_args
        assert at == c.pair_axis.ctypes.data and n == 32
        assert list((ctypes.c_uint8 * n).from_address(at)) == axes == list(c.axes)


def test_axes_assigned_later():
    r = f.Rope(torch.zeros(9, 64))
    assert r.pair_args == (None, 0)
    r.axes = [0, 1] * 16
    at, n = r.pair_args
    assert list((ctypes.c_uint8 * n).from_address(at)) == [0, 1] * 16
    with pytest.raises(ValueError, match="axes names"):
        r.axes = [0] * 31
    assert r.pair_axis.tolist() == list(r.axes) == [0, 1] * 16
    r.axes = None
    assert r.pair_axis is None and r.pair_args == (None, 0)
    given = [2] * 32
    r.axes = given
    given[0] = 0
    assert list(r.axes) == [2] * 32 == r.pair_axis.tolist()


def test_evict_results_over_its_own_input(lib):
    """New lengths over the lengths, moved weights over the weights: heads read them at any time."""
    far = 1 << 30
    ok = dict(ctx=P, nl=P + far, w=P + 2 * far, nw=P + 3 * far, kept=P + 4 * far)
    refused = [dict(nl=P), dict(nl=P + 4), dict(nl=P - 4), dict(nw=P + 2 * far), dict(nw=P + 2 * far + 4 * (2 * 2 * 128 - 1)),
               dict(nw=P + 2 * far - 4 * (2 * 2 * 32 - 1))]
    for kw in refused:
        assert _evict(lib, **{**ok, **kw}) == f.INVALID_ARG
    assert _evict(lib, **{**ok, "b": 0}) == f.OK
