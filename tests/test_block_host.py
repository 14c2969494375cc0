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


@pytest.mark.parametrize("kw", [dict(cache=_block(bs=32)), dict(cache=_block(D=80)), dict(b=65536), dict(mb=2 ** 27), dict(rope=_rope(rot=8))])
def test_block_cache_unsupported(lib, kw):
    assert _block_cache(lib, **kw) == f.UNSUPPORTED


def _decode(lib, **kw):
    a = dict(q=P, b=2, hq=8, cache=_block(), table=P, mb=9, ctx=P, sm=0.0, win=0, out=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.fp8_block_decode_attn(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(b=-1), dict(hq=0), dict(hq=7), dict(mb=0), dict(win=-1), dict(sm=-1.0), dict(sm=float("inf")),
    dict(sm=float("nan")), dict(q=None), dict(out=None), dict(table=None), dict(ctx=None), dict(ws=None), dict(wsb=64),
    dict(ws=P + 128), dict(q=P + 8), dict(out=P + 8), dict(cache=_block(vs=None)), dict(cache=_block(nb=-4)),
])
def test_block_decode_invalid(lib, kw):
    assert _decode(lib, **kw) == f.INVALID_ARG


@pytest.mark.parametrize("kw", [dict(hq=6), dict(hq=64), dict(hq=32, cache=_block(D=256)), dict(cache=_block(D=32)), dict(cache=_block(bs=1)),
                                dict(b=65536), dict(mb=2 ** 27)])
def test_block_decode_unsupported(lib, kw):
    assert _decode(lib, **kw) == f.UNSUPPORTED


def test_block_decode_workspace(lib):
    n = f.fp8_block_decode_attn_workspace_size(2, 8, 2, 128)
    assert n > 0 and _decode(lib, wsb=n - 1) == f.INVALID_ARG
    # counters, and a row per CTA and unit
    assert n >= 4 * 4 + 4 * (128 + 1) * 4 * (152 + 4)
    for bad in ((0, 8, 2, 128), (2, 7, 2, 128), (2, 8, 2, 96), (2, 6, 2, 128), (2, 8, 0, 64), (2, 32, 2, 256)):
        assert f.fp8_block_decode_attn_workspace_size(*bad) == 0


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


@pytest.mark.parametrize("kw", [dict(win=3, causal=0), dict(cache=_block(D=48)), dict(b=65536), dict(mb=2 ** 27), dict(hq=65536 * 2)])
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


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _refused(fn, match, args, **change):
    """The compiled binding refuses the arguments with `change` made (on the CPU: nothing is launched)."""
    a = dict(args)
    a.update(change)
    with pytest.raises(ValueError, match=match):
        getattr(f.load_binding(), fn)(0, *a.values())


def test_compiled_binding_checks_of_the_writes(lib):
    i64 = torch.zeros(5, dtype=torch.int64)
    pool, s, t = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(1), torch.zeros(9, 64)
    wide = _bf(5, 3 * 128)
    a = dict(q=_bf(5, 4, 64), k=wide[:, 128:256].view(5, 2, 64), v=_bf(5, 2, 64), pos=i64, slots=i64, cs=t, il=0, kc=pool, vc=pool,
             fmt=0, ks=s, vs=s, gran=0, layer=0, mask=None, nl=0, skip=0, qo=None, fault=None)
    for match, change in [
        ("positions is Int", dict(pos=i64.int())), (r"positions is Long \[4\]", dict(pos=i64[:4])), ("slot_mapping", dict(slots=i64[:0])),
        ("k's rows are not consecutive", dict(k=wide[:, ::2].unflatten(1, (3, 64))[:, :2])), ("v's rows", dict(v=wide.view(5, 6, 64)[:, ::3])),
        ("k is Float", dict(k=torch.zeros(5, 2, 64))), ("v is BFloat16", dict(v=_bf(4, 2, 64))), ("q is BFloat16", dict(q=_bf(5, 4, 32))),
        ("q is", dict(q=_bf(5, 256))), ("q_out without q", dict(q=None, qo=_bf(5, 4, 64))), ("q_out is", dict(qo=_bf(5, 4, 64).float())),
        ("q_out's rows", dict(qo=_bf(5, 64, 4).transpose(1, 2))), ("k_cache is Byte", dict(skip=1)), ("v_cache", dict(vc=pool[:2])),
        ("k_cache is Byte .*not contiguous", dict(kc=torch.zeros(3, 16, 2, 64, dtype=torch.uint8).transpose(1, 2))),
        ("k_cache", dict(kc=pool[0])), (r"wanted Float \[2\]", dict(gran=1)), ("v_scale is Double", dict(vs=s.double())),
        ("cos_sin", dict(cs=t.half())), ("cos_sin", dict(cs=t[0])), ("fault", dict(fault=i64)), ("not a tensor", dict(v=3)),
        ("not a tensor", dict(v=None)), ("32 bits", dict(layer=1 << 40)),
    ]:
        _refused("kv_rope_cache", match, a, **change)
    i32 = torch.zeros(3, dtype=torch.int32)
    c = dict(k=_bf(5, 2, 64), v=_bf(5, 2, 64), cu=i32, mx=3, kc=pool, vc=pool, ks=torch.ones(3, 2), vs=torch.ones(3, 2),
             tab=torch.zeros(2, 4, dtype=torch.int32), ctx=i32[:2], cs=t, il=0, q=None, qo=None, fault=None)
    for match, change in [
        ("cu_seqlens", dict(cu=i32[:2])), ("cu_seqlens is Long", dict(cu=i32.long())), ("block_table", dict(tab=i32)),
        ("block_table is Int .*not contiguous", dict(tab=torch.zeros(4, 2, dtype=torch.int32).T)), ("context_lens", dict(ctx=i32)),
        ("k_scale", dict(ks=torch.ones(3, 1))), ("v_scale", dict(vs=torch.ones(2, 2))), ("k_cache", dict(k=_bf(5, 3, 64), v=_bf(5, 3, 64))),
        ("v_cache", dict(vc=pool.view(torch.int8))), ("fault", dict(fault=torch.zeros(2, dtype=torch.int32))), ("cos_sin", dict(cs=t.T)),
        ("k is", dict(k=_bf(5, 128))),
    ]:
        _refused("kv_block_cache", match, c, **change)
    with pytest.raises(TypeError):
        f.load_binding().kv_block_cache(0, *dict(c, mx="3").values())
    for n in (3, 20):
        with pytest.raises(ValueError, match="arguments"):
            f.load_binding().kv_block_cache(0, *(list(c.values()) * 2)[:n])


def test_compiled_binding_checks_of_the_attention(lib):
    pool, s, i32 = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(3, 2), torch.zeros(3, dtype=torch.int32)
    tab = torch.zeros(2, 4, dtype=torch.int32)
    d = dict(q=_bf(2, 4, 64), kc=pool, vc=pool, ks=s, vs=s, tab=tab, ctx=i32[:2], sm=0.0, win=0, out=None,
             ws=torch.zeros(1 << 16, dtype=torch.uint8), fault=None)
    for match, change in [
        ("q is BFloat16 .3, 4, 64", dict(q=_bf(3, 4, 64))), ("q is Half", dict(q=_bf(2, 4, 64).half())), ("out is", dict(out=_bf(2, 4, 32))),
        ("k_cache", dict(q=_bf(2, 4, 128))), ("q is", dict(q=_bf(4, 2, 64).transpose(0, 1))), ("workspace", dict(ws=torch.zeros(8, 8)[:, ::2])),
        ("context_lens", dict(ctx=i32)), ("block_table", dict(tab=tab.long())), ("v_scale", dict(vs=s.T.contiguous())),
    ]:
        _refused("fp8_block_decode_attn", match, d, **change)
    p = dict(q=_bf(5, 4, 64), cu=i32, mx=3, kc=pool, vc=pool, ks=s, vs=s, tab=tab, ctx=i32[:2], sm=0.0, causal=1, win=0, out=None, fault=None)
    for match, change in [
        ("q is", dict(q=_bf(4, 5, 64).transpose(0, 1))), ("cu_seqlens_q", dict(cu=i32[:2])), ("out is", dict(out=_bf(6, 4, 64))),
        ("32 bits", dict(mx=1 << 31)), ("fault", dict(fault=i32)), ("not a tensor", dict(cu=None)),
    ]:
        _refused("fp8_block_prefill_attn", match, p, **change)


def test_rope_table():
    t = f.Rope.table(7, 32, base=10000.0, device="cpu")
    assert t.shape == (7, 32) and t.dtype is torch.float32
    assert torch.equal(t[0], torch.cat((torch.ones(16), torch.zeros(16))))
    assert abs(float(t[3, 1]) - torch.cos(torch.tensor(3.0 * 10000.0 ** (-2 / 32), dtype=torch.float64)).item()) < 2 ** -24


def test_empty_tensors_do_nothing(lib):
    """No tokens, with and without queries, through the binding's own tensors (whose addresses are null)."""
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16)  # noqa: E731
    i32, i64 = (lambda *s: torch.zeros(*s, dtype=torch.int32)), torch.zeros(0, dtype=torch.int64)
    pool, s, t = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.ones(3, 2), torch.zeros(9, 64)
    b = f.load_binding()
    for q, out in ((None, None), (e(0, 4, 64), None), (e(0, 4, 64), e(0, 4, 64)), (e(9, 4, 64)[:0], None)):
        st, got = b.kv_rope_cache(0, q, e(0, 2, 64), e(0, 2, 64), i64, i64, t, 0, pool, pool, 0, s[0, :1], s[0, :1], 0, 0, None, 0, 0, out, None)
        assert st == f.OK and (got is None if q is None else got.shape == (0, 4, 64))
        for n, batch in ((0, 2), (0, 0)):
            st, got = b.kv_block_cache(0, e(n, 2, 64), e(n, 2, 64), i32(batch + 1), 3, pool, pool, s, s, i32(batch, 4), i32(batch), t, 0, q, out, None)
            assert st == f.OK and (got is None if q is None else got.shape == (0, 4, 64))
    assert b.fp8_block_prefill_attn(0, e(0, 4, 64), i32(3), 3, pool, pool, s, s, i32(2, 4), i32(2), 0.0, 1, 0, None, None)[0] == f.OK
    ws = torch.zeros(256, dtype=torch.uint8)
    assert b.fp8_block_decode_attn(0, e(0, 4, 64), pool, pool, s, s, i32(0, 4), i32(0), 0.0, 0, None, ws, None)[0] == f.OK
