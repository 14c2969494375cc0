"""The block-scaled attention when a wait of its pipeline runs out: reported, and the next call is sound.  The copies'
wait for a free stage is given less time than the pipeline takes, so that they stop in its midst; what waits for
them gives up after its own 200 ms."""
import pytest
import torch

from test_gpu_block_attn import Case, _i32

f = pytest.importorskip("fp8_kv_cache_quant_gb300")
pytestmark = pytest.mark.gpu


def _runs_out(call, ws=None):
    """call(fault) with the limit and without it, before and after."""
    lib = f.load_library()
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = call(fault)
    torch.cuda.synchronize()
    assert int(fault) == 0
    lib.fkv_set_decode_wait_limit_ns(1)
    try:
        for _ in range(2):
            call(fault)
        torch.cuda.synchronize()
    finally:
        lib.fkv_set_decode_wait_limit_ns(0)
    assert int(fault) == f.FAULT_TIMEOUT
    fault.zero_()
    for _ in range(2):
        assert torch.equal(call(fault), ref)
    assert int(fault) == 0
    if ws is not None:
        assert int(ws[:65536].count_nonzero()) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("g,window", [(4, 0), (8, 3000)])
def test_decode_wait_that_runs_out(d, g, window):
    """64 sequences over the same blocks, so that every CTA has more tiles than stages."""
    base = Case([4000], 2 * g, 2, d, seed=d)
    gen = torch.Generator().manual_seed(g)
    q = torch.randn(64, 2 * g, d, generator=gen).to(torch.bfloat16).cuda()
    cache, table, lens = base.cache(), _i32(base.table).expand(64, -1).contiguous(), _i32([4000 - 9 * b for b in range(63)] + [0])
    ws = f.block_decode_workspace(64, 2 * g, cache)
    _runs_out(lambda fault: f.fp8_block_decode_attn(q, cache, table, lens, window=window, workspace=ws, fault=fault), ws)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("ctx,new,h,window", [([1400] * 8, [400] * 8, 2, 0), ([9000], [9], 2, 0), ([9000, 1500], [60, 100], 1, 8000)])
def test_prefill_wait_that_runs_out(d, ctx, new, h, window):
    """Whole chunks, and few rows whose key tiles a cluster shares."""
    c = Case(ctx, 4, h, d, new=new, seed=d)
    q, cu, cache, table, lens = c.q.cuda(), _i32(c.cu), c.cache(), _i32(c.table), _i32(c.ctx)
    _runs_out(lambda fault: f.fp8_block_prefill_attn(q, cu, max(new), cache, table, lens, window=window, fault=fault))
