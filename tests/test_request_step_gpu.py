"""DecodeStep.prefill on the GPU: the same as the calls it makes, captured too.  A window of
the whole context."""
import pytest
import torch

import _serving_ref as R
from paged_kv_cache_179_gb300 import _abi
from paged_kv_cache_179_gb300.step import DecodeStep

pytestmark = pytest.mark.gpu


def setting(fp8, seed=3):
    g = torch.Generator().manual_seed(seed)
    lens, Hq, Hkv, D, mbs = [700, 90, 31], 8, 2, 64, 44
    tables, nb = R.tables_for(lens, mbs, g)
    if fp8:
        (kc, ks), (vc, vs) = (R.e4m3_pool(g, (nb, Hkv, 16, D)) for _ in "kv")
        pools = dict(k_cache=kc.cuda(), v_cache=vc.cuda(), k_scale=ks.cuda(), v_scale=vs.cuda())
    else:
        pools = dict(zip(("k_cache", "v_cache"), (torch.randn(nb, Hkv, 16, D, generator=g).half().cuda() for _ in "kv")))
    q = torch.randn(100 + 7 + 31, Hq, D, generator=g).half().cuda()
    starts = torch.tensor([0, 100, 107, 138], dtype=torch.int32, device="cuda")
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return pools, dict(block_tables=tables.cuda(), context_lens=L, max_context_len=mbs * 16, scale=.125,
                       num_q_heads=Hq), q, starts


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_step_prefill(fp8, window):
    pools, kw, q, starts = setting(fp8)
    want, out = torch.empty_like(q), torch.empty_like(q)
    ws = _abi.alloc_prefill_workspace(3, q.shape[0], 8, 2, 64, "cuda")
    args = (kw["block_tables"], kw["context_lens"], kw["max_context_len"], starts, kw["scale"], ws)
    if fp8:
        _abi.pa_prefill_fp8(want, q, *pools.values(), *args, window=window)
    else:
        _abi.pa_prefill(want, q, *pools.values(), *args, window=window)
    step = DecodeStep(**pools, **kw, window=window)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="before the capture"), torch.cuda.graph(graph):
        step.prefill(q, out, starts)
    torch.cuda.synchronize()
    step.prefill(q, out, starts)
    assert _abi.pa_get_status() == (0, 0) and torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.prefill(q, out, starts)
    out.zero_()
    graph.replay()
    assert _abi.pa_get_status() == (0, 0) and torch.equal(out, want)


@pytest.mark.parametrize("window", [704, 2 ** 31 - 1])
def test_a_window_of_the_whole_context_is_none(window):
    pools, kw, q, starts = setting(False)
    a, b = torch.empty_like(q), torch.empty_like(q)
    ws = _abi.alloc_prefill_workspace(3, q.shape[0], 8, 2, 64, "cuda")
    for out, w in ((a, 0), (b, window)):
        _abi.pa_prefill(out, q, *pools.values(), kw["block_tables"], kw["context_lens"], 704, starts, .125, ws, window=w)
    assert _abi.pa_get_status() == (0, 0) and torch.equal(a, b)
