"""The calls of include/pa_request.h captured behind other nodes than kernels: first in a graph,
behind a copy, and where two streams join."""
import numpy as np
import pytest
import torch

from paged_kv_cache_179_gb300 import _abi
from test_request_gpu import F16, Prompts, State, gen, i32, logits_case, ok, pools

pytestmark = pytest.mark.gpu


def prompt_call(fp8):
    p = Prompts([1300, 90], [60, 90], 8, 2, 64, F16, fp8)
    p.run()                                 # once, for the tensors
    dev, lens, qkv, ws = p.kept
    q = qkv[:, 64:9 * 64].unflatten(1, (8, 64))
    args = (dev["tables"], lens, p.mbs * 16, dev["starts"], p.scale, ws)
    if fp8:
        ks, vs = p.ks.cuda(), p.vs.cuda()
        return lambda: _abi.pa_prefill_fp8(p.out, q, dev["kc"], dev["vc"], ks, vs, *args), [p.out]
    return lambda: _abi.pa_prefill(p.out, q, dev["kc"], dev["vc"], *args), [p.out]


def page_call(which, NB):
    s = State([3, 4, 2, 5, 0, 0], NB, 10)
    data = [x.cuda() for x in pools(gen(3), NB, 2, 64, False)]
    t, pages, ref = s.dev
    start = [x.clone() for x in s.dev]
    L0, granted = i32([40, 60, 20, 80, 0, 0]), i32([9])
    L, moved, live = L0.clone(), torch.empty_like(ref), i32([0])
    ws = _abi.alloc_compact_workspace(NB, "cuda")
    rows, new, src, dst = i32([1]), i32([100]), i32([3]), i32([4])

    def call():
        for a, b in zip((*s.dev, L), (*start, L0)):
            a.copy_(b)                      # the same state before each
        if which == "free":
            _abi.pa_free_pages(t, pages, rows, ref)
        elif which == "alloc":
            _abi.pa_alloc_pages(t, pages, rows, new, ref, granted)
        elif which == "fork":
            _abi.pa_fork_pages(*data, t, pages, L, src, dst, ref, granted)
        else:
            _abi.pa_compact_pages(*data, t, pages, ref, t, ref, moved, live, ws)
    return call, [t, pages, ref, L]


def logits_call(rows):
    g = gen(4)
    spec = {k: None if v is None else v.cuda() for k, v in logits_case(g, rows, 0, 4000, 50, 3, True).items()}
    x, out = torch.randn(rows, 1, 4000, generator=g).cuda(), torch.zeros(rows, 1, 4000, device="cuda")
    ls = _abi.LogitsSpec(**spec)
    return lambda: _abi.pa_process_logits(out, x, ls, probs=True), [out]


CALLS = {"prefill": lambda: prompt_call(False), "prefill_fp8": lambda: prompt_call(True),
         "free": lambda: page_call("free", 64), "alloc": lambda: page_call("alloc", 64),
         "alloc_large": lambda: page_call("alloc", 20000), "fork": lambda: page_call("fork", 64),
         "compact": lambda: page_call("compact", 64), "compact_large": lambda: page_call("compact", 20000),
         "logits": lambda: logits_call(2), "logits_rows": lambda: logits_call(160)}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("behind", ["nothing", "copy", "join", "itself"])
def test_captured_behind(name, behind):
    call, outs = CALLS[name]()
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    a, b = torch.ones(1 << 16, device="cuda"), torch.zeros(1 << 16, device="cuda")
    graph, stream, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        if behind == "copy":
            b.copy_(a)
        elif behind == "join":
            side.wait_stream(stream)
            with torch.cuda.stream(side):
                b.copy_(a)
                b.mul_(2.)
            a.add_(1.)
            stream.wait_stream(side)
        elif behind == "itself":
            call()
        call()
    for _ in range(3):
        for x in outs:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ok()
        for x, y in zip(outs, want):
            assert np.array_equal(x.cpu().numpy(), y.cpu().numpy(), equal_nan=True)
