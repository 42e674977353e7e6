"""The calls of include/pa_serving.h without a GPU: declared, exported and bound,
and every refusal made on the host before any CUDA call."""
import os
import re

import numpy as np
import pytest
import torch

from paged_kv_cache_179_gb300 import _abi, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10008      # 16-byte aligned and not; never dereferenced
INV, UNS, WSP, OK = (_abi.PA_ERR_INVALID_ARG, _abi.PA_ERR_UNSUPPORTED, _abi.PA_ERR_WORKSPACE,
                     _abi.PA_OK)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def test_header_binding_and_library_agree(lib):
    text = open(os.path.join(ROOT, "include", "pa_serving.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text)))
    assert sorted(_abi.SERVING_SIGNATURES) == names and len(names) == 9
    for n in names:
        assert hasattr(lib, n), n
        # as many arguments as the declaration has
        decl = re.search(n + r"\s*\((.*?)\);", text, flags=re.S).group(1)
        assert len(_abi.SERVING_SIGNATURES[n][0]) == len(decl.split(",")), n


SPEC = _abi.RopeSpec(1e4 ** (-np.arange(32) / 32), np.arange(32) % 3)


def _rope(lib, **kw):
    a = dict(qo=FAKE, q=FAKE, qs=512, ko=FAKE, k=FAKE, ks=128, pos=FAKE, spec=SPEC, T=4, Hq=8,
             Hkv=2, D=64, dtype=0)
    a.update(kw)
    spec = a["spec"].pointer if a["spec"] is not None else None
    return lib.pa_rope(a["qo"], a["q"], a["qs"], a["ko"], a["k"], a["ks"], a["pos"], spec, a["T"],
                       a["Hq"], a["Hkv"], a["D"], a["dtype"], None)


def test_rope_refusals(lib):
    freq = SPEC.inv_freq
    assert _rope(lib, T=0, q=None) == OK                          # nothing to do
    assert _rope(lib, T=-1) == INV
    assert _rope(lib, spec=None) == INV
    assert _rope(lib, q=None) == INV
    assert _rope(lib, k=ODD) == INV
    assert _rope(lib, pos=None) == INV
    assert _rope(lib, qs=511) == INV                              # rows not 16-byte aligned
    assert _rope(lib, qs=504) == INV                              # tokens overlap
    assert _rope(lib, dtype=2) == INV
    assert _rope(lib, D=60) == UNS
    assert _rope(lib, D=264, qs=2112, ks=528) == UNS
    assert _rope(lib, D=56, qs=448, ks=112) == INV                # rotary_dim 64 > head_dim
    assert _rope(lib, qo=FAKE, q=FAKE, qs=1024) == INV            # in place needs a dense input
    S = _abi.RopeSpec
    assert _rope(lib, spec=S(freq[:4])) == INV                    # rotary_dim 8
    assert _rope(lib, spec=S(freq[:20])) == UNS                   # rotary_dim 40
    assert _rope(lib, spec=S(np.full(32, np.nan))) == INV
    assert _rope(lib, spec=S(np.full(32, np.inf))) == INV
    assert _rope(lib, spec=S(freq, amplitude=float("nan"))) == INV
    assert _rope(lib, spec=S(freq, np.full(32, 3), num_axes=3)) == INV
    assert _rope(lib, spec=S(freq, np.full(32, -1), num_axes=3)) == INV
    assert _rope(lib, spec=S(freq, num_axes=2)) == INV            # two axes, none assigned
    assert _rope(lib, spec=S(freq, np.zeros(32), num_axes=5)) == INV
    with pytest.raises(ValueError):
        S(freq, np.zeros(31))


def test_rope_append_refusals(lib):
    def call(fp8=False, **kw):
        a = dict(qo=FAKE, q=FAKE, qs=512, k=FAKE, ks=128, v=FAKE, vs=128, kc=FAKE, vc=FAKE,
                 sc=FAKE, slots=FAKE, pos=FAKE, T=4, Hq=8, Hkv=2, D=64, bs=16, NB=8, dtype=0)
        a.update(kw)
        head = [a["qo"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["kc"], a["vc"]]
        tail = [a["slots"], a["pos"], SPEC.pointer, a["T"], a["Hq"], a["Hkv"], a["D"], a["bs"],
                a["NB"], a["dtype"], None]
        if fp8:
            return lib.pa_rope_append_fp8(*head, a["sc"], a["sc"], *tail)
        return lib.pa_rope_append(*head, *tail)
    assert call(T=0, kc=None) == OK
    for fp8 in (False, True):
        for bad in (dict(slots=None), dict(kc=None), dict(v=ODD), dict(vs=120), dict(ks=132),
                    dict(bs=0), dict(NB=0), dict(Hkv=0), dict(dtype=2), dict(slots=FAKE + 4)):
            assert call(fp8, **bad) == INV, bad
    assert call(True, sc=None) == INV
    assert call(True, bs=32) == UNS
    assert call(True, T=2 ** 30) == UNS
    assert call(Hq=65534, qs=65534 * 64) == UNS                   # more rows a token than a CTA counts
    assert call(True, D=80, qs=640, ks=160, vs=160) == UNS


def test_attention_weights_refusals(lib):
    def call(fp8=False, **kw):
        a = dict(w=FAKE, st=128, q=FAKE, k=FAKE, ks=FAKE, bt=FAKE, mbs=8, cl=FAKE, mx=128, B=2,
                 Hq=8, Hkv=2, D=64, bs=16, NB=32, scale=.125, decay=1., fresh=0, nq=1, dtype=0,
                 ws=FAKE, n=1 << 20)
        a.update(kw)
        tail = [a["bt"], a["mbs"], a["cl"], a["mx"], a["B"], a["Hq"], a["Hkv"], a["D"], a["bs"],
                a["NB"], a["scale"], a["decay"], a["fresh"], a["nq"], a["dtype"], a["ws"], a["n"],
                None]
        if fp8:
            return lib.pa_attention_weights_fp8(a["w"], a["st"], a["q"], a["k"], a["ks"], *tail)
        return lib.pa_attention_weights(a["w"], a["st"], a["q"], a["k"], *tail)
    for fp8 in (False, True):
        assert call(fp8, B=0, w=None) == OK
        for bad in (dict(w=None), dict(q=ODD), dict(k=None), dict(Hq=7), dict(mx=129), dict(st=127),
                    dict(decay=float("nan")), dict(decay=-1.), dict(scale=float("inf")),
                    dict(fresh=-1), dict(nq=0), dict(nq=1025), dict(dtype=2), dict(NB=0),
                    dict(B=-1), dict(mbs=0)):
            assert call(fp8, **bad) == INV, bad
        for bad in (dict(D=96), dict(bs=32, mbs=4), dict(Hq=66)):
            assert call(fp8, **bad) == UNS, bad
        for bad in (dict(ws=None), dict(ws=FAKE + 16)):
            assert call(fp8, **bad) == WSP, bad
    assert call(True, ks=None) == INV
    assert call(mx=2 ** 30 + 1, st=2 ** 31, mbs=2 ** 27, n=1 << 62) == UNS   # indexes end at 2^30
    # 2^31 pages and more in one launch
    assert call(mx=2 ** 31 - 1, st=2 ** 31, mbs=2 ** 27, B=512, n=1 << 62) == UNS
    f = lib.pa_attention_weights_workspace_size
    assert f(2, 7, 2, 128, 1) == 0 and f(2, 8, 2, -1, 1) == 0 and f(2, 8, 2, 128, 0) == 0
    assert f(2, 8, 2, 128, 1) >= 2 * 2 * 8 * 512
    assert f(2, 8, 2, 128, 8) > f(2, 8, 2, 128, 4) > f(2, 8, 2, 128, 2)
    assert f(2, 8, 2, 128, 8) == f(2, 8, 2, 128, 800)


def test_evict_refusals(lib):
    def call(fp8=False, **kw):
        a = dict(k=FAKE, v=FAKE, sc=FAKE, w=FAKE, st=128, wo=FAKE + 4, os=40, bt=FAKE, mbs=8,
                 cl=FAKE, mx=128, sp=FAKE + 4, nsp=3, to=FAKE + 8, nl=FAKE + 4, kept=FAKE, B=2,
                 Hkv=2, D=64, bs=16, NB=32, keep=40, first=4, recent=8, dtype=0)
        a.update(kw)
        tail = [a["w"], a["st"], a["wo"], a["os"], a["bt"], a["mbs"], a["cl"], a["mx"], a["sp"],
                a["nsp"], a["to"], a["nl"], a["kept"], a["B"], a["Hkv"], a["D"], a["bs"], a["NB"],
                a["keep"], a["first"], a["recent"]]
        if fp8:
            return lib.pa_evict_fp8(a["k"], a["v"], a["sc"], a["sc"], *tail, None)
        return lib.pa_evict(a["k"], a["v"], *tail, a["dtype"], None)
    for fp8 in (False, True):
        assert call(fp8, B=0, k=None) == OK
        for bad in (dict(k=None), dict(v=ODD), dict(w=None), dict(keep=0), dict(first=-1),
                    dict(first=33), dict(recent=-1), dict(st=127), dict(os=39), dict(wo=FAKE),
                    dict(nsp=2), dict(nl=FAKE), dict(sp=FAKE), dict(to=FAKE), dict(to=FAKE + 4),
                    dict(kept=None), dict(nl=None), dict(mx=129), dict(B=-1), dict(NB=0),
                    dict(kept=FAKE + 2), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1)):
            assert call(fp8, **bad) == INV, bad
        for bad in (dict(D=96), dict(bs=32, mbs=4), dict(B=70000),
                    dict(mx=2 ** 30 + 1, st=2 ** 31, mbs=2 ** 27)):
            assert call(fp8, **bad) == UNS, bad
    assert call(dtype=2) == INV
    assert call(True, sc=None) == INV


def test_verify_refusals(lib):
    def call(**kw):
        a = dict(out=FAKE, acc=FAKE, p=FAKE, ps=1000, q=FAKE, qs=1000, x=FAKE, nd=FAKE, u=FAKE,
                 B=2, n=3, V=1000, dtype=3)
        a.update(kw)
        return lib.pa_verify_drafts(a["out"], a["acc"], a["p"], a["ps"], a["q"], a["qs"], a["x"],
                                    a["nd"], a["u"], a["B"], a["n"], a["V"], a["dtype"], None)
    assert call(B=0, p=None) == OK
    for bad in (dict(out=None), dict(acc=None), dict(p=None), dict(p=ODD), dict(q=ODD),
                dict(x=None), dict(u=None), dict(u=FAKE + 2), dict(B=-1), dict(n=-1), dict(n=1025),
                dict(V=0), dict(ps=999), dict(qs=999), dict(dtype=2), dict(dtype=4)):
        assert call(**bad) == INV, bad
    assert call(V=2 ** 24 + 1, ps=2 ** 25, qs=2 ** 25) == UNS
    assert call(B=2 ** 24 + 1) == UNS


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a CUDA device")
def test_valid_calls_without_device_report_cuda_error(lib):
    assert _rope(lib) == _abi.PA_ERR_CUDA


def test_bindings_refuse_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 8, 64, dtype=torch.float16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        _abi.pa_rope(x, x, None, None, i, SPEC)
    with pytest.raises(ValueError):
        _abi.pa_rope(None, None, None, None, i, SPEC)
    with pytest.raises(ValueError):
        _abi.pa_attention_weights(torch.zeros(4, 8, 64), x, x, i, i, 16, .1, None)
    with pytest.raises(ValueError):
        _abi.pa_evict(x, x, x, x, i, i, 16, i, i, i, i)
    with pytest.raises(TypeError):
        _abi.pa_verify_drafts(i, i, i, None, i, i)


def test_accumulate_refuses_a_step_whose_window_leaves_tokens_out(lib, monkeypatch):
    """The weights are those of the whole context, which is not what a windowed step
    attended; a window no shorter than the bound leaves nothing out."""
    from paged_kv_cache_179_gb300.step import DecodeStep
    pool = torch.zeros(8, 2, 16, 64, dtype=torch.float16)
    q, w = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 2, 64)

    def step(window):
        return DecodeStep(k_cache=pool, v_cache=pool, block_tables=torch.zeros(2, 4, dtype=torch.int32),
                          context_lens=torch.zeros(2, dtype=torch.int32), max_context_len=64, scale=.125,
                          num_q_heads=4, split_ctas=2, window=window)
    for window in (1, 16, 63):
        for x in (q, q[:, None].expand(2, 3, 4, 64).contiguous()):
            with pytest.raises(ValueError, match="whole context"):
                step(window).accumulate(w, x)
    made = []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(_abi, "alloc_weights_workspace", lambda *a: None)
    monkeypatch.setattr(_abi, "pa_attention_weights", lambda *a, **kw: made.append(kw))
    for window in (0, 64, 1000):
        step(window).accumulate(w, q, decay=.5)
    assert made == [dict(decay=.5, fresh_tokens=0)] * 3


def test_weights_timeout_hook(lib):
    """Declared in a header of its own, bound and exported; what it refuses on the host."""
    text = open(os.path.join(ROOT, "include", "pa_serving_test.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    decl = re.search(r"pa_test_weights_timeout\s*\((.*?)\);", text, flags=re.S).group(1)
    assert set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text)) == set(_abi.SERVING_TEST_SIGNATURES)
    assert len(_abi.SERVING_TEST_SIGNATURES["pa_test_weights_timeout"][0]) == len(decl.split(","))

    def call(**kw):
        a = dict(w=FAKE, st=8000, q=FAKE, k=FAKE, bt=FAKE, mbs=500, cl=FAKE, mx=5000, B=2, Hq=8, Hkv=2,
                 D=64, NB=32, scale=.125, dtype=0, silent=0, limit=1000, ws=FAKE, n=1 << 40)
        a.update(kw)
        return lib.pa_test_weights_timeout(
            a["w"], a["st"], a["q"], a["k"], a["bt"], a["mbs"], a["cl"], a["mx"], a["B"], a["Hq"],
            a["Hkv"], a["D"], a["NB"], a["scale"], a["dtype"], a["silent"], a["limit"], a["ws"],
            a["n"], None)
    for bad in (dict(limit=0), dict(limit=3_000_000_000), dict(B=0), dict(B=513), dict(silent=-1),
                dict(w=None), dict(q=ODD), dict(st=4999), dict(mx=8001)):
        assert call(**bad) == INV, bad
    for bad in (dict(mx=4096), dict(D=96), dict(Hq=66)):
        assert call(**bad) == UNS, bad
    assert call(ws=None) == WSP
