"""The calls of include/pa_request.h without a GPU: declared, exported and bound, and every
refusal made on the host before any CUDA call."""
import ctypes
import os
import re

import pytest
import torch

from paged_kv_cache_179_gb300 import _abi, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = 0x10000, 0x10008      # 256-byte aligned and not; never dereferenced
INV, UNS, WSP, OK = (_abi.PA_ERR_INVALID_ARG, _abi.PA_ERR_UNSUPPORTED, _abi.PA_ERR_WORKSPACE,
                     _abi.PA_OK)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def test_header_binding_and_library_agree(lib):
    text = open(os.path.join(ROOT, "include", "pa_request.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text)))
    assert sorted(_abi.REQUEST_SIGNATURES) == names and len(names) == 9
    for n in names:
        assert hasattr(lib, n), n
        decl = re.search(n + r"\s*\((.*?)\);", text, flags=re.S).group(1)
        assert len(_abi.REQUEST_SIGNATURES[n][0]) == len(decl.split(",")), n
    # the specification's fields, in their order
    body = re.search(r"typedef struct pa_logits_spec \{(.*?)\}", text, flags=re.S).group(1)
    assert re.findall(r"(\w+);", body) == [f[0] for f in _abi._LogitsStruct._fields_]


def test_prefill_refusals(lib):
    def call(fp8=False, **kw):
        a = dict(out=FAKE, q=2 * FAKE, qs=512, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mbs=8, cl=FAKE, mx=128,
                 st=FAKE, T=10, B=2, Hq=8, Hkv=2, D=64, bs=16, NB=32, scale=.125, win=0, dtype=0, ws=FAKE,
                 n=1 << 40)
        a.update(kw)
        head = [a["out"], a["q"], a["qs"], a["k"], a["v"]] + ([a["ks"], a["vs"]] if fp8 else [])
        return (lib.pa_prefill_fp8 if fp8 else lib.pa_prefill)(
            *head, a["bt"], a["mbs"], a["cl"], a["mx"], a["st"], a["T"], a["B"], a["Hq"], a["Hkv"], a["D"],
            a["bs"], a["NB"], a["scale"], a["win"], a["dtype"], a["ws"], a["n"], None)
    for fp8 in (False, True):
        assert call(fp8, B=0, q=None) == OK and call(fp8, T=0, q=None) == OK
        for bad in (dict(out=None), dict(q=None), dict(q=ODD), dict(k=None), dict(v=ODD), dict(bt=None),
                    dict(cl=None), dict(st=None), dict(st=FAKE + 2), dict(qs=511), dict(qs=504), dict(Hq=7),
                    dict(B=-1), dict(T=-1), dict(mbs=0), dict(NB=0), dict(mx=-1), dict(mx=129), dict(win=-1),
                    dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=2), dict(out=FAKE, q=FAKE)):
            assert call(fp8, **bad) == INV, bad
        for bad in (dict(D=96, qs=768), dict(bs=32, mbs=4), dict(Hq=66, qs=66 * 64), dict(B=65536),
                    dict(T=2 ** 28), dict(mx=2 ** 30 + 1, mbs=2 ** 27)):
            assert call(fp8, **bad) == UNS, bad
        for bad in (dict(ws=None), dict(ws=FAKE + 16)):
            assert call(fp8, **bad) == WSP, bad
    assert call(True, ks=None) == INV and call(True, vs=FAKE + 2) == INV
    assert call(NB=2 ** 30) == UNS                                # 2^31 tiles
    f = lib.pa_prefill_workspace_size
    assert f(2, 10, 7, 2, 64) == 0 and f(-1, 10, 8, 2, 64) == 0 and f(2, 10, 8, 2, 80) == 0
    assert f(2, 10, 66, 2, 64) == 0


def test_failure_path_header_and_refusals(lib):
    text = open(os.path.join(ROOT, "include", "pa_request_test.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(pa_test_[a-z0-9_]+)\s*\(", text)))
    assert sorted(_abi.REQUEST_TEST_SIGNATURES) == names and len(names) == 1
    decl = re.search(names[0] + r"\s*\((.*?)\);", text, flags=re.S).group(1)
    assert len(_abi.REQUEST_TEST_SIGNATURES[names[0]][0]) == len(decl.split(","))

    def call(limit, T=10, B=2, drop=0):
        return lib.pa_test_prefill_timeout(FAKE, 2 * FAKE, 512, FAKE, FAKE, FAKE, 8, FAKE, 128, FAKE, T, B, 8, 2,
                                           64, 32, .125, 0, drop, limit, None, 0, None)
    assert call(0) == INV and call(2 * 10 ** 9 + 1) == INV and call(1000, T=0) == INV and call(1000, B=0) == INV
    assert call(1000, drop=-1) == INV
    assert call(1000) == WSP


def test_page_refusals(lib):
    def alloc(**kw):
        a = dict(bt=FAKE, mbs=8, np=FAKE, R=4, rows=FAKE, lens=FAKE, n=3, ref=FAKE, NB=32, bs=16, g=FAKE)
        a.update(kw)
        return lib.pa_alloc_pages(a["bt"], a["mbs"], a["np"], a["R"], a["rows"], a["lens"], a["n"], a["ref"],
                                  a["NB"], a["bs"], a["g"], None)

    def free(**kw):
        a = dict(bt=FAKE, mbs=8, np=FAKE, R=4, rows=FAKE, n=3, ref=FAKE, NB=32)
        a.update(kw)
        return lib.pa_free_pages(a["bt"], a["mbs"], a["np"], a["R"], a["rows"], a["n"], a["ref"], a["NB"], None)

    def fork(**kw):
        a = dict(k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE, mbs=8, np=FAKE, cl=FAKE, R=4, src=FAKE, dst=FAKE, n=3,
                 ref=FAKE, NB=32, Hkv=2, D=64, bs=16, type=0, g=FAKE)
        a.update(kw)
        return lib.pa_fork_pages(a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["mbs"], a["np"], a["cl"], a["R"],
                                 a["src"], a["dst"], a["n"], a["ref"], a["NB"], a["Hkv"], a["D"], a["bs"],
                                 a["type"], a["g"], None)

    def compact(**kw):
        a = dict(k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE, mbs=8, np=FAKE, R=4, ref=FAKE, NB=32, Hkv=2, D=64,
                 bs=16, type=0, to=FAKE, ro=FAKE, mv=2 * FAKE, nl=FAKE, ws=FAKE, wn=1 << 20)
        a.update(kw)
        return lib.pa_compact_pages(a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["mbs"], a["np"], a["R"], a["ref"],
                                    a["NB"], a["Hkv"], a["D"], a["bs"], a["type"], a["to"], a["ro"], a["mv"],
                                    a["nl"], a["ws"], a["wn"], None)
    for call in (alloc, free, fork):
        assert call(n=0, bt=None) == OK
        assert call(n=-1) == INV
    for call in (alloc, free, fork, compact):
        for bad in (dict(bt=None), dict(bt=FAKE + 2), dict(np=None), dict(ref=None), dict(ref=ODD), dict(mbs=0),
                    dict(R=0), dict(NB=0)):
            assert call(**bad) == INV, (call, bad)
        assert call(NB=2 ** 30 + 1) == UNS
    for bad in (dict(rows=None), dict(lens=None), dict(g=None), dict(rows=FAKE + 1)):
        assert alloc(**bad) == INV, bad
    assert alloc(bs=32) == UNS and alloc(n=32769) == UNS
    assert free(rows=None) == INV and free(n=2 ** 24 + 1) == UNS
    for bad in (dict(src=None), dict(dst=None), dict(cl=None), dict(g=None), dict(k=None), dict(v=ODD),
                dict(type=3), dict(type=2), dict(ks=FAKE), dict(Hkv=0)):
        assert fork(**bad) == INV, bad
    for call in (fork, compact):
        for bad in (dict(D=96), dict(bs=32), dict(Hkv=65536)):
            assert call(**bad) == UNS, bad
        assert call(type=2, ks=FAKE) == INV
    assert fork(n=32769) == UNS
    for bad in (dict(to=None), dict(ro=None), dict(mv=None), dict(nl=None), dict(mv=FAKE), dict(nl=FAKE + 1)):
        assert compact(**bad) == INV, bad
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(wn=100)):
        assert compact(**bad) == WSP, bad
    f = lib.pa_compact_workspace_size
    assert f(0) == 0 and f(-1) == 0 and f(2 ** 30 + 1) == 0 and f(1000) >= 8000


def test_logits_refusals(lib):
    def call(spec={}, **kw):
        a = dict(out=FAKE, os=1000, x=2 * FAKE, xs=1000, B=2, rows=1, V=1000, dtype=0, probs=0)
        a.update(kw)
        st = _abi._LogitsStruct(**spec)
        return lib.pa_process_logits(a["out"], a["os"], a["x"], a["xs"],
                                     None if spec is None else ctypes.c_void_p(ctypes.addressof(st)),
                                     a["B"], a["rows"], a["V"], a["dtype"], a["probs"], None)
    assert call(B=0, x=None) == OK
    assert lib.pa_process_logits(FAKE, 10, FAKE, 10, None, 1, 1, 10, 0, 0, None) == INV
    for bad in (dict(out=None), dict(out=ODD), dict(x=None), dict(x=ODD), dict(os=999), dict(xs=999), dict(B=-1),
                dict(rows=0), dict(rows=1026), dict(V=0), dict(dtype=2), dict(probs=2),
                dict(out=FAKE, x=FAKE, probs=1), dict(out=FAKE, x=FAKE, xs=1008)):
        assert call(**bad) == INV, bad
    for bad in (dict(V=2 ** 19 + 1, os=2 ** 20, xs=2 ** 20), dict(B=2 ** 24, rows=2)):
        assert call(**bad) == UNS, bad
    for bad in (dict(history=FAKE), dict(history=FAKE, history_lens=FAKE, history_stride=-1),
                dict(prompt_lens=FAKE), dict(bias_tokens=FAKE), dict(bias_values=FAKE), dict(num_bias=1),
                dict(num_bias=-1), dict(allowed=FAKE, allowed_stride=31), dict(temperature=FAKE + 2)):
        assert call(bad) == INV, bad
    assert call(dict(bias_tokens=FAKE, bias_values=FAKE, num_bias=1025)) == UNS
    assert call(dict(history=FAKE, history_lens=FAKE, history_stride=2 ** 30 + 1)) == UNS


def test_specification_refusals():
    t = torch.zeros(2, 3, dtype=torch.int32)
    for bad in (dict(history=t), dict(history_lens=t), dict(bias_tokens=t), dict(bias_values=t.float()),
                dict(prompt_lens=t[0])):
        with pytest.raises(ValueError):
            _abi.LogitsSpec(**bad)
    x = torch.zeros(2, 8)
    with pytest.raises((ValueError, TypeError)):
        _abi.pa_process_logits(x, x, _abi.LogitsSpec())       # not on a GPU
    with pytest.raises(TypeError):
        _abi.pa_process_logits(x, x, None)
