"""The launch forms of the calls in include/pa_serving.h that their sizes choose between:
prompts, evictions in two launches, every tile and pool of the attention weights in both
of their launches, calls at once on two streams.  Against the plain 64-bit statements."""
import numpy as np
import pytest
import torch

import _serving_ref as R
from paged_kv_cache_179_gb300 import _abi
from test_serving_gpu import (BF16, F16, evict_case, gen, ok, randn, rope_tol, run_evict,
                              run_weights, spec_for, weights_case)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rotation
# Up to twice as many tokens as SMs a CTA has 512 threads, above that 128; from eight
# times as many on it serves two tokens, unless they have more than 1024 rows each.
PROMPTS = [  # T, Hq, Hkv, D, rotary, axes, adjacent, dtype
    (400, 6, 2, 64, 64, 1, False, F16),
    (401, 28, 4, 128, 96, 3, True, BF16),
    (1501, 6, 2, 64, 64, 2, False, BF16),      # two tokens a CTA, the last one alone
    (1501, 3, 1, 128, 32, 3, True, F16),
    (2430, 1, 1, 72, 48, 1, False, F16),       # nine chunks a row
    (1499, 5, 0, 16, 16, 1, True, F16),        # q alone, one item a row
    (2431, 28, 4, 128, 128, 3, False, F16),
    (1217, 1300, 0, 16, 16, 1, False, F16),    # more rows than two tokens may have
]


def tokens_a_cta(T, rows):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 2 if rows > 1 and 4 * rows <= 4096 and T // 2 >= 4 * sms else 1


@pytest.mark.parametrize("T,Hq,Hkv,D,rotary,axes,adjacent,dtype", PROMPTS)
def test_rope_of_a_prompt(T, Hq, Hkv, D, rotary, axes, adjacent, dtype):
    assert T > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = gen(T + Hq)
    spec, inv, axis = spec_for(rotary // 2, axes, adjacent, 1.25)
    pos = torch.randint(0, 1 << 20, (axes, T), generator=g, dtype=torch.int32)
    x = randn(g, T, Hq + Hkv, D, dtype=dtype)
    d = x.cuda()
    qo = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    ko = torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
    _abi.pa_rope(qo, d[:, :Hq], ko if Hkv else None, d[:, Hq:] if Hkv else None, pos.cuda(), spec)
    ok()
    ref = R.rope(R.f64(x), pos.numpy(), inv, axis, adjacent, 1.25)
    got = np.concatenate([R.f64(qo), R.f64(ko)], 1)
    # positions are below 2^20: 2^-53 of the 64-bit reference's angle is nothing
    assert (np.abs(got - ref) <= rope_tol(R.f64(x), ref, dtype, 1.25)).all()
    assert torch.equal(d.cpu(), x)
    # in place (each side dense): the same bits
    q2 = x[:, :Hq].contiguous().cuda()
    _abi.pa_rope(q2, q2, None, None, pos.cuda(), spec)
    ok()
    assert torch.equal(q2, qo)


@pytest.mark.parametrize("T,bs,D,dtype", [(400, 16, 128, BF16), (1501, 16, 64, F16), (1502, 8, 72, BF16)])
def test_rope_append_of_a_prompt(T, bs, D, dtype):
    """Slots that append nothing, and one outside the pool, as the first and as the second
    token of a CTA."""
    Hq, Hkv = 6, 2
    if T > 1000:
        assert tokens_a_cta(T, Hq + 2 * Hkv) == 2
    g = gen(T)
    spec, _, _ = spec_for(32, 2, False)
    pos = torch.randint(0, 9000, (2, T), generator=g, dtype=torch.int32).cuda()
    qkv = randn(g, T, Hq + 2 * Hkv, D, dtype=dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g)[:T]
    for at in (0, 3, 10, 11, T - 1):
        slots[at] = -1 - at
    pools = [randn(g, NB, Hkv, bs, D, dtype=dtype).cuda() for _ in "kv"]
    for bad in (None, 20, 21):
        s = slots.clone()
        if bad is not None:
            s[bad] = NB * bs
        a, b = ([t.clone() for t in pools] for _ in "ab")
        qo, q2 = (torch.empty(T, Hq, D, dtype=dtype, device="cuda") for _ in "ab")
        kr = torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
        _abi.pa_rope_append(qo, q, k, v, *a, s.cuda(), pos, spec)
        if bad is None:
            ok()
        else:
            assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_SLOT)
            s[bad] = -1
        _abi.pa_rope(q2, q, kr, k, pos, spec)
        _abi.pa_cache_append(kr, v.contiguous(), *b, s.cuda())
        ok()
        assert torch.equal(qo, q2) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rope_append_fp8_of_many_tokens():
    T, Hq, Hkv, D = 1501, 6, 3, 64
    g = gen(7)
    spec, _, _ = spec_for(16, 2, False)
    state = [torch.zeros(T + 2, Hkv, 16, D, dtype=torch.uint8, device="cuda") for _ in "kv"] + \
        [torch.ones(T + 2, Hkv, device="cuda") for _ in "kv"]
    other = [t.clone() for t in state]
    page = torch.randperm(T + 2, generator=g)[:T]
    for row, size in ((0, 1.), (1, 4.), (2, .5)):
        qkv = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * size).to(BF16).cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.randint(0, 9000, (2, T), generator=g, dtype=torch.int32).cuda()
        slots = page * 16 + row
        slots[7::50] = -1
        slots = slots.cuda()
        qo, q2 = (torch.empty(T, Hq, D, dtype=BF16, device="cuda") for _ in "ab")
        kr = torch.empty(T, Hkv, D, dtype=BF16, device="cuda")
        _abi.pa_rope_append_fp8(qo, q, k, v, *state, slots, pos, spec)
        _abi.pa_rope(q2, q, kr, k, pos, spec)
        _abi.pa_cache_append_fp8(kr, v.contiguous(), *other, slots)
        ok()
        assert torch.equal(qo, q2) and all(torch.equal(x, y) for x, y in zip(state, other))
