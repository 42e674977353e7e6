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


# ------------------------------------------------------------------ eviction
# A cut is moved within the selection's launch while keep x head_dim is at most 16384 a
# CTA of the unit (1, 2, 4 or 8 for bounds to 8192, 16384, 32768 and longer), else by a
# launch of its own; a selection over more than 65536 tokens reads its weights anew.
CUTS = [  # lens, Hkv, D, keep, first, recent, pool, kind; the last page of a cut is not full
    ([2000, 600, 40, 515], 2, 128, 515, 4, 100, "fp8", "random"),
    ([2000, 600, 40, 515], 2, 64, 515, 4, 100, "fp8", "ties"),
    ([1500, 129], 3, 128, 129, 0, 0, "fp8", "odd"),            # nine pages, the last of one row
    ([1500, 1023, 1024, 0], 2, 128, 1023, 4, 100, "16", "random"),
    ([1500, 1300], 1, 64, 1029, 0, 1029, "16", "random"),      # the recent ones alone
    ([900, 70], 2, 128, 131, 131, 0, "16", "ties"),            # the first ones alone
    ([30000, 20000], 1, 128, 777, 5, 20, "fp8", "odd"),        # four CTAs a unit
    ([9000, 8193], 1, 128, 401, 0, 7, "16", "equal"),          # two
    ([70000, 66000, 9], 1, 64, 2101, 1, 2, "16", "ties"),      # more than the registers hold
    ([70000, 65537], 1, 128, 1111, 3, 64, "fp8", "random"),
    ([66000, 900], 2, 64, 130, 3, 64, "fp8", "odd"),           # the same, moved within the selection
]


def moves_along(max_len, keep, D):
    cluster = 1
    while cluster < 8 and max_len > cluster * 8192:
        cluster *= 2
    return keep * D <= 16384 * cluster


def check_evict(got, pools, scales, w, bt, L, spare, keep, first, recent):
    p, s, w_out, tables, new, kept = got
    ref_new, ref_kept, ref_tables = R.evict(pools, scales, w.numpy(), bt, L.numpy(), spare, keep, first, recent)
    assert np.array_equal(new.cpu().numpy(), ref_new)
    assert torch.equal(tables.cpu(), ref_tables)
    kept, w_out = kept.cpu().numpy(), w_out.cpu().numpy()
    for (b, h), at in ref_kept.items():
        assert np.array_equal(kept[b, h, :len(at)], at) and (kept[b, h, len(at):] == -3).all()
        assert np.array_equal(w_out[b, h, :len(at)], w[b, h].numpy()[at], equal_nan=True)
        assert (w_out[b, h, len(at):] == -7).all()
    for a, b in zip(p, pools):                                  # whole pools, bit for bit
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
    for a, b in zip(s, scales):
        assert b is None or torch.equal(a.cpu(), b)


@pytest.mark.parametrize("lens,Hkv,D,keep,first,recent,pool,kind", CUTS)
def test_evict_in_two_launches(lens, Hkv, D, keep, first, recent, pool, kind):
    case = evict_case(lens, Hkv, D, keep, pool, F16, keep, kind)
    pools, scales, w, bt, L, spare = case
    assert moves_along(bt.shape[1] * 16, keep, D) == (keep == 130)
    check_evict(run_evict(*case, keep, first, recent), *case, keep, first, recent)
    ok()


def test_evict_forms_are_what_the_comment_says():
    """Of the cuts above, each of the two moves of either pool and head size, and all three
    selections of long and of short bounds, are made by some."""
    made = {(pool, D, moves_along(max(lens), keep, D)) for lens, _, D, keep, _, _, pool, _ in CUTS}
    assert {(pool, D, False) for pool in ("16", "fp8") for D in (64, 128)} <= made
    assert {moves_along(max(lens), keep, D) for lens, _, D, keep, *_ in CUTS if max(lens) > 65536} == {True, False}


@pytest.mark.parametrize("pool,D", [("16", 128), ("fp8", 64)])
def test_evict_in_two_launches_captured_and_on_another_stream(pool, D):
    """The move is a programmatic dependent of the selection: replayed from a graph, with
    other weights in the same tensors, and behind other work of its stream."""
    lens, Hkv, keep = [3000, 700, 610], 2, 613
    pools, scales, w, bt, L, spare = evict_case(lens, Hkv, D, keep, pool, F16, 5, "random")
    assert not moves_along(bt.shape[1] * 16, keep, D)
    d, sc = [t.cuda() for t in pools], [None if t is None else t.cuda() for t in scales]
    wd, btd, Ld, spd = w.cuda(), bt.cuda(), L.cuda(), spare.cuda()
    w_out = torch.empty(3, Hkv, keep + 3, device="cuda")
    tables, new = torch.empty_like(spd), torch.empty(3, dtype=torch.int32, device="cuda")
    kept = torch.empty(3, Hkv, keep, dtype=torch.int32, device="cuda")

    def call():
        args = (wd, w_out, btd, Ld, bt.shape[1] * 16, spd, tables, new, kept)
        kw = dict(first_tokens=3, recent_tokens=50)
        if pool == "16":
            _abi.pa_evict(*d, *args, **kw)
        else:
            _abi.pa_evict_fp8(*d, *sc, *args, **kw)

    def fresh(weights):
        for t, x in zip(d + [t for t in sc if t is not None], pools + [t for t in scales if t is not None]):
            t.copy_(x)
        wd.copy_(weights)
        for t, x in ((w_out, -7), (tables, -9), (new, -5), (kept, -3)):
            t.fill_(x)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    side = torch.cuda.Stream()
    for i, weights in enumerate((w, w.flip(-1).contiguous(), w)):
        fresh(weights)
        if i == 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                call()
            torch.cuda.current_stream().wait_stream(side)
        else:
            graph.replay()
        check_evict((d, sc, w_out, tables, new, kept), [t.clone() for t in pools],
                    [None if t is None else t.clone() for t in scales], weights, bt, L, spare, keep, 3, 50)
        ok()


@pytest.mark.parametrize("pool", ["16", "fp8"])
def test_evict_in_two_launches_skips_and_reports_bad_blocks(pool):
    keep = 611
    pools, scales, w, bt, L, spare = evict_case([1500, 900], 1, 64, keep, pool, F16, 6, "random")
    NB = pools[0].shape[0]
    want = [t.clone() for t in pools], [None if t is None else t.clone() for t in scales]
    R.evict(*want, w.numpy(), bt, L.numpy(), spare, keep, 0, 0)
    bad = spare.clone()
    bad[0, 1], bad[1, keep // 16] = NB, -1          # two pages that are not written
    p, s, _, tables, new, kept = run_evict(pools, scales, w, bt, L, bad, keep, 0, 0)
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_BLOCK)
    for got, start, full in zip(p, pools, want[0]):
        full = full.clone()
        for d in (spare[0, 1], spare[1, keep // 16]):
            full[int(d)] = start[int(d)]
        assert torch.equal(got.cpu(), full)
    assert new.tolist() == [keep, keep] and torch.equal(tables.cpu(), bad)
    none = bt.clone()
    none[1] = NB + 5                                # nothing of the second one can be read
    p, s, *_ = run_evict(pools, scales, w, none, L, spare, keep, 0, 0)
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_BLOCK)
    for got, start, full in zip(p, pools, want[0]):
        full = full.clone()
        full[spare[1].long()] = start[spare[1].long()]
        assert torch.equal(got.cpu(), full)


# ---------------------------------------------------------- attention weights
# Bounds up to 4096 take clusters, longer ones the cooperative launch; 8, 16 and 32 query
# rows, both head sizes, and four kinds of pool and query: 48 kernels.
@pytest.mark.parametrize("bound", [512, 5008])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pool,dtype", [("16", F16), ("16", BF16), ("fp8", F16), ("fp8", BF16)])
@pytest.mark.parametrize("group,n_q", [(7, 1), (5, 3), (7, 4)])
def test_attention_weights_of_every_kind(bound, D, pool, dtype, group, n_q):
    lens, Hkv = [500, 33, 0, 272, 2], 2
    q, kc, ks, bt, L, w = weights_case(lens, Hkv * group, Hkv, D, n_q, pool, dtype, D + group + n_q)
    wide = torch.full((len(lens), bound // 16), -1, dtype=torch.int32)
    wide[:, :bt.shape[1]] = bt
    w = torch.rand(len(lens), Hkv, bound + 4, generator=gen(3))
    scale = float(np.float32(D ** -.5))
    ref, tol = R.attention_weights(R.f64(w), R.f64(q), kc, ks, wide, L, scale, .5, n_q)
    got = R.f64(run_weights(q, kc, ks, wide, L, w, scale, .5, n_q))
    ok()
    assert (np.abs(got - ref) <= tol).all()
    assert np.array_equal(got[1, :, 33:], R.f64(w)[1, :, 33:])      # entries behind the context


# -------------------------------------------------------------- calls at once
def test_calls_at_once_on_two_streams():
    """Two long weights calls (cooperative launches) with a workspace each, an eviction and
    a verification, on two streams that do not wait for each other, many times over: each
    gives what it gives alone."""
    sides = []
    for i in range(2):
        lens, Hkv, D, keep = [20000 - 7000 * i, 300, 9000], 2, 64, 700
        q, kc, ks, bt, L, w = weights_case(lens, 8, Hkv, D, 1, "16", F16, 30 + i, garbage=False)
        nb, kb = kc.shape[0], (keep + 15) // 16
        room = torch.zeros(3 * kb, Hkv, 16, D, dtype=F16)
        spare = torch.arange(nb, nb + 3 * kb, dtype=torch.int32).view(3, kb)
        p = torch.softmax(torch.randn(5, 3, 33000, generator=gen(i)) * 3, -1)
        sides.append(dict(
            stream=torch.cuda.Stream(), mx=bt.shape[1] * 16, w=torch.zeros_like(w).cuda(), q=q.cuda(), bt=bt.cuda(),
            L=L.cuda(), k=torch.cat([kc, room]).cuda(), v=torch.cat([kc, room]).cuda(), spare=spare.cuda(),
            new=torch.empty(3, dtype=torch.int32, device="cuda"), p=p.cuda(), u=torch.rand(5, 3, generator=gen(i)).cuda(),
            kept=torch.empty(3, Hkv, keep, dtype=torch.int32, device="cuda"),
            x=torch.randint(0, 33000, (5, 2), generator=gen(i), dtype=torch.int32).cuda(),
            out=torch.empty(5, 3, dtype=torch.int32, device="cuda"), acc=torch.empty(5, dtype=torch.int32, device="cuda"),
            ws=_abi.alloc_weights_workspace(3, 8, Hkv, bt.shape[1] * 16, 1, "cuda")))

    def calls(s):
        for n in ("w", "kept", "out"):      # entries behind a sequence's own are left as they are
            s[n].zero_()
        _abi.pa_attention_weights(s["w"], s["q"], s["k"], s["bt"], s["L"], s["mx"], .125, s["ws"], decay=0.)
        _abi.pa_evict(s["k"], s["v"], s["w"], None, s["bt"], s["L"], s["mx"], s["spare"], None, s["new"], s["kept"],
                      first_tokens=2, recent_tokens=50)
        _abi.pa_verify_drafts(s["out"], s["acc"], s["p"], None, s["x"], s["u"])

    results = ("w", "k", "v", "new", "kept", "out", "acc")
    alone = []
    for s in sides:
        calls(s)
        ok()
        alone.append({n: s[n].clone() for n in results})
    torch.cuda.synchronize()
    for _ in range(50):
        for s in sides:
            with torch.cuda.stream(s["stream"]):
                calls(s)
    torch.cuda.synchronize()
    ok()
    for s, want in zip(sides, alone):
        for n in results:
            assert torch.equal(s[n], want[n]), n


# --------------------------------------------------------------- verification
def test_verify_shares_over_a_product_grid():
    """The first token out has the target's distribution, whatever the drafts: over every
    pair of an N x N grid of u's the shares are those of p to the grid's steps.  The
    acceptance of draft x is u q(x) < p(x): its share min(1, p(x) / q(x)) is met to 1 / N
    (N (+-1 / 2) of N points, and one more for a point on the border); a rejected row draws
    from the rest over the same even grid of the second u, each token to 1 / N again.
    Token t gets its share as a draft, weighted by q(t) (1 / N), and from the rejections, whose
    weights add up to at most 1 (the acceptances' 1 / N and the draw's 1 / N): 3 / N."""
    N, V = 64, 6
    p = torch.tensor([.4, .3, .15, .1, .05, 0.])
    q = torch.tensor([.05, .1, .15, .3, .1, .3])
    grid = (torch.arange(N) + .5) / N
    u = torch.cartesian_prod(grid, grid).cuda()
    count = torch.zeros(V, dtype=torch.float64)
    for x in range(V):
        out = torch.empty(N * N, 2, dtype=torch.int32, device="cuda")
        acc = torch.empty(N * N, dtype=torch.int32, device="cuda")
        _abi.pa_verify_drafts(out, acc, p.expand(N * N, 2, V).contiguous().cuda(),
                              q.expand(N * N, 1, V).contiguous().cuda(),
                              torch.full((N * N, 1), x, dtype=torch.int32, device="cuda"), u)
        ok()
        first = torch.bincount(out[:, 0].cpu().long(), minlength=V)
        assert first.sum() == N * N and first[5] == 0          # a token without weight is never drawn
        taken = int(acc.sum())
        assert abs(taken / N ** 2 - min(1., float(p[x] / q[x]))) <= 1 / N
        assert first[x] == taken or p[x] > q[x]                # a rejected draft is not drawn again
        count += float(q[x]) * first.double() / N ** 2
    assert (count - p.double()).abs().max() <= 3 / N
