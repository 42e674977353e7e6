"""The calls of include/pa_request.h on the GPU against their plain 64-bit statements."""
import numpy as np
import pytest
import torch

import _request_ref as Q
import _serving_ref as R
from paged_kv_cache_179_gb300 import _abi

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF_STEP = {F16: 2. ** -11, BF16: 2. ** -8, F32: 2. ** -24}


def ok():
    assert _abi.pa_get_status() == (0, 0)


def status(bits):
    rc, got = _abi.pa_get_status()
    assert rc == _abi.PA_ERR_BOUNDS and got == bits, (rc, got)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F16):
    return torch.randn(*shape, generator=g).to(dtype)


# ------------------------------------------------------------------- prefill
class Prompts:
    """Sequences of lens[b] cached tokens, news[b] of them queries."""

    def __init__(self, lens, news, Hq, Hkv, D, dtype=F16, fp8=False, window=0, seed=0, lead=0, behind=0,
                 spread=1.):
        g = self.g = gen(seed + sum(lens) + 7 * Hq + D)
        self.lens, self.news, self.dtype, self.fp8, self.window = list(lens), list(news), dtype, fp8, window
        self.Hq, self.Hkv, self.D, self.scale = Hq, Hkv, D, float(np.float32(D ** -.5))
        self.mbs = max(1, (max(lens) + 15) // 16)
        self.tables, self.NB = R.tables_for(lens, self.mbs, g)
        starts = lead + np.concatenate([[0], np.cumsum(news)])
        self.starts = torch.tensor(starts, dtype=torch.int32)
        self.T = int(starts[-1]) + behind
        # q is a view of one projection's output
        self.qkv = randn(g, self.T, (Hq + 2) * D, dtype=dtype)
        self.q = self.qkv[:, D:(Hq + 1) * D].unflatten(1, (Hq, D))
        self.ks = self.vs = None
        if fp8:
            self.kc, self.ks = R.e4m3_pool(g, (self.NB, Hkv, 16, D))
            self.vc, self.vs = R.e4m3_pool(g, (self.NB, Hkv, 16, D))
            if spread != 1.:            # page scales that lie far apart
                f = torch.exp2(torch.randint(-12, 1, self.vs.shape, generator=g).float()) * spread
                self.vs = self.vs * f
        else:
            self.kc, self.vc = (randn(g, self.NB, Hkv, 16, D, dtype=dtype) for _ in "kv")
        # what no query may see: the rows behind each context
        for b, L in enumerate(lens):
            if L % 16:
                p = int(self.tables[b, L // 16])
                for t in (self.kc, self.vc):
                    t[p, :, L % 16:] = 0x7f if fp8 else float("nan")

    def run(self, out=None, prepared=False, ws=None):
        dev = {n: getattr(self, n).cuda() for n in ("kc", "vc", "tables", "starts")}
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        qkv = self.qkv.cuda()
        q = qkv[:, self.D:(self.Hq + 1) * self.D].unflatten(1, (self.Hq, self.D))
        if out is None:
            out = torch.full((self.T, self.Hq, self.D), 7., dtype=self.dtype, device="cuda")
        if ws is None:
            ws = _abi.alloc_prefill_workspace(len(self.lens), self.T, self.Hq, self.Hkv, self.D, "cuda")
            ws.fill_(255)               # of any contents
        mx = getattr(self, "max_context", self.mbs * 16)
        args = (dev["tables"], lens, mx, dev["starts"], self.scale, ws)
        if self.fp8:
            call = lambda: _abi.pa_prefill_fp8(out, q, dev["kc"], dev["vc"], self.ks.cuda(),  # noqa: E731
                                               self.vs.cuda(), *args, window=self.window)
        else:
            call = lambda: _abi.pa_prefill(out, q, dev["kc"], dev["vc"], *args, window=self.window)  # noqa: E731
        call()
        self.call, self.out, self.kept = call, out, (dev, lens, qkv, ws)
        return out

    def check(self, out):
        before = np.full((self.T, self.Hq, self.D), 7.)
        clean = self.vc.clone()
        ref, mass, big = Q.prefill(before, R.f64(self.q), self.kc, clean, self.ks, self.vs, self.tables.numpy(),
                                   self.lens, self.starts.numpy(),
                                   getattr(self, "max_context", self.mbs * 16), self.scale, self.window)
        f16_products = self.fp8 or self.dtype == F16
        tol = Q.prefill_tol(ref, mass, big, HALF_STEP[self.dtype], 2. ** -11 if f16_products else 2. ** -8)
        if f16_products:                # weights below fp16's normal range: 2^-31 each of the largest value
            v = R.f64(self.vc.view(torch.float8_e4m3fn).float()) * R.f64(self.vs)[:, :, None, None] if self.fp8 \
                else R.f64(self.vc)
            tol = tol + max(self.lens) * 2. ** -31 * np.nanmax(np.abs(np.where(np.isfinite(v), v, 0)), initial=0.)
        got = R.f64(out)
        same = np.isnan(ref) & np.isnan(got) | (ref == got)
        bad = ~same & ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


PROMPTS = [  # lens, news, Hq, Hkv, D, dtype, fp8, window
    ([1], [1], 1, 1, 64, F16, False, 0),
    ([5], [5], 8, 2, 64, F16, False, 0),
    ([1, 17, 100, 256], [1, 17, 33, 0], 8, 2, 64, F16, False, 0),
    ([129, 128, 127], [129, 128, 127], 4, 4, 128, BF16, False, 0),
    ([300, 40, 16, 700], [1, 40, 3, 130], 28, 4, 128, F16, False, 0),
    ([513, 2], [200, 1], 14, 2, 128, BF16, False, 0),
    ([1000], [77], 15, 5, 64, BF16, False, 0),
    ([700], [5], 32, 1, 128, F16, False, 0),            # one kv head, 32 query heads
    ([260], [260], 31, 1, 64, F16, False, 0),
    ([640, 33], [300, 33], 6, 2, 128, F16, False, 50),  # a window inside one tile
    ([900, 1200], [128, 700], 7, 1, 128, BF16, False, 300),
    ([400], [400], 2, 2, 64, F16, False, 1),            # each query sees itself alone
    ([3, 20], [9, 25], 4, 2, 64, F16, False, 0),        # queries before position 0
    ([0, 50, 0], [0, 10, 4], 4, 2, 128, F16, False, 0),  # empty contexts
    ([2100], [9], 8, 1, 128, F16, False, 0),            # few rows, a long context
    ([3000, 2500], [1, 2], 28, 4, 128, BF16, False, 0),
    ([256, 100], [100, 100], 8, 2, 64, F16, True, 0),
    ([300, 40, 16, 700], [1, 40, 3, 130], 28, 4, 128, BF16, True, 0),
    ([130, 513], [130, 200], 5, 5, 128, F16, True, 0),
    ([900, 1200], [128, 300], 7, 1, 128, BF16, True, 300),
    ([2100, 1], [6, 1], 8, 2, 64, BF16, True, 0),
    ([1500], [1500], 7, 1, 128, BF16, False, 0),        # whole tiles, cut items
    ([1400, 1300], [1, 1300], 3, 1, 64, F16, False, 0),
    ([1700], [900], 10, 2, 128, F16, True, 0),
    ([1600], [700], 4, 1, 64, BF16, True, 1000),        # a window over whole tiles
    ([1999], [1300], 5, 1, 128, F16, False, 777),
    ([129] * 40, [2] * 40, 12, 12, 64, F16, False, 0),
]


@pytest.mark.parametrize("lens,news,Hq,Hkv,D,dtype,fp8,window", PROMPTS)
def test_prefill(lens, news, Hq, Hkv, D, dtype, fp8, window):
    p = Prompts(lens, news, Hq, Hkv, D, dtype, fp8, window)
    out = p.run()
    ok()
    p.check(out)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_leaves_tokens_of_no_sequence_alone(fp8):
    p = Prompts([70, 20], [30, 20], 8, 2, 64, F16, fp8, lead=3, behind=5)
    out = p.run()
    ok()
    assert bool((out[:3] == 7).all()) and bool((out[-5:] == 7).all())
    p.check(out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6])
def test_prefill_passes_over_invalid_pages(fp8, bad):
    p = Prompts([200, 300, 30], [60, 40, 30], 8, 2, 128, F16, fp8)
    p.tables[0, 3] = bad
    p.tables[0, 12] = bad                   # the last one
    p.tables[1, :9] = bad                   # a whole tile
    p.tables[2, :] = bad                    # everything: zeros
    out = p.run()
    status(_abi.PA_STATUS_BAD_BLOCK)
    p.check(out)
    assert bool((out[100:130] == 0).all())


def test_prefill_bad_lengths_and_starts():
    p = Prompts([100, 50, 60, 30], [20, 10, 10, 5], 8, 2, 64)
    p.lens[1], p.lens[2] = -3, 10 ** 6
    out = p.run()
    status(_abi.PA_STATUS_BAD_LEN)
    p.lens[2] = p.mbs * 16 + 1
    p.check(out)
    p = Prompts([100, 50, 60], [20, 10, 10], 8, 2, 64)
    p.starts = torch.tensor([0, 20, 15, 999], dtype=torch.int32)
    out = p.run()
    status(_abi.PA_STATUS_BAD_LEN)
    assert bool((out[20:] == 7).all())
    p.starts = torch.tensor([0, 20, 20, 20], dtype=torch.int32)
    p.check(out)


@pytest.mark.parametrize("dtype,value", [(F16, float("nan")), (F16, float("inf")), (BF16, float("-inf"))])
@pytest.mark.parametrize("where", ["k", "v"])
def test_prefill_masked_values_do_not_matter(dtype, value, where):
    """A token's key or value that is not a number reaches the queries from its position on
    (and, with a window, up to where it leaves it), and no other."""
    for window in (0, 60):
        p = Prompts([330, 64], [200, 64], 6, 2, 128, dtype, window=window)
        at = 290
        (p.kc if where == "k" else p.vc)[int(p.tables[0, at // 16]), 1, at % 16, 5] = value
        clean = Prompts([330, 64], [200, 64], 6, 2, 128, dtype, window=window)
        got, want = p.run(), clean.run()
        ok()
        n = at - (330 - 200)                # query n is the first that sees it
        last = 200 if not window else min(200, n + window)
        sees = np.zeros((p.T, 6), dtype=bool)
        sees[n:last, 3:] = True
        got, want = R.f64(got), R.f64(want)
        assert np.isfinite(got[~sees]).all()
        if where == "k":
            assert np.array_equal(got[~sees], want[~sees])
        else:                               # (that tile's products are summed in another order: within the
            #                                  tolerance of the definition, not bit by bit)
            assert not np.isfinite(got[sees][:, 5]).any()
            rest = np.delete(np.arange(128), 5)
            clean.check(torch.from_numpy(np.where(sees[..., None] & (np.arange(128) == 5), want, got)))
            assert np.isfinite(got[sees][:, rest]).all()


def test_prefill_large_logits_and_scales():
    """Logits that differ by thousands, a negative and a zero scale."""
    for scale in (4., -1., 0., 1e-6):
        p = Prompts([400, 130], [140, 130], 4, 2, 128, BF16)
        p.qkv *= 4
        p.scale = scale
        out = p.run()
        ok()
        p.check(out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prefill_weights_that_outgrow_their_offset(fp8, dtype):
    """Scores that rise by hundreds in the middle of a long context, in the first half of a
    tile and in the second, after the offset has stood for many tiles; and one key that
    outweighs all others by more than the products' range."""
    for at in (700, 780, 1155):
        p = Prompts([1300], [100], 4, 2, 128, dtype, fp8)
        for page in range(at // 16, 81):
            k = p.kc[int(p.tables[0, page])]
            if fp8:
                p.ks[int(p.tables[0, page])] *= 40
            else:
                k *= 40
        out = p.run()
        ok()
        p.check(out)
    p = Prompts([1300], [100], 2, 1, 64, dtype, fp8)
    if fp8:
        p.ks[int(p.tables[0, 50])] *= 300
    else:
        p.kc[int(p.tables[0, 50]), 0, 5] *= 300
    out = p.run()
    ok()
    p.check(out)


def test_prefill_not_finite_in_long_contexts():
    """A key or value that is not a number, far from any edge: the queries get what the
    definition says, nothing hangs and other sequences do not notice."""
    for where, value in (("k", float("nan")), ("k", float("inf")), ("v", float("inf"))):
        p = Prompts([1300, 200], [60, 50], 4, 2, 128, F16)
        clean = Prompts([1300, 200], [60, 50], 4, 2, 128, F16)
        (p.kc if where == "k" else p.vc)[int(p.tables[0, 30]), 1, 3, 7] = value
        got, want = R.f64(p.run()), R.f64(clean.run())
        ok()
        assert np.array_equal(got[60:], want[60:]) and np.array_equal(got[:60, :2], want[:60, :2])
        if where == "v":
            assert not np.isfinite(got[:60, 2:, 7]).any()
        elif value != value:
            assert np.isnan(got[:60, 2:]).all()


def test_prefill_page_scales_far_apart():
    for spread in (1e-3, 30.):
        p = Prompts([700], [200], 8, 2, 128, BF16, True, spread=spread)
        out = p.run()
        ok()
        p.check(out)


def test_prefill_rising_logits():
    """Each key beats all before it, so every running maximum moves at every step."""
    p = Prompts([600], [300], 2, 1, 64, F16)
    rise = torch.linspace(0.01, 12, 608).view(38, 16)
    for j in range(38):
        p.kc[int(p.tables[0, j]), 0] = (rise[j, :, None] * torch.ones(64)).half()
    p.qkv.fill_(1.)
    p.q = p.qkv[:, 64:192].unflatten(1, (2, 64))
    out = p.run()
    ok()
    p.check(out)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_equals_decode_at_one_token(fp8):
    """Against the decode step's own kernel: one query token a sequence."""
    p = Prompts([100, 700, 33], [1, 1, 1], 28, 4, 128, F16, fp8)
    out = p.run()
    q = p.q.contiguous().cuda()
    got = torch.empty_like(q)
    ws = _abi.alloc_workspace(3, 28, 128, 0, "cuda")
    lens = torch.tensor(p.lens, dtype=torch.int32).cuda()
    if fp8:
        _abi.pa_decode_fp8(got, q, p.kc.cuda(), p.vc.cuda(), p.ks.cuda(), p.vs.cuda(), p.tables.cuda(), lens,
                           p.mbs * 16, p.scale, 0, ws)
    else:
        _abi.pa_decode(got, q, p.kc.cuda(), p.vc.cuda(), p.tables.cuda(), lens, p.mbs * 16, p.scale, 0, ws)
    ok()
    # Both round the definition's value once, after weights that are off by 2^-11 at most: 16-bit pools
    # hold values of order one (results below 4: a step of 2^-9, weights 2^-11 of 4, each twice);
    # the E4M3 pools' values reach 14, where fp16's step is 2^-7 and 2^-11 of them as much again.
    diff = float((got.double() - out.double()).abs().max())
    assert diff <= (3e-2 if fp8 else 6e-3)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_captured_and_repeated(fp8):
    """A captured call replays with the lengths, tables and queries of the moment, and gives
    the same bits each time."""
    p = Prompts([700, 90, 300], [200, 90, 1], 14, 2, 128, BF16, fp8)
    p.run()
    first = p.out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    dev, lens, qkv, ws = p.kept
    ks, vs = (p.ks.cuda(), p.vs.cuda()) if fp8 else (None, None)
    q = qkv[:, 128:15 * 128].unflatten(1, (14, 128))
    args = (dev["tables"], lens, p.mbs * 16, dev["starts"], p.scale, ws)
    with torch.cuda.graph(graph):
        if fp8:
            _abi.pa_prefill_fp8(p.out, q, dev["kc"], dev["vc"], ks, vs, *args)
        else:
            _abi.pa_prefill(p.out, q, dev["kc"], dev["vc"], *args)
    for _ in range(3):
        p.out.fill_(7.)
        graph.replay()
        assert torch.equal(p.out, first)
    lens.copy_(torch.tensor([650, 80, 290], dtype=torch.int32))
    dev["starts"].copy_(torch.tensor([0, 10, 90, 291], dtype=torch.int32))
    p.out.fill_(7.)
    graph.replay()
    ok()
    p.lens, p.starts = [650, 80, 290], dev["starts"].cpu()
    p.check(p.out)


def test_prefill_on_another_stream_and_two_at_once():
    a = Prompts([900, 40], [300, 40], 8, 2, 128, F16)
    b = Prompts([500, 600], [500, 2], 8, 2, 128, F16, True)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    a.run(), b.run()                        # once, for the tensors
    torch.cuda.synchronize()
    a.out.fill_(7.), b.out.fill_(7.)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s):
            a.call()
        with torch.cuda.stream(t):
            b.call()
    torch.cuda.synchronize()
    ok()
    a.check(a.out)
    b.check(b.out)


def test_prefill_more_sequences_than_one_launch_sorts():
    n = 1500
    g = gen(5)
    lens = torch.randint(1, 40, (n,), generator=g).tolist()
    news = [min(x, int(torch.randint(0, 6, (1,), generator=g))) for x in lens]
    p = Prompts(lens, news, 2, 1, 64)
    out = p.run()
    ok()
    p.check(out)


# --------------------------------------------------------------------- pages
class State:
    """Rows of ``held`` pages each, in a pool of NB; ``shared``: rows that begin with the first
    row's pages."""

    def __init__(self, held, NB, mbs, seed=0, shared=()):
        g = gen(seed + NB)
        self.tables = torch.full((len(held), mbs), -1, dtype=torch.int32)
        perm = torch.randperm(NB, generator=g).to(torch.int32)
        c = 0
        for r, n in enumerate(held):
            self.tables[r, :n] = perm[c:c + n]
            c += n
        for r in shared:
            self.tables[r, :min(held[0], held[r])] = self.tables[0, :min(held[0], held[r])]
        self.held = torch.tensor(held, dtype=torch.int32)
        self.ref = torch.zeros(NB, dtype=torch.int32)
        for r, n in enumerate(held):
            for p in self.tables[r, :n].tolist():
                self.ref[p] += 1
        self.host = Q.Pages(self.tables, self.held, self.ref)
        self.dev = [x.cuda() for x in (self.tables, self.held, self.ref)]

    def same(self):
        for got, want in zip(self.dev, (self.host.tables, self.host.held, self.host.ref)):
            assert np.array_equal(got.cpu().numpy(), want)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("NB", [7, 64, 1021, 70001, 1 << 20])
def test_alloc_and_free(NB):
    n = min(NB // 3, 50)
    s = State([1] * n + [0] * 4, NB, max(8, min(NB // 2, 40000)), shared=range(1, min(3, n)))
    rows = [n, 0, n + 1, n + 3, n - 1]
    lens = [16 * min(NB // 4, 40000), 1, 17, 0, 33]
    granted = i32([9] * 5)
    t, held, ref = s.dev
    _abi.pa_alloc_pages(t, held, i32(rows), i32(lens), ref, granted)
    ok()
    assert granted.tolist() == s.host.alloc(rows, lens)
    s.same()
    _abi.pa_free_pages(t, held, i32([n, n, 1, n + 2]), ref)      # one listed twice, an empty one
    ok()
    s.host.free([n, 1, n + 2])
    s.same()


def test_alloc_stops_where_the_pool_ends():
    s = State([2, 3, 1, 0, 0, 0], 20, 16)
    rows, lens = [3, 4, 5, 0], [16 * 5, 16 * 10, 16, 32]
    granted = i32([9] * 4)
    t, held, ref = s.dev
    _abi.pa_alloc_pages(t, held, i32(rows), i32(lens), ref, granted)
    ok()
    # 14 free: 5, then 10 are not there; those behind get nothing, even where they need nothing
    assert granted.tolist() == [1, 0, 0, 0] == s.host.alloc(rows, lens)
    s.same()
    _abi.pa_alloc_pages(t, held, i32([4]), i32([16 * 9]), ref, granted[:1].clone())
    s.host.alloc([4], [16 * 9])
    s.same()
    assert int((ref == 0).sum()) == 0
    _abi.pa_alloc_pages(t, held, i32([5, 0]), i32([0, 30]), ref, granted[:2])   # need nothing
    ok()
    assert granted.tolist()[:2] == [1, 1]


def test_alloc_many_rows():
    n = 5000
    g = gen(3)
    s = State([0] * n, 40000, 20)
    rows = torch.randperm(n, generator=g).tolist()
    lens = torch.randint(0, 16 * 20 + 1, (n,), generator=g).tolist()
    granted = i32([9] * n)
    t, held, ref = s.dev
    _abi.pa_alloc_pages(t, held, i32(rows), i32(lens), ref, granted)
    ok()
    assert granted.tolist() == s.host.alloc(rows, lens)
    assert 0 < sum(granted.tolist()) < n
    s.same()


def test_alloc_as_many_items_as_a_call_takes():
    n = 32768
    s = State([0] * n, 40000, 2)
    granted = i32([9] * n)
    t, held, ref = s.dev
    rows = torch.arange(n - 1, -1, -1, dtype=torch.int32)
    lens = torch.full((n,), 7, dtype=torch.int32)
    _abi.pa_alloc_pages(t, held, rows.cuda(), lens.cuda(), ref, granted)
    ok()
    assert bool((granted == 1).all()) and torch.equal(t[:, 0].cpu(), rows)
    assert bool((ref[:n] == 1).all()) and bool((ref[n:] == 0).all())


def test_page_calls_pass_over_bad_items():
    s = State([2, 3, 1, 0], 40, 4)
    t, held, ref = s.dev
    granted = i32([9] * 5)
    _abi.pa_alloc_pages(t, held, i32([3, 4, 0, -1, 2]), i32([30, 10, 40, 10, 20]), ref, granted)
    status(_abi.PA_STATUS_BAD_ROW)
    assert granted.tolist() == [1, 0, 1, 0, 1] == s.host.alloc([3, 4, 0, -1, 2], [30, 10, 40, 10, 20])
    s.same()
    _abi.pa_alloc_pages(t, held, i32([3, 0]), i32([65, -1]), ref, granted[:2])
    status(_abi.PA_STATUS_BAD_LEN)
    assert granted.tolist()[:2] == [0, 0]
    s.same()
    _abi.pa_free_pages(t, held, i32([7, -2 ** 31, 1]), ref)
    status(_abi.PA_STATUS_BAD_ROW)
    s.host.free([1])
    s.same()
    # entries that are no page, or of a free one
    t[0, 0] = 999
    t[0, 1] = int((ref == 0).nonzero()[0])
    s.host.tables = t.cpu().numpy().astype(np.int64)
    _abi.pa_free_pages(t, held, i32([0]), ref)
    status(_abi.PA_STATUS_BAD_BLOCK)
    s.host.free([0])
    s.same()
    held[2] = 5                              # more than a row has
    _abi.pa_free_pages(t, held, i32([2]), ref)
    status(_abi.PA_STATUS_BAD_LEN)
    assert held.tolist()[2] == 5


def pools(g, NB, Hkv, D, fp8, dtype=F16):
    if fp8:
        (kc, ks), (vc, vs) = (R.e4m3_pool(g, (NB, Hkv, 16, D)) for _ in "kv")
        return [kc, vc, ks, vs]
    return [randn(g, NB, Hkv, 16, D, dtype=dtype) for _ in "kv"]


def scales(dev):
    return dict(k_scale=dev[2], v_scale=dev[3]) if len(dev) == 4 else {}


@pytest.mark.parametrize("Hkv,D,fp8", [(1, 64, False), (4, 128, False), (5, 64, True), (8, 128, True), (40, 128, False)])
def test_fork(Hkv, D, fp8):
    g = gen(Hkv + D)
    lens = [100, 16, 1, 0, 250, 33, 7, 64, 5]
    held = [7, 2, 1, 0, 16, 3, 1, 5, 1]       # some hold more than their context
    s = State(held, 60, 16, shared=[7])
    data = pools(g, 60, Hkv, D, fp8)
    dev = [x.cuda() for x in data]
    L = i32(lens)
    src, dst = [0, 0, 7, 4, 3, 1], [2, 5, 6, 8, 1, 3]
    src, dst = src[:5], dst[:5]
    t, pages, ref = s.dev
    granted = i32([9] * 5)
    _abi.pa_free_pages(t, pages, i32(dst), ref)
    s.host.free(dst)
    _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, i32(src), i32(dst), ref, granted, **scales(dev))
    ok()
    host_lens = list(lens)
    assert granted.tolist() == s.host.fork(src, dst, host_lens, data) == [1] * 5
    assert L.tolist() == host_lens
    s.same()
    for a, b in zip(dev, data):
        assert torch.equal(a.cpu(), b)


def test_fork_many_of_one_and_pool_ends():
    g = gen(8)
    s = State([3] + [0] * 30, 22, 6)
    data = pools(g, 22, 2, 64, False, BF16)
    dev = [x.cuda() for x in data]
    lens = [40] + [5] * 30
    L = i32(lens)
    dst = list(range(30, 0, -1))
    t, pages, ref = s.dev
    granted = i32([9] * 30)
    _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, i32([0] * 30), i32(dst), ref, granted)
    ok()
    assert granted.tolist() == s.host.fork([0] * 30, dst, lens, data) == [1] * 19 + [0] * 11
    assert L.tolist() == lens
    s.same()
    for a, b in zip(dev, data):
        assert torch.equal(a.cpu(), b)
    # a full last page needs none: granted while nothing before it failed
    L[0] = 32
    lens[0] = 32
    _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, i32([0, 0]), i32([1, 2]), ref, granted[:2])
    ok()
    assert granted.tolist()[:2] == s.host.fork([0, 0], [1, 2], lens, data) == [1, 1]
    s.same()


def test_fork_passes_over_bad_pairs():
    g = gen(9)
    s = State([2, 2, 2, 0, 0, 0], 30, 4)
    data = pools(g, 30, 2, 64, False)
    dev = [x.cuda() for x in data]
    t, pages, ref = s.dev
    lens = [20, 33, -1, 0, 0, 0]              # the second's is beyond what it holds
    L = i32(lens)
    src, dst = [0, 1, 2, 9, 0, 0, 0], [3, 4, 5, 4, -1, 0, 6]
    granted = i32([9] * 7)
    _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, i32(src), i32(dst), ref, granted)
    status(_abi.PA_STATUS_BAD_ROW | _abi.PA_STATUS_BAD_LEN)
    assert granted.tolist() == s.host.fork(src, dst, lens, data) == [1, 0, 0, 0, 0, 0, 0]
    s.same()
    t[1] = i32([500, -1, -1, -1])             # entries outside the pool are taken over as they are
    L[1] = 20
    s.host.tables[1], lens[1] = [500, -1, -1, -1], 20
    _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, i32([1]), i32([4]), ref, granted[:1])
    status(_abi.PA_STATUS_BAD_BLOCK)
    assert s.host.fork([1], [4], lens, data) == [1]
    s.same()
    for a, b in zip(dev, data):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("NB,Hkv,D,fp8", [(9, 2, 64, False), (64, 1, 64, True), (300, 5, 128, False),
                                          (1030, 3, 128, True), (9001, 2, 64, True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(NB, Hkv, D, fp8, in_place):
    g = gen(NB)
    rows = max(2, NB // 12)
    held = torch.randint(0, 12, (rows,), generator=g).tolist()
    held[0] = min(held[0], 5)
    while sum(held) > NB * 3 // 4:
        held[held.index(max(held))] -= 1
    s = State(held, NB, 14, shared=[1])
    data = pools(g, NB, Hkv, D, fp8)
    dev = [x.cuda() for x in data]
    t, pages, ref = s.dev
    t2, ref2 = (t, ref) if in_place else (torch.full_like(t, 5), torch.full_like(ref, 5))
    moved, live = torch.full_like(ref, 77), i32([0])
    ws = _abi.alloc_compact_workspace(NB, "cuda")
    ws.fill_(255)
    _abi.pa_compact_pages(dev[0], dev[1], t, pages, ref, t2, ref2, moved, live, ws, **scales(dev))
    ok()
    to, n = s.host.compact(data)
    assert live.tolist() == [n] and np.array_equal(moved.cpu().numpy(), to)
    s.dev = [t2, pages, ref2]
    s.same()
    for a, b in zip(dev, data):
        assert torch.equal(a.cpu(), b)


def test_compact_full_empty_and_bad_entries():
    g = gen(12)
    data = pools(g, 40, 2, 64, False)
    for held in ([20, 20], [0, 0]):           # nothing to move
        s = State(held, 40, 20)
        dev = [x.cuda() for x in data]
        t, pages, ref = s.dev
        moved, live = torch.full_like(ref, 77), i32([9])
        _abi.pa_compact_pages(dev[0], dev[1], t, pages, ref, t, ref, moved, live,
                              _abi.alloc_compact_workspace(40, "cuda"))
        ok()
        to, n = s.host.compact(data)
        assert live.tolist() == [n] and np.array_equal(moved.cpu().numpy(), to)
        s.same()
    s = State([3, 2], 40, 20)
    t, pages, ref = s.dev
    t[0, 1], t[1, 0] = 4000, int((ref == 0).nonzero()[3])
    ref2, t2 = torch.empty_like(ref), torch.empty_like(t)
    moved, live = torch.empty_like(ref), i32([9])
    _abi.pa_compact_pages(dev[0], dev[1], t, pages, ref, t2, ref2, moved, live,
                          _abi.alloc_compact_workspace(40, "cuda"))
    status(_abi.PA_STATUS_BAD_BLOCK)
    assert int(t2[0, 1]) == 4000 and int(t2[1, 0]) == -1
    assert bool((t2[:, 3:] == -1).all())


def test_page_calls_captured():
    """One captured turn: rows end, others begin, forks are made, the pool is compacted."""
    g = gen(15)
    s = State([3, 4, 2, 5, 0], 64, 10)
    data = pools(g, 64, 2, 64, False)
    dev = [x.cuda() for x in data]
    t, pages, ref = s.dev
    L, ends, rows, new = i32([40, 60, 20, 80, 0]), i32([1]), i32([1, 0]), i32([100, 50])
    src, dst, granted, got = i32([3]), i32([4]), i32([9]), i32([9, 9])
    moved, live, ws = torch.empty_like(ref), i32([0]), _abi.alloc_compact_workspace(64, "cuda")

    def turn():
        _abi.pa_free_pages(t, pages, ends, ref)
        _abi.pa_alloc_pages(t, pages, rows, new, ref, got)
        _abi.pa_free_pages(t, pages, dst, ref)
        _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, src, dst, ref, granted)
        _abi.pa_compact_pages(dev[0], dev[1], t, pages, ref, t, ref, moved, live, ws)
    lens = [40, 60, 20, 80, 0]

    def host(ends, rows, new, src, dst):
        s.host.free(ends)
        s.host.alloc(rows, new)
        s.host.free(dst)
        s.host.fork(src, dst, lens, data)
        s.host.compact(data)
    turn()
    host([1], [1, 0], [100, 50], [3], [4])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    graph.replay()
    host([1], [1, 0], [100, 50], [3], [4])
    ends.copy_(i32([2])), rows.copy_(i32([2, 3])), new.copy_(i32([31, 99])), src.copy_(i32([0])), dst.copy_(i32([1]))
    graph.replay()
    host([2], [2, 3], [31, 99], [0], [1])
    ok()
    s.same()
    for a, b in zip(dev, data):
        assert torch.equal(a.cpu(), b)


# -------------------------------------------------------------------- logits
def logits_case(g, B, n, V, H=0, bias=0, mask=False, parts=("repetition", "presence", "frequency", "temperature"),
                prompt=True):
    spec = {k: None for k in ("history", "history_lens", "prompt_lens", "draft_tokens", "repetition", "presence",
                              "frequency", "temperature", "bias_tokens", "bias_values", "allowed")}
    if H:
        spec["history"] = (V ** torch.rand(B, H, generator=g)).int().clamp(max=V) - 1
        spec["history_lens"] = torch.randint(0, H + 1, (B,), generator=g, dtype=torch.int32)
        if prompt:
            spec["prompt_lens"] = (spec["history_lens"] * torch.rand(B, generator=g)).int()
    if n:
        spec["draft_tokens"] = torch.randint(-1, V, (B, n), generator=g, dtype=torch.int32)
    draws = dict(repetition=lambda u: .5 + u, presence=lambda u: u - .3, frequency=lambda u: u - .2,
                 temperature=lambda u: (u * 2 - .4).clamp(min=0))
    for k in parts:
        spec[k] = draws[k](torch.rand(B, generator=g))
    if bias:
        spec["bias_tokens"] = torch.randint(-2, min(V, 40 + V // 3), (B, bias), generator=g, dtype=torch.int32)
        spec["bias_values"] = torch.randn(B, bias, generator=g) * 4
    if mask:
        words = (V + 31) // 32 + 1
        spec["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (B, n + 1, words), generator=g).int()
        spec["allowed"][0, 0] = 0                         # a row that allows nothing
        if B > 1:
            spec["allowed"][1] &= 0x100
    return spec


def run_logits(x, spec, probs, out=None):
    dev = {k: None if v is None else v.cuda() for k, v in spec.items()}
    x = x.cuda() if not x.is_cuda else x
    if out is None:
        out = torch.full(x.shape, 7., dtype=F32 if probs else x.dtype, device="cuda")
    _abi.pa_process_logits(out, x, _abi.LogitsSpec(**dev), probs=probs)
    return out


def check_logits(x, spec, probs, out):
    """Adjusted logits: each of at most four roundings is half a step of a partial sum, which
    is at most `size`, and a bias list of n values adds one each; then half a step of the result's
    type.  Probabilities: exp(x / T) takes the error of (x - max) / T, relative, for itself and
    in the sum; the difference, the product with log2(e) / T (two roundings) and the exponential
    add 2^-22 (1 + |d| / T) relative, the sums of up to 2^19 terms in a tree with 32 a thread
    under 2^-18."""
    host = {k: None if v is None else v.cpu().numpy() for k, v in spec.items()}
    xs, got = R.f64(x), R.f64(out)
    if xs.ndim == 2:
        xs, got = xs[:, None], got[:, None]
    if host["allowed"] is not None and host["allowed"].ndim == 2:
        host["allowed"] = host["allowed"][:, None]
    n_bias = 0 if host["bias_tokens"] is None else host["bias_tokens"].shape[1]
    for b in range(xs.shape[0]):
        T = 1. if host["temperature"] is None else float(host["temperature"][b])
        for i in range(xs.shape[1]):
            want, size = Q.logits(xs[b, i], host, b, i)
            tol = (4 + n_bias) * 2. ** -24 * size
            if not probs:
                fine = (got[b, i] == want) | (np.abs(got[b, i] - np.where(np.isinf(want), 0, want)) <=
                                              tol + HALF_STEP[x.dtype] * (np.abs(want) + tol) + 2. ** -25)
                fine |= np.isnan(want) & np.isnan(got[b, i])
                assert fine.all(), (b, i, np.flatnonzero(~fine)[:5])
                continue
            p = Q.probabilities(want, T)
            if not T > 0:
                at = np.flatnonzero(got[b, i])
                if p.max() == 0:
                    assert at.size == 0
                    continue
                # the largest, or one that rounding cannot tell from it
                top = want[int(np.argmax(p))]
                assert at.size == 1 and got[b, i, at[0]] == 1
                assert want[at[0]] >= top - 2 * tol[np.isfinite(want)].max(initial=0.) or want[at[0]] == top
                continue
            finite = np.isfinite(want)
            d = np.where(finite, np.where(finite, want, 0).max() - np.where(finite, want, 0), 0) / T
            err = 2 * tol[finite].max(initial=0.) / T + 2. ** -21 * (1 + d) + 2. ** -18
            off = np.abs(got[b, i] - p)
            fine = off <= p * (2 * np.expm1(np.minimum(err, 50)) + 2 * np.expm1(min(50., 2 * tol[finite].max(initial=0.) / T))) + 2. ** -120
            assert fine.all(), (b, i, T, np.flatnonzero(~fine)[:5], off.max())


LOGITS = [  # B, n, V, H, bias, mask, dtype
    (1, 0, 1, 0, 0, False, F32),
    (2, 0, 7, 5, 3, True, F32),
    (3, 2, 513, 20, 17, True, BF16),
    (1, 0, 32000, 300, 8, False, F32),
    (5, 3, 50257, 1000, 300, True, F16),      # rows that are not aligned
    (2, 1, 50257, 70, 0, False, F32),
    (40, 1, 16384, 100, 5, True, BF16),
    (2, 0, 128000, 9000, 1024, True, F32),
    (1, 1, 300001, 50, 20, True, BF16),
    (1, 0, 1 << 19, 400, 0, False, F16),
    (700, 2, 1000, 30, 2, False, F16),
    (160, 0, 4, 9, 3, True, F32),             # rows for all SMs, the shortest that is read by fours
    (155, 0, 12344, 900, 40, True, BF16),
    (40, 3, 33000, 5000, 1024, True, F32),    # nearly as many known tokens as the table takes
    (152, 0, 2000, 6000, 200, False, F16),    # more than it takes
]


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("B,n,V,H,bias,mask,dtype", LOGITS)
def test_logits(B, n, V, H, bias, mask, dtype, probs):
    g = gen(V + B)
    x = (torch.randn(B, n + 1, V, generator=g) * 3).to(dtype)
    spec = logits_case(g, B, n, V, H, bias, mask)
    out = run_logits(x, spec, probs)
    ok()
    check_logits(x, spec, probs, out)


@pytest.mark.parametrize("part", ["none", "repetition", "presence", "frequency", "temperature", "bias", "mask",
                                  "no prompt"])
@pytest.mark.parametrize("probs", [False, True])
def test_logits_parts_alone(part, probs):
    g = gen(4)
    x = torch.randn(3, 2, 999, generator=g)
    spec = logits_case(g, 3, 1, 999, 40, 5 if part == "bias" else 0, part == "mask",
                       [part] if part in ("repetition", "presence", "frequency", "temperature") else
                       ["repetition", "frequency"] if part == "no prompt" else [], part != "no prompt")
    out = run_logits(x, spec, probs)
    ok()
    check_logits(x, spec, probs, out)
    if part == "none" and not probs:
        assert torch.equal(out.cpu(), x)


def test_logits_in_place_padded_rows_and_two_dims():
    g = gen(6)
    for V, pad, dtype in ((1000, 24, BF16), (1001, 6, F32), (998, 1, F16)):
        base = (torch.randn(4, V + pad, generator=g) * 2).to(dtype)
        spec = logits_case(g, 4, 0, V, 50, 4, True)
        spec["allowed"] = spec["allowed"][:, 0]
        dev = base.cuda()
        rows = dev[:, :V]
        run_logits(rows, spec, False, out=rows)
        ok()
        check_logits(base[:, :V], spec, False, rows)
        assert torch.equal(dev[:, V:].cpu(), base[:, V:])         # what lies between the rows
        out = torch.full((4, V + 8), 7., device="cuda")
        run_logits(base.cuda()[:, :V], spec, True, out=out[:, :V])
        check_logits(base[:, :V], spec, True, out[:, :V])
        assert bool((out[:, V:] == 7).all())


def test_logits_of_many_rows_padded_and_in_place():
    """Rows for all SMs, of a length that is no multiple of four, apart from one another."""
    g = gen(16)
    V, B = 1003, 200
    base = (torch.randn(B, V + 5, generator=g) * 2).to(BF16)
    spec = logits_case(g, B, 0, V, 60, 9, True)
    out = torch.full((B, V + 1), 7., device="cuda")
    run_logits(base.cuda()[:, :V], spec, True, out=out[:, :V])
    check_logits(base[:, :V], spec, True, out[:, :V])
    assert bool((out[:, V:] == 7).all())
    dev = base.cuda()
    run_logits(dev[:, :V], spec, False, out=dev[:, :V])
    ok()
    check_logits(base[:, :V], spec, False, dev[:, :V])
    assert torch.equal(dev[:, V:].cpu(), base[:, V:])
    x = torch.randn(B, V + 1, generator=g)                        # fp32 logits to their own place
    dev = x.cuda()
    run_logits(dev, logits_case(g, B, 0, V + 1, parts=()), True, out=dev)
    ok()
    assert float((dev.cpu() - x.softmax(-1)).abs().max()) <= 1e-6


@pytest.mark.parametrize("rows", [6, 160])
def test_logits_bad_tokens_and_lengths_of_few_and_many_rows(rows):
    g = gen(17)
    x = torch.randn(rows, 2, 400, generator=g)
    spec = logits_case(g, rows, 1, 400, 30, 6)
    spec["history_lens"][:] = 30
    spec["history"][3, 7], spec["bias_tokens"][5, 2] = 400, 2 ** 31 - 1
    spec["draft_tokens"][2, 0] = 4000
    out = run_logits(x, spec, True)
    status(_abi.PA_STATUS_BAD_TOKEN)
    check_logits(x, spec, True, out)
    spec = logits_case(g, rows, 1, 400, 30, 6)
    spec["history_lens"][1], spec["history_lens"][4] = -1, 31
    out = run_logits(x, spec, False)
    status(_abi.PA_STATUS_BAD_LEN)
    check_logits(x, spec, False, out)


def test_logits_padding_and_bad_tokens():
    g = gen(7)
    x = torch.randn(2, 3, 100, generator=g)
    spec = logits_case(g, 2, 2, 100, 30, 6)
    spec["history"][:, ::3] = -1
    spec["history"][0, 1] = -2 ** 31
    spec["draft_tokens"][:] = torch.tensor([[-1, 5], [7, -9]], dtype=torch.int32)
    spec["history_lens"][:] = 30
    ok_out = run_logits(x, spec, False)
    ok()
    check_logits(x, spec, False, ok_out)
    spec["history"][0, 4], spec["bias_tokens"][1, 2], spec["draft_tokens"][1, 0] = 100, 2 ** 31 - 1, 105
    out = run_logits(x, spec, False)
    status(_abi.PA_STATUS_BAD_TOKEN)
    check_logits(x, spec, False, out)
    for L in (-1, 31):
        spec = logits_case(g, 2, 2, 100, 30, 6)
        spec["history_lens"][0] = L
        spec["prompt_lens"][0] = 3
        out = run_logits(x, spec, False)
        status(_abi.PA_STATUS_BAD_LEN)
        check_logits(x, spec, False, out)
    spec = logits_case(g, 2, 2, 100, 30, 6)
    spec["prompt_lens"][0], spec["prompt_lens"][1] = 99, -4       # all of it, none of it
    out = run_logits(x, spec, False)
    ok()
    check_logits(x, spec, False, out)


@pytest.mark.parametrize("copies", [1, 40])
def test_logits_not_finite(copies):
    """Few rows, and enough that each is a CTA's."""
    x = torch.randn(6, 300, generator=gen(1))
    inf, nan = float("inf"), float("nan")
    x[0, 5] = x[0, 270] = inf                        # they share the row
    x[1, :] = -inf
    x[2, 3] = nan
    x[3, :] = nan
    x[4, 7] = -inf
    x[5, 9] = inf
    spec = logits_case(gen(2), 6 * copies, 0, 300, parts=())
    many = x.repeat(copies, 1)
    for temp in (None, .5, 0., 1e-38, inf, 1e38, nan):
        spec["temperature"] = None if temp is None else torch.full((6 * copies,), temp)
        out = run_logits(many, spec, True).cpu()
        ok()
        assert not torch.isnan(out).any()
        assert torch.equal(out, out[:6].repeat(copies, 1))
        if temp in (0., 1e-38) or temp != temp:
            best = torch.nan_to_num(x, nan=-inf, posinf=inf, neginf=-inf).argmax(-1)
            for r in (2, 4, 5):
                assert out[r].sum() == 1 and out[r, best[r]] == 1
            assert out[0, 5] == 1 if temp != 1e-38 else out[0, 5] == .5
        else:
            assert out[0, 5] == out[0, 270] == .5 and out[0].sum() == 1
            check_logits(x[2:3], {k: None if v is None else v[2:3] for k, v in spec.items()}, True, out[2:3])
        assert out[1].sum() == 0 and out[3].sum() == 0 and out[2, 3] == 0 and out[4, 7] == 0
    got = run_logits(many, spec, False).cpu()
    assert torch.equal(torch.nan_to_num(got, nan=3.25), torch.nan_to_num(many, nan=3.25))


@pytest.mark.parametrize("copies", [1, 60])
def test_logits_ties_go_to_the_lowest_token(copies):
    x = torch.zeros(3, 1, 70000, dtype=BF16)
    x[1, 0, 60001:] = 2
    x[2, 0, [69999, 17, 30000]] = 5
    spec = logits_case(gen(2), 3 * copies, 0, 70000, parts=())
    spec["temperature"] = torch.zeros(3 * copies)
    spec["bias_tokens"] = torch.full((3 * copies, 1), 60001, dtype=torch.int32)   # a known token among them
    spec["bias_values"] = torch.zeros(3 * copies, 1)
    out = run_logits(x.repeat(copies, 1, 1), spec, True)
    ok()
    assert out.argmax(-1).flatten().tolist() == [0, 60001, 17] * copies
    assert out.sum(-1).flatten().tolist() == [1, 1, 1] * copies


@pytest.mark.parametrize("B", [2, 200])
def test_penalised_logits_of_any_magnitude(B):
    """x / r for logits and penalties whose quotient leaves fp32's range, or whose
    reciprocal does: within a step of the 64-bit quotient, inf where that is."""
    x = torch.tensor([1e38, 3e38, 1e-38, 1., 7., float("inf"), 1e-30, 5e37], dtype=torch.float32)
    logits = x.repeat(B, 1).cuda()
    rep = torch.tensor([.1, 1e38, 3e-39, 1.3, 3e38, 1e-20, 2., .9], dtype=torch.float32).repeat((B + 7) // 8)[:B].cuda()
    hist = torch.arange(8, dtype=torch.int32).repeat(B, 1).cuda()
    lens = torch.full((B,), 8, dtype=torch.int32, device="cuda")
    out = torch.empty_like(logits)
    _abi.pa_process_logits(out, logits, _abi.LogitsSpec(history=hist, history_lens=lens, repetition=rep))
    assert _abi.pa_get_status() == (0, 0)
    want = logits.double().cpu() / rep.double().cpu()[:, None]
    got = out.double().cpu()
    top = torch.finfo(torch.float32).max
    big = want > top
    # a rounding of the quotient and one of its correction, each half a step (2^-24), and below the
    # normal range a step of 2^-149 each
    near = (got - want).abs() <= want * 2. ** -23 + 2. ** -148
    assert bool(torch.where(big, torch.isinf(got) | (got >= top), near).all())


def test_logits_captured_and_on_another_stream():
    g = gen(11)
    x = torch.randn(4, 2, 5000, generator=g)
    spec = logits_case(g, 4, 1, 5000, 60, 5, True)
    want = run_logits(x, spec, True).clone()
    dev = {k: None if v is None else v.cuda() for k, v in spec.items()}
    xs, out = x.cuda(), torch.zeros_like(want)
    ls = _abi.LogitsSpec(**dev)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        _abi.pa_process_logits(out, xs, ls, probs=True)
    graph.replay()
    assert torch.equal(out, want)
    dev["history"][:, 0] = 3
    spec["history"][:, 0] = 3
    call = _abi.prepare(lambda: _abi.pa_process_logits(out, xs, ls, probs=True), stream)
    del ls
    torch.cuda.synchronize()
    for _ in range(3):
        call()
    graph.replay()
    torch.cuda.synchronize()
    ok()
    check_logits(x, spec, True, out)


def test_a_request_from_its_pages_to_its_next_token():
    """As they are used together: pages for two prompts, their keys appended, their attention in
    chunks, a fork, a decode step of all three, the pool compacted with the same result after,
    and a drawn token each."""
    g = gen(21)
    Hq, Hkv, D, NB, V, mbs = 8, 2, 64, 64, 1000, 16
    kc, vc = (torch.full((NB, Hkv, 16, D), float("nan"), dtype=F16, device="cuda") for _ in "kv")
    t = torch.full((3, mbs), -1, dtype=torch.int32, device="cuda")
    pages, L, ref, granted = i32([0, 0, 0]), i32([0, 0, 0]), i32([0] * NB), i32([0, 0])
    ref[3:9] = 1                                     # someone else's
    lens = [100, 37]
    _abi.pa_alloc_pages(t, pages, i32([0, 1]), i32([101, 37]), ref, granted)
    ok()
    assert granted.tolist() == [1, 1] and pages.tolist() == [7, 3, 0]
    K = [randn(g, n, Hkv, D) for n in lens]
    Vv = [randn(g, n, Hkv, D) for n in lens]
    qs = [randn(g, n, Hq, D) for n in lens]
    ws = _abi.alloc_prefill_workspace(2, 137, Hq, Hkv, D, "cuda")
    done, outs = [0, 0], [[], []]
    for chunk in ((60, 20), (40, 17)):               # two chunks of each prompt
        slots = []
        for b, c in enumerate(chunk):
            at = torch.arange(done[b], done[b] + c)
            slots.append(t[b].cpu().long()[at // 16] * 16 + at % 16)
        part = lambda x: torch.cat([x[b][done[b]:done[b] + c] for b, c in enumerate(chunk)]).cuda()  # noqa: E731
        _abi.pa_cache_append(part(K), part(Vv), kc, vc, torch.cat(slots).cuda())
        q = part(qs)
        done = [d + c for d, c in zip(done, chunk)]
        L[:2] = i32(done)
        out = torch.empty_like(q)
        _abi.pa_prefill(out, q, kc, vc, t[:2], L[:2], 256, i32([0, chunk[0], sum(chunk)]), .125, ws)
        for b, o in enumerate(out.split(list(chunk))):
            outs[b].append(o)
    ok()
    for b in range(2):
        k, v = (x.double().repeat_interleave(4, 1) for x in (K[b], Vv[b]))
        s = torch.einsum("ihd,jhd->hij", qs[b].double(), k) * .125
        s = s.masked_fill(torch.ones(lens[b], lens[b]).triu(1).bool(), -float("inf"))
        want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v)
        assert float((torch.cat(outs[b]).double().cpu() - want).abs().max()) <= 4e-3
    _abi.pa_fork_pages(kc, vc, t, pages, L, i32([0]), i32([2]), ref, granted[:1])
    ok()
    assert granted.tolist()[0] == 1 and L.tolist() == [100, 37, 100] and pages.tolist() == [7, 3, 7]
    q = randn(g, 3, Hq, D).cuda()
    q[2] = q[0]
    dec = _abi.alloc_workspace(3, Hq, D, 0, "cuda")
    before, after = torch.empty_like(q), torch.empty_like(q)
    _abi.pa_decode(before, q, kc, vc, t, L, 256, .125, 0, dec)
    assert torch.equal(before[0], before[2])
    moved, live = torch.empty_like(ref), i32([0])
    _abi.pa_free_pages(t, pages, i32([1]), ref)
    L[1] = 0
    _abi.pa_compact_pages(kc, vc, t, pages, ref, t, ref, moved, live, _abi.alloc_compact_workspace(NB, "cuda"))
    _abi.pa_decode(after, q, kc, vc, t, L, 256, .125, 0, dec)
    ok()
    assert live.tolist() == [6 + 7 + 1] and int((ref > 0).sum()) == 14 and bool((ref[14:] == 0).all())
    assert int(t[t >= 0].max()) < 14
    assert float((after[[0, 2]].float() - before[[0, 2]].float()).abs().max()) <= 2e-3
    logits = (after.flatten(1).float() @ randn(g, Hq * D, V, dtype=F32).cuda())
    allowed = torch.zeros(3, (V + 31) // 32, dtype=torch.int32, device="cuda")
    allowed[:, 5] = 0x10                             # the grammar leaves one token
    allowed[2, 7] = 1
    probs = torch.empty(3, 1, V, device="cuda")
    _abi.pa_process_logits(probs[:, 0], logits, _abi.LogitsSpec(
        history=i32([[164] * 9] * 3), history_lens=i32([9] * 3), frequency=torch.full((3,), 1e4, device="cuda"),
        allowed=allowed), probs=True)
    out, acc = torch.empty(3, 1, dtype=torch.int32, device="cuda"), i32([9] * 3)
    _abi.pa_verify_drafts(out, acc, probs, None, torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                          torch.full((3, 1), .5, device="cuda"))
    ok()
    assert out.flatten().tolist() == [164, 164, 224]
