"""The calls of include/pa_serving.h on the GPU against their plain 64-bit statements."""
import numpy as np
import pytest
import torch

import _serving_ref as R
from paged_kv_cache_179_gb300 import _abi

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
HALF_STEP = {F16: 2. ** -11, BF16: 2. ** -8}


def ok():
    assert _abi.pa_get_status() == (0, 0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=F16):
    return torch.randn(*shape, generator=g).to(dtype)


# ------------------------------------------------------------------ rotation
def rope_tol(x, ref, dtype, amplitude=1.):
    """Half a step of the result's type (fp16's smallest step is 2^-24), and the
    fp32 rotation's error: cos and sin are off by at most 2^-24 pi (the angle's
    conversion), 2^-32 of a turn and two units in their last place, together
    under 5e-7; product and sum add 2^-24 each of at most |x| + |y|.  A pair's
    elements are bounded by the row's largest."""
    big = np.abs(x).max(-1, keepdims=True) * 2 * max(1., abs(amplitude))
    return HALF_STEP[dtype] * np.abs(ref) + 7e-7 * big + 2. ** -25


def spec_for(half, axes, adjacent, amplitude=1., base=1e6):
    inv = base ** (-np.arange(half) / half)
    axis = np.arange(half) * axes // half
    return _abi.RopeSpec(inv, axis, adjacent=adjacent, amplitude=amplitude, num_axes=axes), inv, axis


ROPE = [  # T, Hq, Hkv, D, rotary, axes, adjacent, dtype
    (1, 8, 2, 64, 64, 1, False, F16),
    (1, 1, 1, 16, 16, 1, True, BF16),
    (5, 28, 4, 128, 128, 3, False, BF16),
    (7, 28, 4, 128, 96, 3, True, F16),
    (33, 3, 1, 80, 80, 2, False, F16),
    (3, 40, 5, 72, 32, 4, True, BF16),       # nine chunks a row, the last one alone
    (2, 65, 1, 256, 256, 1, False, F16),     # more rows than one pass of a CTA takes
    (129, 15, 5, 64, 48, 3, False, BF16),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rotary,axes,adjacent,dtype", ROPE)
def test_rope(T, Hq, Hkv, D, rotary, axes, adjacent, dtype):
    g = gen(T + D)
    spec, inv, axis = spec_for(rotary // 2, axes, adjacent, 1.25 if adjacent else 1.)
    amp = 1.25 if adjacent else 1.
    pos = torch.randint(-70000, 1 << 20, (axes, T), generator=g, dtype=torch.int32)
    pos[0, 0] = 2 ** 31 - 1
    pos[-1, -1] = -2 ** 31
    qkv = randn(g, T, (Hq + 2 * Hkv) * D + 8, dtype=dtype)        # tokens apart, as in a projection
    q = qkv[:, :Hq * D].view(T, Hq, D) if T == 1 else qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    dev = qkv.cuda()
    qd = dev[:, :Hq * D].unflatten(1, (Hq, D))
    kd = dev[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    qo = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    ko = torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
    _abi.pa_rope(qo, qd, ko, kd, pos.cuda(), spec)
    ok()
    for x, got in ((q, qo), (k, ko)):
        x = R.f64(x)
        ref = R.rope(x, pos.numpy(), inv, axis, adjacent, amp)
        # the angle of a far position: 2^31 times a frequency's 2^-53
        tol = rope_tol(x, ref, dtype, amp) + 2. ** -20 * np.abs(x).max()
        assert (np.abs(R.f64(got) - ref) <= tol).all()
    assert torch.equal(dev.cpu(), qkv)                              # the inputs stay as they are


@pytest.mark.parametrize("exponents", [(-20, 0), (0, 20), (20, 40)])
def test_rope_angles_of_any_frequency_at_far_positions(exponents):
    """Whole turns are dropped without rounding: frequencies up to 2^40 radians a
    position (of either sign) and positions up to 2^31, against exact fractions.  The
    tolerance is the rotation's own: the fraction of a frequency is within 2^-63 of a
    turn, which position 2^31 makes 2^-32, one of the terms that rope_tol counts."""
    g = gen(61)
    T, half = 12, 32
    inv = 2. ** np.linspace(*exponents, half) * (1 + torch.rand(half, generator=g, dtype=torch.float64).numpy())
    inv = np.minimum(inv, 2. ** 40)
    inv[1::3] *= -1
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[:4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 1, 0], dtype=torch.int32)
    x = randn(g, T, 3, 2 * half)
    out = torch.empty(T, 3, 2 * half, dtype=F16, device="cuda")
    _abi.pa_rope(out, x.cuda(), None, None, pos.cuda(), _abi.RopeSpec(inv))
    ok()
    a = R.rope_angles(pos.tolist(), inv)[:, None]
    v = R.f64(x)
    lo, hi = v[..., :half], v[..., half:]
    ref = np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)
    assert (np.abs(R.f64(out) - ref) <= rope_tol(v, ref, F16)).all()


def test_rope_in_place_one_side_and_empty():
    g = gen(3)
    spec, inv, axis = spec_for(32, 1, False)
    pos = torch.arange(9, dtype=torch.int32)
    q = randn(g, 9, 4, 64)
    ref = R.rope(R.f64(q), pos.numpy()[None], inv, axis, False)
    d = q.cuda()
    _abi.pa_rope(d, d, None, None, pos.cuda(), spec)
    assert (np.abs(R.f64(d) - ref) <= rope_tol(R.f64(q), ref, F16)).all()
    k = q.cuda()
    out = torch.empty_like(k)
    _abi.pa_rope(None, None, out, k, pos.cuda()[None], spec)
    assert torch.equal(out, d)
    e = torch.empty(0, 4, 64, dtype=F16, device="cuda")
    _abi.pa_rope(e, e, None, None, torch.empty(0, dtype=torch.int32, device="cuda"), spec)
    ok()
    with pytest.raises(_abi.PAError):       # in place, tokens apart
        x = torch.zeros(9, 512, dtype=F16, device="cuda")[:, :256].unflatten(1, (4, 64))
        _abi._check(_abi.load().pa_rope(x.data_ptr(), x.data_ptr(), 512, None, None, 0,
                                        pos.cuda().data_ptr(), spec.pointer, 9, 4, 0, 64, 0, None),
                    "pa_rope")


def test_rope_turning_back_restores():
    """The rotation by minus the position undoes it, to the rounding in between."""
    g = gen(4)
    spec, _, _ = spec_for(64, 3, True)
    pos = torch.randint(0, 200000, (3, 50), generator=g, dtype=torch.int32).cuda()
    x = randn(g, 50, 6, 128, dtype=F16).cuda()
    y = torch.empty_like(x)
    _abi.pa_rope(y, x, None, None, pos, spec)
    _abi.pa_rope(y, y, None, None, -pos, spec)
    # half a step of the turned value, then of the result; a pair's elements
    # are at most sqrt(2) times the row's largest
    tol = (2 * 2 ** -11 * 2 ** .5 + 2e-6) * x.float().abs().amax(-1, keepdim=True) + 2 ** -24
    assert ((y.float() - x.float()).abs() <= tol).all()


@pytest.mark.parametrize("T,Hq,Hkv,D,bs,dtype", [(1, 4, 2, 64, 16, F16), (53, 28, 4, 128, 16, BF16),
                                                 (9, 3, 3, 72, 8, F16)])
def test_rope_append(T, Hq, Hkv, D, bs, dtype):
    g = gen(T)
    spec, _, _ = spec_for(32, 3, False)
    pos = torch.randint(0, 9000, (3, T), generator=g, dtype=torch.int32).cuda()
    qkv = randn(g, T, Hq + 2 * Hkv, D, dtype=dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    NB = T // bs + 3
    slots = torch.randperm(NB * bs, generator=g)[:T]
    if T > 1:
        slots[::5] = -1
    slots = slots.cuda()
    kc = randn(g, NB, Hkv, bs, D, dtype=dtype).cuda()
    vc = randn(g, NB, Hkv, bs, D, dtype=dtype).cuda()
    k2, v2 = kc.clone(), vc.clone()
    qo, q2 = torch.empty(T, Hq, D, dtype=dtype, device="cuda"), torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    kr = torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
    _abi.pa_rope_append(qo, q, k, v, kc, vc, slots, pos, spec)
    _abi.pa_rope(q2, q, kr, k, pos, spec)
    _abi.pa_cache_append(kr, v.contiguous(), k2, v2, slots)
    ok()
    assert torch.equal(qo, q2) and torch.equal(kc, k2) and torch.equal(vc, v2)


def test_rope_append_reports_a_slot_outside_the_pool():
    spec, _, _ = spec_for(32, 1, False)
    z = torch.ones(2, 2, 64, dtype=F16, device="cuda")
    pool, pool_v = (torch.zeros(4, 2, 16, 64, dtype=F16, device="cuda") for _ in "kv")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    qo = torch.empty_like(z)
    _abi.pa_rope_append(qo, z, z, z, pool, pool_v, torch.tensor([64, 3], device="cuda"), pos, spec)
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_SLOT)
    assert pool[0, :, 3].eq(1).all() and pool.sum().item() == 2 * 64
    assert torch.equal(qo, z)                     # position 0 turns nothing


@pytest.mark.parametrize("D,dtype,adjacent,rotary", [(64, F16, False, 64), (128, BF16, False, 128),
                                                     (128, F16, True, 96), (64, BF16, True, 16),
                                                     (128, BF16, False, 32)])
def test_rope_append_fp8_equals_the_separate_calls(D, dtype, adjacent, rotary):
    """Bit for bit pa_rope then pa_cache_append_fp8: a page's first rows, later
    rows and rows that re-scale their page."""
    g = gen(D + rotary)
    T, Hq, Hkv, NB = 11, 6, 3, 12
    spec, _, _ = spec_for(rotary // 2, 2, adjacent, 1.5)
    kc = torch.zeros(NB, Hkv, 16, D, dtype=torch.uint8, device="cuda")
    state = [kc, kc.clone(), torch.ones(NB, Hkv, device="cuda"), torch.ones(NB, Hkv, device="cuda")]
    other = [t.clone() for t in state]
    page = torch.randperm(NB, generator=g)[:T]
    for row, size in ((0, 1.), (1, .5), (2, 8.), (3, 1.)):
        qkv = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * size).to(dtype).cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.randint(0, 9000, (2, T), generator=g, dtype=torch.int32).cuda()
        slots = (page * 16 + row)
        slots[3] = -1
        slots = slots.cuda()
        qo, q2 = torch.empty(T, Hq, D, dtype=dtype, device="cuda"), torch.empty(T, Hq, D, dtype=dtype, device="cuda")
        kr = torch.empty(T, Hkv, D, dtype=dtype, device="cuda")
        _abi.pa_rope_append_fp8(qo, q, k, v, *state, slots, pos, spec)
        _abi.pa_rope(q2, q, kr, k, pos, spec)
        _abi.pa_cache_append_fp8(kr, v.contiguous(), *other, slots)
        ok()
        assert torch.equal(qo, q2)
        for x, y in zip(state, other):
            assert torch.equal(x, y)


# ------------------------------------------------------- attention weights
def weights_case(lens, Hq, Hkv, D, n_q, pool, dtype, seed, garbage=True):
    g = gen(seed)
    B = len(lens)
    mbs = max(1, max((x + 15) // 16 for x in lens))
    bt, nb = R.tables_for(lens, mbs, g)
    q = randn(g, B, n_q, Hq, D, dtype=dtype) * 1.5
    ks = None
    if pool == "fp8":
        kc, ks = R.e4m3_pool(g, (nb, Hkv, 16, D))
    else:
        kc = randn(g, nb, Hkv, 16, D, dtype=dtype)
        if garbage:         # what no token was written to: NaN
            for b, L in enumerate(lens):
                if L % 16:
                    kc[int(bt[b, L // 16]), :, L % 16:] = float("nan")
    w = torch.rand(B, Hkv, mbs * 16 + 4, generator=g)
    return q, kc, ks, bt, torch.tensor(lens, dtype=torch.int32), w


def run_weights(q, kc, ks, bt, lens, w, scale, decay, fresh, max_len=None, ws=None):
    B, n_q, Hq, D = q.shape
    Hkv = kc.shape[1]
    mx = bt.shape[1] * 16 if max_len is None else max_len
    n = _abi.pa_attention_weights_workspace_size(B, Hq, Hkv, mx, n_q)
    if ws is None:
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        ws[n // 2:] = 255          # what another call may leave in the scores and statistics
        ws[:1 << 16] = 0
    wd = w.cuda()
    args = (bt.cuda(), lens.cuda(), mx, scale, ws)
    if ks is None:
        _abi.pa_attention_weights(wd, q.cuda(), kc.cuda(), *args, decay=decay, fresh_tokens=fresh)
    else:
        _abi.pa_attention_weights_fp8(wd, q.cuda(), kc.cuda(), ks.cuda(), *args, decay=decay,
                                      fresh_tokens=fresh)
    return wd


WEIGHTS = [  # lens, Hq, Hkv, D, n_q, pool, dtype, decay, fresh
    ([1], 1, 1, 64, 1, "16", F16, 1., 0),
    ([1, 17, 100, 256], 8, 2, 64, 1, "16", F16, 1., 1),
    ([0, 15, 16, 0, 33, 1], 28, 4, 128, 1, "16", F16, .5, 1),
    ([700, 3, 0, 64], 14, 2, 128, 2, "16", BF16, 0., 2),        # 14 rows
    ([5, 1, 300], 28, 4, 128, 4, "16", F16, 1., 4),             # 28 rows; fewer tokens than queries
    ([90, 2], 32, 1, 64, 1, "16", BF16, .25, 0),                # one kv head, 32 rows
    ([130, 40], 14, 2, 64, 11, "16", F16, .5, 3),               # 77 rows: several passes
    ([64, 1, 2000], 15, 5, 64, 3, "fp8", BF16, 1., 0),
    ([31, 500], 28, 4, 128, 1, "fp8", F16, .5, 1),
    ([16, 260], 24, 1, 128, 1, "fp8", BF16, 0., 0),             # 24 rows
    ([20000, 1], 4, 1, 128, 1, "16", F16, 1., 1),               # long: every warp has a part of it
    ([4100, 0, 33, 700], 28, 4, 64, 1, "16", BF16, .5, 1),      # shared by the warps of several units
    ([4500, 90], 8, 1, 128, 3, "fp8", F16, 1., 3),
    ([5000, 17], 30, 1, 64, 1, "fp8", BF16, .5, 0),
    ([4000, 2900, 1], 16, 2, 128, 2, "16", F16, .5, 2),         # clusters, more pages than they keep
    ([3000, 4096], 28, 1, 128, 1, "16", F16, 0., 0),
    ([700, 65, 0], 20, 1, 64, 1, "16", BF16, 1., 1),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,n_q,pool,dtype,decay,fresh", WEIGHTS)
def test_attention_weights(lens, Hq, Hkv, D, n_q, pool, dtype, decay, fresh):
    q, kc, ks, bt, L, w = weights_case(lens, Hq, Hkv, D, n_q, pool, dtype, Hq + D + n_q)
    scale = float(np.float32(D ** -.5))
    ref, tol = R.attention_weights(R.f64(w), R.f64(q), kc, ks, bt, L, scale, decay, fresh)
    # an old weight that is not read may be anything
    for b, n in enumerate(lens):
        w[b, :, (max(0, n - fresh) if decay else 0):n] = float("nan")
    got = run_weights(q, kc, ks, bt, L, w, scale, decay, fresh)
    ok()
    got = R.f64(got)
    assert (np.abs(got - ref) <= tol).all()
    # every query adds 1 to its head group's total
    if decay == 0:
        for b, n in enumerate(lens):
            rows = sum(min(1, max(0, n - n_q + 1 + i)) for i in range(n_q)) * (Hq // Hkv)
            assert np.allclose(got[b, :, :n].sum(-1), rows, rtol=1e-5, atol=0)


def test_attention_weights_of_one_token_and_zero_queries():
    """A context of one token gets weight 1 a row; q = 0 spreads it evenly."""
    q, kc, ks, bt, L, w = weights_case([1, 48], 4, 2, 64, 1, "16", F16, 9)
    got = run_weights(q * 0, kc, ks, bt, L, w, .125, 0., 0).cpu()
    ok()
    assert got[0, :, 0].eq(2).all()
    assert (got[1, :, :48] - 2 / 48).abs().max() < 2 ** -22
    assert torch.equal(got[:, :, 48:], w[:, :, 48:])      # entries behind the context


@pytest.mark.parametrize("Hq,n_q,n,max_len", [(9, 1, 100, None), (9, 1, 40, 5008), (15, 2, 200, None), (30, 2, 77, None),
                                               (30, 4, 90, 5008)])
def test_attention_weights_of_infinite_keys(Hq, n_q, n, max_len):
    """A key that makes a logit -inf has weight 0, one that makes it +inf or NaN makes the
    row's weights NaN, as the softmax has it; rows and passes that do not fill a
    tile change nothing."""
    Hkv, D, group = 3, 64, Hq // 3
    q, kc, ks, bt, L, w = weights_case([n], Hq, Hkv, D, n_q, "16", F16, 17)
    if max_len:
        bt = torch.cat([bt, torch.full((1, max_len // 16 - bt.shape[1]), -1, dtype=torch.int32)], 1)
        w = torch.zeros(1, Hkv, max_len)
    q[..., 0] = 1
    q[:, :, 2 * group:, 0] = -1
    for at in (5, n - 1):                       # the last token: the last query alone sees it
        kc[int(bt[0, at // 16]), 0, at % 16, 0] = float("-inf")
    kc[int(bt[0, 1]), 1, 3, 0] = float("nan")
    kc[int(bt[0, 2]), 2, 3, 0] = float("inf")   # -inf after q's sign
    got = R.f64(run_weights(q, kc, ks, bt, L, w, .125, 0., 0, max_len=max_len))
    ok()
    assert np.isnan(got[0, 1, :n]).all()
    for h in (0, 2):
        K = R.keys(kc, ks, bt[0], h, n)
        size = .125 * (np.abs(np.where(np.isinf(K), 0, K)) @ np.abs(R.f64(q[0, :, h * group:(h + 1) * group])).reshape(-1, D).T)
        assert size.max() <= 16
        ref = np.zeros(n)
        for i in range(n_q):
            m = n - n_q + 1 + i
            for j in range(group):
                s = .125 * (K[:m] @ R.f64(q[0, i, h * group + j]))
                e = np.exp(s - s.max())
                ref[:m] += e / e.sum()
        # as for finite keys: a logit of 4 steps is off by 4 * 2^-22 * 16 + 2^-22 * 16, a weight
        # by its own and its row's largest, 160 * 2^-22, and 2^-20 for the rest: under 2^-14
        assert (np.abs(got[0, h, :n] - ref) <= 2. ** -14 * ref).all()
        assert got[0, h, 5 if h == 0 else 35] == 0


def test_attention_weights_is_deterministic_and_shares_blocks():
    """Sequences with the same blocks get what private copies get, bit for bit
    and in every run."""
    q, kc, ks, bt, L, w = weights_case([200, 200], 8, 2, 128, 1, "16", F16, 10)
    scale = 128 ** -.5
    pool = kc.clone()
    pool[bt[1].long()] = pool[bt[0].long()]
    one = run_weights(q, pool, ks, bt, L, w, scale, 1., 0)
    shared = bt.clone()
    shared[1] = bt[0]
    two = run_weights(q, pool, ks, shared, L, w, scale, 1., 0)
    ok()
    assert torch.equal(one, two)


def test_attention_weights_batch_above_one_launch():
    lens = [(7 * i) % 40 for i in range(520)]
    q, kc, ks, bt, L, w = weights_case(lens, 2, 1, 64, 1, "16", F16, 11)
    ref, tol = R.attention_weights(R.f64(w), R.f64(q), kc, ks, bt, L, .125, 1., 0)
    got = run_weights(q, kc, ks, bt, L, w, .125, 1., 0)
    ok()
    assert (np.abs(R.f64(got) - ref) <= tol).all()


@pytest.mark.parametrize("B,Hq,Hkv,D,n_q,pool,dtype", [
    (150, 2, 2, 128, 1, "16", F16),     # 34 pages a warp, old weights beyond those copied ahead
    (150, 2, 2, 64, 1, "fp8", BF16),
    (35, 20, 2, 128, 1, "16", BF16),    # 10 rows
    (20, 28, 2, 128, 2, "fp8", BF16),   # 28 rows
    (20, 28, 2, 128, 2, "16", F16),
    (60, 40, 2, 64, 1, "16", F16)])     # 20 rows
def test_attention_weights_of_more_pages_than_a_warp_keeps(B, Hq, Hkv, D, n_q, pool, dtype):
    _, kc, ks, bt, L, _ = weights_case([4500, 4400, 4097], Hq, Hkv, D, n_q, pool, dtype, 19)
    g = gen(20)
    at = torch.arange(B) % 3            # the sequences share blocks
    bt, L = bt[at].contiguous(), L[at].contiguous()
    q, w = randn(g, B, n_q, Hq, D, dtype=dtype) * 1.5, torch.rand(B, Hkv, bt.shape[1] * 16, generator=g)
    scale = float(np.float32(D ** -.5))
    ref, tol = R.attention_weights(R.f64(w), R.f64(q), kc, ks, bt, L, scale, .5, 1)
    got = run_weights(q, kc, ks, bt, L, w, scale, .5, 1)
    ok()
    assert (np.abs(R.f64(got) - ref) <= tol).all()


@pytest.mark.parametrize("Hq", [20, 56])          # 10 and 28 rows
def test_attention_weights_of_more_pages_than_a_cluster_keeps(Hq):
    lens = [4096, 2000] + [1] * 80
    q, kc, ks, bt, L, w = weights_case(lens, Hq, 2, 128, 1, "16", F16, 22)
    scale = float(np.float32(128 ** -.5))
    ref, tol = R.attention_weights(R.f64(w), R.f64(q), kc, ks, bt, L, scale, .5, 1)
    got = run_weights(q, kc, ks, bt, L, w, scale, .5, 1)
    ok()
    assert (np.abs(R.f64(got) - ref) <= tol).all()


def test_attention_weights_bad_indexes_are_skipped_and_reported():
    q, kc, ks, bt, L, w = weights_case([64, 32, 20], 4, 2, 64, 1, "16", F16, 12, garbage=False)
    bad = bt.clone()
    bad[0, 1] = kc.shape[0]               # one past the pool
    got = run_weights(q, kc, ks, bad, L, w, .125, 0., 0).cpu()
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_BLOCK)
    assert got[0, :, 16:32].eq(0).all()   # its tokens count for nothing
    assert torch.allclose(got[0, :, :64].sum(-1), torch.full((2,), 2.))
    L2 = L.clone()
    L2[1] = 65                            # above the bound: the sequence is skipped
    got = run_weights(q, kc, ks, bt, L2, w, .125, 0., 0).cpu()
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_LEN)
    assert torch.equal(got[1], w[1])
    L2[1] = -1
    got = run_weights(q, kc, ks, bt, L2, w, .125, 0., 0).cpu()
    assert _abi.pa_get_status()[1] == _abi.PA_STATUS_BAD_LEN
    assert torch.equal(got[1], w[1])


def test_attention_weights_reports_a_workspace_that_was_not_cleared():
    q, kc, ks, bt, L, w = weights_case([4200, 3], 4, 2, 64, 1, "16", F16, 14)   # beyond one cluster
    n = _abi.pa_attention_weights_workspace_size(2, 4, 2, bt.shape[1] * 16, 1)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ws[:4] = 0x7f
    run_weights(q, kc, ks, bt, L, w, .125, 0., 0, ws=ws)
    assert _abi.pa_get_status() == (_abi.PA_ERR_WORKSPACE, _abi.PA_STATUS_WS_DIRTY)
    ws.zero_()
    got = run_weights(q, kc, ks, bt, L, w, .125, 0., 0, ws=ws)
    ok()
    again = run_weights(q, kc, ks, bt, L, w, .125, 0., 0, ws=ws)   # left as it was needed
    ok()
    assert torch.equal(got, again) and not ws[:4].any()


@pytest.mark.parametrize("D,pool,lens", [(128, "16", [100, 33]), (64, "16", [4500, 7]),
                                         (128, "fp8", [4500, 7]), (64, "fp8", [90])])
def test_attention_weights_of_a_pool_that_begins_at_16_bytes(D, pool, lens):
    """Pools are 16-byte aligned, no more."""
    q, kc, ks, bt, L, w = weights_case(lens, 8, 2, D, 1, pool, F16, 15, garbage=False)
    want = run_weights(q, kc, ks, bt, L, w, .125, .5, 0)
    off = 16 // kc.element_size()
    room = torch.empty(kc.numel() + 64, dtype=kc.dtype, device="cuda")
    moved = room[off:off + kc.numel()].view(kc.shape)
    moved.copy_(kc)
    assert moved.data_ptr() % 32 == 16
    got = run_weights(q, moved, ks, bt, L, w, .125, .5, 0)
    ok()
    assert torch.equal(got, want)


def test_attention_weights_long_contexts_in_a_graph():
    """The cooperative launch, captured: every replay adds what the first call added,
    and two graphs may use one workspace in turn."""
    q, kc, ks, bt, L, w = weights_case([6000, 40, 5000], 8, 2, 64, 1, "16", F16, 16)
    mx = bt.shape[1] * 16
    ws = _abi.alloc_weights_workspace(3, 8, 2, mx, 1, "cuda")
    d = [t.cuda() for t in (q, kc, bt, L)]
    wd = w.cuda()
    call = lambda decay: _abi.pa_attention_weights(wd, *d, mx, .125, ws, decay=decay)  # noqa: E731
    call(0.)
    once = wd.clone()
    graphs = []
    for decay in (0., 1.):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(decay)
        graphs.append(g)
    wd.zero_()
    graphs[0].replay()
    graphs[1].replay()
    graphs[1].replay()
    ok()
    live = torch.arange(wd.shape[2], device="cuda") < L.cuda()[:, None, None]
    assert torch.allclose(wd[live.expand_as(wd)], 3 * once[live.expand_as(wd)], rtol=2 ** -22, atol=0)
    graphs[0].replay()
    ok()
    assert torch.equal(wd[live.expand_as(wd)], once[live.expand_as(wd)])


def test_attention_weights_workspace_too_small():
    q, kc, ks, bt, L, w = weights_case([64], 4, 2, 64, 1, "16", F16, 13)
    n = _abi.pa_attention_weights_workspace_size(1, 4, 2, 64, 1)
    with pytest.raises(_abi.PAError) as e:
        run_weights(q, kc, ks, bt, L, w, .125, 0., 0, ws=torch.zeros(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.code == _abi.PA_ERR_WORKSPACE


# ------------------------------------------------------------------ eviction
def evict_case(lens, Hkv, D, keep, pool, dtype, seed, kind):
    g = gen(seed)
    B = len(lens)
    mbs = max(1, max((x + 15) // 16 for x in lens))
    bt, nb = R.tables_for(lens, mbs, g)
    kb = (keep + 15) // 16 + 1
    spare = (nb + torch.randperm(B * kb, generator=g)).to(torch.int32).view(B, kb)
    NB = nb + B * kb
    w = torch.rand(B, Hkv, mbs * 16, generator=g)
    if kind == "ties":
        w = (w * 4).floor()
    elif kind == "equal":
        w = torch.zeros_like(w)
        w[..., ::3] = -0.
    elif kind == "odd":
        w[..., 5::7] = float("nan")
        w[..., 3::11] = float("inf")
        w[..., 2::11] = float("-inf")
        w[..., 1::5] *= -1
        w[..., 4::13] = 1e-42             # denormal
    if pool == "fp8":
        a, b = R.e4m3_pool(g, (NB, Hkv, 16, D)), R.e4m3_pool(g, (NB, Hkv, 16, D))
        pools, scales = [a[0], b[0]], [a[1], b[1]]
    else:
        pools = [randn(g, NB, Hkv, 16, D, dtype=dtype) for _ in "kv"]
        scales = [None, None]
    return pools, scales, w, bt, torch.tensor(lens, dtype=torch.int32), spare


def run_evict(pools, scales, w, bt, lens, spare, keep, first, recent, max_len=None, out=True):
    B, Hkv = w.shape[:2]
    p = [x.cuda() for x in pools]
    s = [None if x is None else x.cuda() for x in scales]
    w_out = torch.full((B, Hkv, keep + 3), -7., device="cuda") if out else None
    tables = torch.full_like(spare, -9).cuda() if out else None
    new = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    kept = torch.full((B, Hkv, keep), -3, dtype=torch.int32, device="cuda")
    args = (w.cuda(), w_out, bt.cuda(), lens.cuda(), bt.shape[1] * 16 if max_len is None else max_len,
            spare.cuda(), tables, new, kept)
    kw = dict(first_tokens=first, recent_tokens=recent)
    if s[0] is None:
        _abi.pa_evict(*p, *args, **kw)
    else:
        _abi.pa_evict_fp8(*p, *s, *args, **kw)
    return p, s, w_out, tables, new, kept


EVICT = [  # lens, Hkv, D, keep, first, recent, pool, dtype, kind
    ([2], 1, 64, 1, 0, 0, "16", F16, "random"),
    ([65, 64, 63, 0, 200, 1], 2, 64, 64, 4, 16, "16", F16, "random"),
    ([300, 129, 128], 3, 128, 99, 1, 31, "16", BF16, "ties"),
    ([100, 40], 2, 128, 39, 0, 39, "16", F16, "random"),        # the recent ones alone
    ([100, 41], 2, 64, 40, 40, 0, "16", F16, "random"),         # the first ones alone
    ([500, 77], 1, 64, 33, 3, 5, "16", F16, "equal"),           # all alike: the lowest indexes
    ([600, 80, 49], 2, 128, 48, 2, 6, "16", F16, "odd"),
    ([5000, 1030, 1024], 2, 64, 1023, 4, 100, "16", F16, "random"),
    ([9000, 8193], 1, 64, 4000, 0, 7, "16", F16, "ties"),       # two CTAs a unit, and so on
    ([20000, 30000], 1, 64, 700, 5, 20, "16", F16, "odd"),
    ([40000, 33000, 100], 1, 64, 700, 5, 20, "16", F16, "random"),
    ([40000], 1, 64, 20001, 0, 0, "16", F16, "equal"),
    ([70000, 66000, 9], 1, 64, 333, 1, 2, "16", F16, "ties"),   # more than the registers hold
    ([65, 64, 200], 2, 64, 64, 4, 16, "fp8", F16, "random"),
    ([300, 129, 20], 3, 128, 99, 1, 31, "fp8", F16, "ties"),
]


@pytest.mark.parametrize("lens,Hkv,D,keep,first,recent,pool,dtype,kind", EVICT)
def test_evict(lens, Hkv, D, keep, first, recent, pool, dtype, kind):
    pools, scales, w, bt, L, spare = evict_case(lens, Hkv, D, keep, pool, dtype, keep + D, kind)
    p, s, w_out, tables, new, kept = run_evict(pools, scales, w, bt, L, spare, keep, first, recent)
    ok()
    ref_new, ref_kept, ref_tables = R.evict(pools, scales, w.numpy(), bt, L.numpy(), spare, keep,
                                            first, recent)
    assert np.array_equal(new.cpu().numpy(), ref_new)
    assert torch.equal(tables.cpu(), ref_tables)
    kept, w_out = kept.cpu().numpy(), w_out.cpu().numpy()
    for b in range(len(lens)):
        for h in range(Hkv):
            at = ref_kept[b, h]
            assert np.array_equal(kept[b, h, :len(at)], at)
            assert (kept[b, h, len(at):] == -3).all()           # left as they were
            assert np.array_equal(w_out[b, h, :len(at)], w[b, h].numpy()[at], equal_nan=True)
            assert (w_out[b, h, len(at):] == -7).all()
    for got, want in zip(p, pools):                             # whole pools, bit for bit
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
    for got, want in zip(s, scales):
        assert want is None or torch.equal(got.cpu(), want)


@pytest.mark.parametrize("pool", ["16", "fp8"])
def test_evict_of_a_budget_that_nothing_exceeds(pool):
    pools, scales, w, bt, L, spare = evict_case([600, 48, 0], 2, 64, 608, pool, F16, 18, "random")
    p, s, w_out, tables, new, kept = run_evict(pools, scales, w, bt, L, spare, 608, 2, 300)
    ok()
    assert new.tolist() == [600, 48, 0]
    want = torch.full_like(spare, -1)
    want[:, :bt.shape[1]] = bt[:, :want.shape[1]]
    assert torch.equal(tables.cpu(), want)
    for b, n in enumerate(new.tolist()):
        assert torch.equal(kept[b, :, :n].cpu(), torch.arange(n, dtype=torch.int32).expand(2, n))
        assert torch.equal(w_out[b, :, :n].cpu(), w[b, :, :n])
    for a, b in zip(p, pools):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def test_evict_of_many_small_sequences():
    lens = [(5 * i) % 61 for i in range(300)]
    pools, scales, w, bt, L, spare = evict_case(lens, 3, 64, 21, "fp8", F16, 8, "ties")
    p, s, w_out, tables, new, kept = run_evict(pools, scales, w, bt, L, spare, 21, 2, 3)
    ok()
    ref_new, ref_kept, ref_tables = R.evict(pools, scales, w.numpy(), bt, L.numpy(), spare, 21, 2, 3)
    assert np.array_equal(new.cpu().numpy(), ref_new) and torch.equal(tables.cpu(), ref_tables)
    kept = kept.cpu().numpy()
    assert all(np.array_equal(kept[k][:len(v)], v) for k, v in ref_kept.items())
    assert all(torch.equal(a.cpu(), b) for a, b in zip(p + s, pools + scales))


def test_blocks_behind_two_billion_elements():
    """Block ids whose elements lie behind 2^31: append, weights and eviction."""
    g = gen(41)
    Hkv, D, n = 1, 128, 5
    NB = 2 ** 31 // (16 * D) + 64
    kc, vc = (torch.empty(NB, Hkv, 16, D, dtype=F16, device="cuda") for _ in "kv")
    table = torch.arange(NB - n, NB, dtype=torch.int32)[None]
    spare = torch.arange(NB - 20, NB - 16, dtype=torch.int32)[None]
    T = 16 * n - 3
    slots = (table[0].long()[torch.arange(T) // 16] * 16 + torch.arange(T) % 16).cuda()
    q, k, v = (randn(g, T, 1, D).cuda() for _ in "qkv")
    spec, inv, axis = spec_for(64, 1, False)
    pos = torch.arange(T, dtype=torch.int32).cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    _abi.pa_rope_append(qo, q, k, v, kc, vc, slots, pos, spec)
    _abi.pa_rope(None, None, ko, k, pos, spec)
    assert torch.equal(kc[-n:].view(-1, D)[:T], ko[:, 0]) and torch.equal(vc[-n:].view(-1, D)[:T], v[:, 0])
    L = torch.tensor([T], dtype=torch.int32).cuda()
    w = torch.zeros(1, 1, 16 * n, device="cuda")
    ws = _abi.alloc_weights_workspace(1, 1, 1, 16 * n, 1, "cuda")
    _abi.pa_attention_weights(w, qo[-1:], kc, table.cuda(), L, 16 * n, .088, ws, decay=0.)
    x = R.f64(qo[-1, 0]) @ R.f64(ko[:, 0]).T * np.float64(np.float32(.088))
    e = np.exp(x - x.max())
    # tolerances as derived beside R.attention_weights
    S = .088 * (np.abs(R.f64(ko[:, 0])) @ np.abs(R.f64(qo[-1, 0])))
    err = 2. ** -19 * S + 2. ** -22 * np.abs(x)
    assert (np.abs(R.f64(w[0, 0, :T]) - e / e.sum()) <= e / e.sum() * (err + err.max() + 2. ** -18)).all()
    new, kept = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, 1, 50, dtype=torch.int32, device="cuda")
    _abi.pa_evict(kc, vc, w, None, table.cuda(), L, 16 * n, spare.cuda(), None, new, kept,
                  first_tokens=1, recent_tokens=9)
    ok()
    at = R.evict_choice(w[0, 0].cpu().numpy(), T, 50, 1, 9)
    assert np.array_equal(kept[0, 0].cpu().numpy(), at)
    at = torch.from_numpy(at).cuda()
    assert torch.equal(kc[NB - 20:NB - 16].view(-1, D)[:50], ko[at, 0])
    assert torch.equal(vc[NB - 20:NB - 16].view(-1, D)[:50], v[at, 0])


def test_evict_without_the_optional_outputs():
    pools, scales, w, bt, L, spare = evict_case([90], 2, 64, 32, "16", F16, 1, "random")
    p, _, _, _, new, _ = run_evict(pools, scales, w, bt, L, spare, 32, 0, 0, out=False)
    ok()
    R.evict(pools, scales, w.numpy(), bt, L.numpy(), spare, 32, 0, 0)
    assert new.tolist() == [32] and torch.equal(p[0].cpu(), pools[0])


@pytest.mark.parametrize("pool", ["16", "fp8"])
def test_evict_bad_indexes_are_skipped_and_reported(pool):
    pools, scales, w, bt, L, spare = evict_case([90, 70, 80], 2, 64, 32, pool, F16, 2, "random")
    NB = pools[0].shape[0]
    spare[0, 1] = NB                      # that page is not written
    before = [x.clone() for x in pools]
    p, *_ = run_evict(pools, scales, w, bt, L, spare, 32, 0, 0)
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_BLOCK)
    bt2 = bt.clone()
    bt2[1, :] = -1                        # nothing of sequence 1 can be read
    spare[0, 1] = spare[0, 2]
    p, *_ = run_evict(pools, scales, w, bt2, L, spare, 32, 0, 0)
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_BLOCK)
    d = spare[1, :2].long()
    assert torch.equal(p[0].cpu()[d], before[0][d])
    L2 = L.clone()
    L2[2] = 10 ** 6
    *_, new, kept = run_evict(pools, scales, w, bt, L2, spare, 32, 0, 0)
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_LEN)
    assert new.tolist() == [32, 32, 0] and kept[2].eq(-3).all()


# -------------------------------------------------------------- verification
def probs(g, *shape, sharp=3.):
    return torch.softmax(torch.randn(*shape, generator=g) * sharp, -1)


VERIFY = [  # B, n, V, dtype, draft, pad
    (1, 1, 1, torch.float32, True, 0),
    (1, 4, 1000, torch.float32, True, 0),
    (7, 3, 515, torch.float32, True, 5),          # padded rows, odd sizes
    (5, 0, 33, torch.float32, False, 0),          # a plain draw
    (6, 5, 50257, torch.bfloat16, False, 0),
    (9, 2, 4099, F16, True, 1),
    (3, 8, 32000, torch.float32, False, 0),
    (40, 3, 129, BF16, True, 0),
    (1, 1, 300001, torch.float32, True, 0),       # a warp's part is narrowed down twice
    (2, 2, 400000, torch.float32, False, 0),
    (3, 1, 300008, BF16, True, 0),
    (700, 1, 40, torch.float32, True, 0),         # more sequences than CTAs fit at once
]


@pytest.mark.parametrize("B,n,V,dtype,draft,pad", VERIFY)
def test_verify(B, n, V, dtype, draft, pad):
    g = gen(V + n)
    p = probs(g, B, n + 1, V).to(dtype)
    q = (p[:, :n].float() * (torch.rand(B, n, V, generator=g) + .5)).to(dtype) if draft else None
    x = torch.randint(0, V, (B, n), generator=g, dtype=torch.int32)
    if n:       # likely tokens, so that some are accepted
        x[::2] = p[::2, :n].float().argmax(-1).to(torch.int32)
    nd = torch.randint(0, n + 1, (B,), generator=g, dtype=torch.int32)
    nd[::2] = n
    u = torch.rand(B, n + 1, generator=g)
    if pad:
        room = torch.full((B, n + 1, V + pad), 9.).to(dtype).cuda()
        room[..., :V] = p.cuda()
        pd = room[..., :V]
    else:
        pd = p.cuda()
    for drafts in (nd, None):
        out = torch.full((B, n + 1), -9, dtype=torch.int32, device="cuda")
        acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        _abi.pa_verify_drafts(out, acc, pd, None if q is None else q.cuda(), x.cuda(), u.cuda(),
                              num_drafts=None if drafts is None else drafts.cuda())
        ok()
        for b in range(B):
            want = R.verify(R.f64(p[b]), None if q is None else R.f64(q[b]), x[b].numpy(),
                            R.f64(u[b]), n if drafts is None else int(drafts[b]), n)
            assert (out[b].tolist(), int(acc[b])) == want, b


def verify_one(p, q, x, u, **kw):
    n = len(x)
    out = torch.full((1, n + 1), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    t = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")[None]  # noqa: E731
    _abi.pa_verify_drafts(out, acc, t(p), None if q is None else t(q),
                          torch.tensor([x], dtype=torch.int32, device="cuda"), t(u), **kw)
    return out[0].tolist(), int(acc)


def test_verify_edges():
    even = [.25] * 4
    last = 1 - 2. ** -24
    # borders of the draw: u = 0 draws the first token with weight, u on a border the next one
    assert verify_one([[0, .5, .5, 0]], None, [], [0.]) == ([1], 0)
    assert verify_one([even], None, [], [.25]) == ([1], 0)
    assert verify_one([even], None, [], [.25 - 2. ** -26]) == ([0], 0)
    assert verify_one([[.5, .5, 0, 0]], None, [], [last]) == ([1], 0)
    assert verify_one([[.5, .5, 0, 0]], None, [], [1.]) == ([1], 0)      # outside [0, 1): the last
    # u q = p is not below p: rejected; one step lower is accepted
    assert verify_one([even, even], [[.5, .5, 0, 0]], [0], [.5, 0.])[1] == 0
    assert verify_one([even, even], [[.5, .5, 0, 0]], [0], [.5 - 2. ** -25, 0.])[1] == 1
    # a product that fp32 would round onto p: u q = (1 - 2^-24)^2 < p = 1 - 2^-23
    assert verify_one([[1 - 2. ** -23, 0], [1, 0]], [[last, 0]], [0], [last, 0.])[1] == 0
    # the rest is p - q where that is positive
    assert verify_one([even, even], [[1, 0, 0, 0]], [0], [.5, 0.]) == ([1, -1], 0)
    # nothing is left of p - q: drawn from p
    assert verify_one([[0, 1], [1, 0]], [[0, 1]], [0], [.5, .5]) == ([1, -1], 0)
    # a draft without probabilities is taken out of p
    assert verify_one([[.5, .5], [1, 0]], None, [0], [.75, 0.]) == ([1, -1], 0)
    assert verify_one([[1, 0], [1, 0]], None, [1], [.5, 0.]) == ([0, -1], 0)
    # NaN, negative and infinite values; a row of zeros
    nan, inf = float("nan"), float("inf")
    assert verify_one([[nan, -1, .5, .5]], None, [], [.4]) == ([2], 0)
    assert verify_one([[0, inf, 1, 0]], None, [], [.6]) == ([1], 0)      # 2 and 1
    assert verify_one([[0, inf, 1, 0]], None, [], [.7]) == ([2], 0)
    assert verify_one([[0, 0]], None, [], [.5]) == ([-1], 0)
    ok()


def test_verify_far_tail_is_not_lost():
    """A token of probability 2^-50 behind 4095 large ones still has its place."""
    V = 4096
    p = torch.full((1, 1, V), 2. ** -13)
    p[0, 0, -1] = 2. ** -50
    out = torch.empty(1, 1, dtype=torch.int32, device="cuda")
    acc = torch.empty(1, dtype=torch.int32, device="cuda")
    none = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    u = torch.tensor([[2.]], device="cuda")              # beyond the total: the last with weight
    _abi.pa_verify_drafts(out, acc, p.cuda(), None, none, u)
    ok()
    assert out.item() == V - 1


def test_verify_bad_indexes_are_skipped_and_reported():
    even = [.25] * 4
    out, acc = verify_one([even] * 3, [even] * 2, [0, 4], [0., 0., 0.])
    assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_TOKEN)
    assert (out, acc) == ([0, 0, -1], 1)                 # p - q is zero: drawn from p
    out, acc = verify_one([even] * 3, None, [0, -1], [0., 0., 0.])
    assert _abi.pa_get_status()[1] == _abi.PA_STATUS_BAD_TOKEN and (out, acc) == ([0, 0, -1], 1)
    for nd in (3, -1):
        got = verify_one([even] * 3, None, [0, 1], [0., 0., 0.],
                         num_drafts=torch.tensor([nd], dtype=torch.int32, device="cuda"))
        assert _abi.pa_get_status() == (_abi.PA_ERR_BOUNDS, _abi.PA_STATUS_BAD_LEN)
        assert got == ([-1] * 3, 0)


def test_verify_follows_the_target():
    """Whatever the drafts, the first token out has the target's distribution:
    the even grid of u's gives each token its share to 1 / grid."""
    N, V = 1024, 6
    p = torch.tensor([.4, .3, .15, .1, .05, 0.])
    q = torch.tensor([.05, .1, .15, .3, .1, .3])
    grid = (torch.arange(N) + .5) / N
    # every draft token in its share of q, each with every pair of u's
    count = torch.zeros(V)
    for x in range(V):
        u = torch.stack([grid.repeat_interleave(32)[::32], grid[torch.randperm(N, generator=gen(x))]], 1)
        out = torch.empty(N, 2, dtype=torch.int32, device="cuda")
        acc = torch.empty(N, dtype=torch.int32, device="cuda")
        _abi.pa_verify_drafts(out, acc, p.expand(N, 2, V).contiguous().cuda(),
                              q.expand(N, 1, V).contiguous().cuda(),
                              torch.full((N, 1), x, dtype=torch.int32, device="cuda"), u.cuda())
        count += q[x] * torch.bincount(out[:, 0].cpu().long(), minlength=V).float() / N
    ok()
    # the draws after a rejection are a random subset of the grid: 4 sigma of its shares
    assert (count - p).abs().max() < 4 * (.25 / N) ** .5 + 2 / N


# ------------------------------------------------- streams, graphs, bound calls
def test_calls_on_two_streams_and_in_a_graph():
    """Weights, eviction and verification on a side stream and replayed from a
    graph give what the direct call gives; new inputs in the same tensors are seen."""
    lens = [300, 90, 0, 47]
    q, kc, ks, bt, L, w = weights_case(lens, 8, 2, 64, 1, "16", F16, 21)
    want = run_weights(q, kc, ks, bt, L, w, .125, .5, 1)
    B, mx = len(lens), bt.shape[1] * 16
    st = dict(w=w.cuda(), q=q.cuda(), k=kc.cuda(), bt=bt.cuda(), L=L.cuda())
    pools = [torch.cat([st["k"], torch.zeros(16, 2, 16, 64, dtype=F16, device="cuda")]) for _ in "kv"]
    nb = kc.shape[0]
    spare = torch.arange(nb, nb + 16, dtype=torch.int32, device="cuda").view(4, 4)
    ws = _abi.alloc_weights_workspace(B, 8, 2, mx, 1, "cuda")
    w_out = torch.zeros(B, 2, 64, device="cuda")
    tables, new = torch.zeros_like(spare), torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = torch.zeros(B, 2, 50, dtype=torch.int32, device="cuda")
    p = probs(gen(1), 3, 4, 700).cuda()
    x = torch.randint(0, 700, (3, 3), generator=gen(2), dtype=torch.int32).cuda()
    u = torch.rand(3, 4, generator=gen(3)).cuda()
    out, acc = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")

    def calls():
        _abi.pa_attention_weights(st["w"], st["q"], st["k"], st["bt"], st["L"], mx, .125, ws,
                                  decay=.5, fresh_tokens=1)
        _abi.pa_evict(*pools, st["w"], w_out, st["bt"], st["L"], mx, spare, tables, new, kept,
                      first_tokens=2, recent_tokens=8)
        _abi.pa_verify_drafts(out, acc, p, None, x, u)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    ok()
    assert torch.equal(st["w"], want)
    first = [t.clone() for t in (w_out, tables, new, kept, out, acc, *pools)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        st["w"].copy_(w.cuda())
        for t in (w_out, tables, new, kept, out, acc):
            t.zero_()
        graph.replay()
        ok()
        assert torch.equal(st["w"], want)
        for a, b in zip(first, (w_out, tables, new, kept, out, acc, *pools)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))   # pools hold NaN
    # other inputs in the same tensors
    q2 = q.flip(0).contiguous()
    st["q"].copy_(q2)
    st["w"].copy_(w)
    graph.replay()
    ok()
    assert torch.equal(st["w"], run_weights(q2, kc, ks, bt, L, w, .125, .5, 1))


def test_bound_call_keeps_its_rotation_alive():
    g = gen(5)
    x = randn(g, 3, 2, 64).cuda()
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    out, ref = torch.empty_like(x), torch.empty_like(x)

    def bind():
        spec, _, _ = spec_for(32, 1, False)
        return _abi.prepare(lambda: _abi.pa_rope(out, x, None, None, pos, spec))
    call = bind()
    import gc
    gc.collect()
    spec, _, _ = spec_for(32, 1, False)
    _abi.pa_rope(ref, x, None, None, pos, spec)
    call()
    ok()
    assert torch.equal(out, ref)


def test_wrong_shapes_types_and_layouts_are_refused():
    spec, _, _ = spec_for(32, 2, False)
    x = torch.zeros(4, 8, 64, dtype=F16, device="cuda")
    pos = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        _abi.pa_rope(x, x, None, None, pos[:, :3].contiguous(), spec)
    with pytest.raises(ValueError):
        _abi.pa_rope(x, x.transpose(0, 1), None, None, pos, spec)
    with pytest.raises(TypeError):
        _abi.pa_rope(x, x, None, None, pos.long(), spec)
    with pytest.raises(TypeError):
        _abi.pa_rope(x, x, x, x.bfloat16(), pos, spec)
    with pytest.raises(ValueError):
        _abi.pa_rope(x, x, None, x, pos, spec)
    p = torch.zeros(2, 4, 10, device="cuda")
    i = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    out, acc, u = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), i[:, 0].contiguous(), p[:, :, 0].contiguous()
    with pytest.raises(ValueError):
        _abi.pa_verify_drafts(out, acc, p[:, :3], None, i, u)
    with pytest.raises(TypeError):
        _abi.pa_verify_drafts(out, acc, p, p[:, :3].half(), i, u)
    with pytest.raises(ValueError):
        _abi.pa_verify_drafts(out, acc, p.transpose(0, 1).contiguous().transpose(0, 1), None, i, u)


@pytest.mark.parametrize("pool", ["16", "fp8"])
def test_decode_step_methods_make_these_calls(pool):
    """DecodeStep.rope_append, accumulate and evict over its own pools and tables."""
    from paged_kv_cache_179_gb300.step import DecodeStep
    lens, Hq, Hkv, D, keep = [70, 33], 6, 2, 64, 32
    g = gen(51)
    pools, scales, w, bt, L, spare = evict_case(lens, Hkv, D, keep, pool, F16, 51, "random")
    d = [t.cuda() for t in pools]
    sc = [None if t is None else t.cuda() for t in scales]
    kw = {} if pool == "16" else dict(k_scale=sc[0], v_scale=sc[1])
    step = DecodeStep(k_cache=d[0], v_cache=d[1], block_tables=bt.cuda(), context_lens=L.cuda(),
                      max_context_len=bt.shape[1] * 16, scale=.125, num_q_heads=Hq, split_ctas=2, **kw)
    spec, _, _ = spec_for(32, 1, True)
    q, k, v = randn(g, 2, Hq, D).cuda(), randn(g, 2, Hkv, D).cuda(), randn(g, 2, Hkv, D).cuda()
    pos = (L - 1).cuda()
    slots = (bt.gather(1, ((L - 1) // 16).long()[:, None])[:, 0].long() * 16 + (L - 1) % 16).cuda()
    qo, q2, kr = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    copies = [t.clone() for t in d], [None if t is None else t.clone() for t in sc]
    step.rope_append(qo, q, k, v, slots, pos, spec)
    _abi.pa_rope(q2, q, kr, k, pos, spec)
    if pool == "16":
        _abi.pa_cache_append(kr, v, *copies[0], slots)
    else:
        _abi.pa_cache_append_fp8(kr, v, *copies[0], *copies[1], slots)
    ok()
    assert torch.equal(qo, q2) and all(torch.equal(a, b) for a, b in zip(d, copies[0]))
    out = torch.empty_like(q)
    step.decode(qo, out)
    wd = w.cuda()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):     # the first call allocates: not in a capture
        with pytest.raises(RuntimeError, match="before the capture"):
            step.accumulate(wd, qo, decay=.5, fresh_tokens=1)
        out.zero_()
    want = run_weights(qo.cpu()[:, None], d[0].cpu(), None if pool == "16" else sc[0].cpu(), bt, L, w, .125, .5, 1)
    step.accumulate(wd, qo, decay=.5, fresh_tokens=1)
    assert torch.equal(wd, want)
    kept = torch.empty(2, Hkv, keep, dtype=torch.int32, device="cuda")
    new, tables = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(spare).cuda()
    step.evict(wd, None, spare.cuda(), tables, new, kept, first_tokens=1, recent_tokens=4)
    ok()
    assert new.tolist() == [keep] * 2 and torch.equal(tables.cpu(), spare)
    for b in range(2):
        for h in range(Hkv):
            assert np.array_equal(kept[b, h].cpu().numpy(), R.evict_choice(wd[b, h].cpu().numpy(), lens[b], keep, 1, 4))


# ------------------------------------------------------- the calls together
@pytest.mark.parametrize("pool", ["16", "fp8"])
def test_speculative_steps_over_a_cache_that_is_cut(pool):
    """Three speculative steps of a serving loop: append the drafts' rotated
    keys, decode their queries in one call, verify, keep the accepted ones,
    accumulate the attention weights, cut what has outgrown its budget, go on
    in the spare blocks.  Against the same steps in 64 bits (the cache's own
    contents are compared after every step)."""
    g = gen(31)
    B, Hq, Hkv, D, n_q, V, keep, budget = 3, 8, 2, 64, 4, 97, 48, 64
    lens = [60, 20, 70]
    mbs = 8
    NB = B * mbs * 2
    perm = torch.randperm(NB, generator=g).to(torch.int32)
    tables, spare = perm[:B * mbs].view(B, mbs).clone(), perm[B * mbs:].view(B, mbs).clone()
    dt = F16
    scale = float(np.float32(D ** -.5))
    spec, inv, axis = spec_for(32, 3, False)
    if pool == "fp8":
        (kc, ks), (vc, vs) = R.e4m3_pool(g, (NB, Hkv, 16, D)), R.e4m3_pool(g, (NB, Hkv, 16, D))
        ksd, vsd = ks.cuda(), vs.cuda()
    else:
        kc, vc = randn(g, NB, Hkv, 16, D), randn(g, NB, Hkv, 16, D)
    kd, vd = kc.cuda(), vc.cuda()
    w = torch.zeros(B, Hkv, mbs * 16)
    wd, w_next = w.cuda(), torch.zeros(B, Hkv, mbs * 16, device="cuda")
    L = torch.tensor(lens, dtype=torch.int32)
    place = L.clone()                        # positions go on where eviction shortens the cache
    td, sd = tables.cuda(), spare.cuda()
    ws = _abi.alloc_workspace(B, Hq, D, 4, "cuda", query_rows=n_q * Hq // Hkv)
    ww = _abi.alloc_weights_workspace(B, Hq, Hkv, mbs * 16, n_q, "cuda")
    for step in range(3):
        qkv = randn(g, B * n_q, Hq + 2 * Hkv, D, dtype=dt)
        pos = (place.view(B, 1) + torch.arange(n_q)).view(1, -1).repeat(3, 1).to(torch.int32)
        at = (L.view(B, 1) + torch.arange(n_q)).long()
        slots = tables.gather(1, at // 16).long() * 16 + at % 16
        d = qkv.cuda()
        q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]
        q_rot = torch.empty(B * n_q, Hq, D, dtype=dt, device="cuda")
        if pool == "fp8":                    # tokens of one page in separate calls
            for i in range(n_q):
                one = torch.arange(i, B * n_q, n_q, device="cuda")
                qi = torch.empty(B, Hq, D, dtype=dt, device="cuda")
                _abi.pa_rope_append_fp8(qi, q[one], k[one], v[one], kd, vd, ksd, vsd,
                                        slots[:, i].contiguous().cuda(), pos[:, i::n_q].contiguous().cuda(), spec)
                q_rot[one] = qi
        else:
            _abi.pa_rope_append(q_rot, q, k, v, kd, vd, slots.view(-1).cuda(), pos.cuda(), spec)
        L = L + n_q
        Ld = L.cuda()
        out = torch.empty(B, n_q, Hq, D, dtype=dt, device="cuda")
        qq = q_rot.view(B, n_q, Hq, D)
        mx = mbs * 16
        if pool == "fp8":
            _abi.pa_decode_fp8(out, qq, kd, vd, ksd, vsd, td, Ld, mx, scale, 4, ws)
        else:
            _abi.pa_decode(out, qq, kd, vd, td, Ld, mx, scale, 4, ws)
        # the model's head: any distribution will do
        p = probs(g, B, n_q, V)
        x = p[:, :n_q - 1].argmax(-1).to(torch.int32)
        u = torch.rand(B, n_q, generator=g)
        tok = torch.empty(B, n_q, dtype=torch.int32, device="cuda")
        acc = torch.empty(B, dtype=torch.int32, device="cuda")
        _abi.pa_verify_drafts(tok, acc, p.cuda(), None, x.cuda(), u.cuda())
        if pool == "fp8":
            _abi.pa_attention_weights_fp8(wd, qq, kd, ksd, td, Ld, mx, scale, ww, decay=.9, fresh_tokens=n_q)
        else:
            _abi.pa_attention_weights(wd, qq, kd, td, Ld, mx, scale, ww, decay=.9, fresh_tokens=n_q)
        ok()
        # --- the same in 64 bits
        ref_q = R.rope(R.f64(qkv[:, :Hq]), pos.numpy(), inv, axis, False)
        assert (np.abs(R.f64(q_rot) - ref_q) <= rope_tol(R.f64(qkv[:, :Hq]), ref_q, dt)).all()
        kc, vc = kd.cpu(), vd.cpu()
        ks, vs = (ksd.cpu(), vsd.cpu()) if pool == "fp8" else (None, None)
        if pool == "16":
            ref_k = R.rope(R.f64(qkv[:, Hq:Hq + Hkv]), pos.numpy(), inv, axis, False)
            got_k = R.f64(kc)[slots.view(-1) // 16, :, slots.view(-1) % 16]
            assert (np.abs(got_k - ref_k) <= rope_tol(R.f64(qkv[:, Hq:Hq + Hkv]), ref_k, dt)).all()
        for b in range(B):
            assert (tok[b].tolist(), int(acc[b])) == R.verify(R.f64(p[b]), None, x[b].numpy(), R.f64(u[b]), n_q - 1, n_q - 1)
        qr = R.f64(q_rot).reshape(B, n_q, Hq, D)
        ref_w, tol = R.attention_weights(R.f64(w), qr, kc, ks, tables, L, scale, float(np.float32(.9)), n_q)
        assert (np.abs(R.f64(wd) - ref_w) <= tol).all()
        for b in range(B):
            n = int(L[b])
            for h in range(Hkv):
                K, Vv = R.keys(kc, ks, tables[b], h, n), R.keys(vc, vs, tables[b], h, n)
                for i in range(n_q):
                    m = n - n_q + 1 + i
                    for j in range(Hq // Hkv):
                        s = scale * (K[:m] @ qr[b, i, h * 4 + j])
                        e = np.exp(s - s.max())
                        o = (e / e.sum()) @ Vv[:m]
                        # the decode path's stated tolerances
                        assert np.abs(R.f64(out[b, i, h * 4 + j]) - o).max() < (3e-2 if pool == "fp8" else 2e-3)
        # --- the accepted tokens stay, the rest of the drafts is forgotten
        L = L - (n_q - 1 - acc.cpu())
        place = place + 1 + acc.cpu()
        Ld = L.cuda()
        w = wd.cpu()
        # --- what has outgrown its budget is cut to `keep`, into the spare blocks
        if int(L.max()) > budget:
            t_next, new = torch.empty_like(td), torch.empty(B, dtype=torch.int32, device="cuda")
            kept = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")
            pools = [kd, vd]
            scales = [ksd, vsd] if pool == "fp8" else [None, None]
            cpu_pools = [t.cpu() for t in pools]
            cpu_scales = [None if t is None else t.cpu() for t in scales]
            args = (wd, w_next, td, Ld, mx, sd, t_next, new, kept)
            if pool == "fp8":
                _abi.pa_evict_fp8(*pools, *scales, *args, first_tokens=2, recent_tokens=16)
            else:
                _abi.pa_evict(*pools, *args, first_tokens=2, recent_tokens=16)
            ok()
            n, at, t = R.evict(cpu_pools, cpu_scales, w.numpy(), tables, L.numpy(), spare, keep, 2, 16)
            assert np.array_equal(new.cpu().numpy(), n) and torch.equal(t_next.cpu(), t)
            for a, b in zip(pools, cpu_pools):
                assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
            cut = L > keep
            spare = torch.where(cut[:, None], tables, spare)     # the old blocks are free now
            tables, L = t, torch.from_numpy(n).to(torch.int32)
            wd, w_next = w_next, wd
            w, td, sd = wd.cpu(), tables.cuda(), spare.cuda()
    assert int(L.min()) > 0
