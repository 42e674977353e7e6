"""Page calls over pools that a cluster of CTAs ranks and with more pairs than shared memory keeps
the places of, and prompts of more sequences than one launch sorts whose items are cut."""
import numpy as np
import pytest
import torch

from paged_kv_cache_179_gb300 import _abi
from test_request_gpu import BF16, F16, Prompts, State, gen, i32, ok, pools, scales, status

pytestmark = pytest.mark.gpu


def take_all_but(s, free):
    """Only the pages ``free`` of the pool are left, and those that the rows hold."""
    taken = s.host.ref <= 0
    taken[free] = False
    s.host.ref[taken] = 1
    s.dev[2].copy_(torch.from_numpy(s.host.ref).to(torch.int32))


def free_of(s, n, g):
    """n pages that no row holds, anywhere in the pool."""
    at = np.flatnonzero(s.host.ref <= 0)
    return at[torch.randperm(len(at), generator=g)[:n].numpy()]


@pytest.mark.parametrize("Hkv,fp8", [(1, False), (2, True)])
@pytest.mark.parametrize("NB", [16385, 40003])
def test_fork_in_large_pools(NB, Hkv, fp8):
    """Part-full and full last pages, one source often, a pool that runs out in the middle."""
    g = gen(NB + Hkv)
    held = [40, 3, 1, 0, 9] + [0] * 40
    lens = [631, 48, 5, 0, 130] + [0] * 40
    s = State(held, NB, 40, shared=[4])
    data = pools(g, NB, Hkv, 64, fp8)
    dev = [x.cuda() for x in data]
    take_all_but(s, free_of(s, 17, g))
    src = [0, 1, 0, 2, 4, 1, 3, 0] * 5
    dst = list(range(44, 4, -1))
    t, pages, ref = s.dev
    L, granted = i32(lens), i32([9] * len(src))
    _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, i32(src), i32(dst), ref, granted, **scales(dev))
    ok()
    assert granted.tolist() == s.host.fork(src, dst, lens, data)
    assert 17 < sum(granted.tolist()) < len(src)
    assert L.tolist() == lens
    s.same()
    for a, b in zip(dev, data):
        assert torch.equal(a.cpu(), b)


def test_fork_of_many_pairs():
    """More than shared memory keeps the places of; bad pairs among them."""
    g = gen(31)
    n, NB = 9000, 20011
    s = State([2, 1, 3] + [0] * n, NB, 3)
    lens = [20, 16, 48] + [0] * n
    data = pools(g, NB, 1, 64, False)
    dev = [x.cuda() for x in data]
    src = [(0, 1, 0, 2)[i % 4] for i in range(n)]
    dst = list(range(n + 2, 2, -1))
    src[5], src[4001], dst[8500] = -1, n + 3, -7
    take_all_but(s, free_of(s, 4300, g))
    t, pages, ref = s.dev
    L, granted = i32(lens), i32([9] * n)
    _abi.pa_fork_pages(dev[0], dev[1], t, pages, L, i32(src), i32(dst), ref, granted)
    status(_abi.PA_STATUS_BAD_ROW)
    assert granted.tolist() == s.host.fork(src, dst, lens, data)
    assert 8000 < sum(granted.tolist()) < n - 3
    assert L.tolist() == lens
    s.same()
    for a, b in zip(dev, data):
        assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("NB", [(1 << 21) + 1003, (1 << 22) + 129])
def test_alloc_and_free_in_very_large_pools(NB):
    """Chunks of more than 512 pages each; free pages far apart, then none."""
    g = gen(NB)
    s = State([1] * 30 + [0] * 10, NB, 600, shared=[1, 2])
    take_all_but(s, free_of(s, 1500, g))
    rows = [39, 0, 38, 5, 37, 36, 4]
    lens = [16 * 500, 40, 16 * 450, 1, 16 * 400 + 1, 16 * 600, 33]
    t, held, ref = s.dev
    granted = i32([9] * 7)
    _abi.pa_alloc_pages(t, held, i32(rows), i32(lens), ref, granted)
    ok()
    assert granted.tolist() == s.host.alloc(rows, lens) == [1, 1, 1, 1, 1, 0, 0]
    s.same()
    _abi.pa_free_pages(t, held, i32([38, 1, 39, 38]), ref)
    ok()
    s.host.free([38, 1, 39])
    s.same()
    _abi.pa_alloc_pages(t, held, i32(rows[-2:]), i32(lens[-2:]), ref, granted[:2])
    ok()
    assert granted.tolist()[:2] == s.host.alloc(rows[-2:], lens[-2:]) == [1, 1]
    s.same()


@pytest.mark.parametrize("fp8,dtype", [(False, BF16), (True, F16)])
def test_prefill_of_many_sequences_with_cut_items(fp8, dtype):
    """Two launches that sort 512 sequences each share the workspace of the items they cut."""
    g = gen(9)
    n = 700
    lens = torch.randint(1, 60, (n,), generator=g).tolist()
    news = [min(x, int(torch.randint(0, 3, (1,), generator=g))) for x in lens]
    for b, (L, m) in {3: (2500, 9), 400: (1300, 40), 511: (3000, 2), 512: (2900, 33), 699: (2200, 5)}.items():
        lens[b], news[b] = L, m
    p = Prompts(lens, news, 4, 1, 64, dtype, fp8)
    out = p.run()
    ok()
    p.check(out)
