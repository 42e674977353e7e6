"""The bounded wait of pa_attention_weights' cooperative launch, run out on purpose.

Its warps wait for the softmax statistics of the warps that share their first and
their last (sequence, kv head).  Here one warp announces nothing, so that the others
give up after 1 ms: the kernel returns, the status word reports PA_STATUS_TIMEOUT,
what they waited for is not written, and after a zero-fill of the workspace the next
call gives what it gave before.  Nothing here faults, traps or waits without bound.
"""
import time

import pytest
import torch

import _serving_ref as R
from paged_kv_cache_179_gb300 import _abi

pytestmark = pytest.mark.gpu

LIMIT_NS = 1_000_000   # 1 ms
BOUND = 5008           # above 4096: the cooperative launch, whatever the lengths
F16 = torch.float16


class Case:
    """Short contexts under a long bound: while there are fewer pages than warps, warp w
    takes page w of the line of all (sequence, kv head, page)s."""

    def __init__(self, lens, Hq, Hkv, D, seed, bound=BOUND):
        g = torch.Generator().manual_seed(seed)
        bt, nb = R.tables_for(lens, bound // 16, g)
        self.bound, self.lens = bound, lens
        self.q = torch.randn(len(lens), Hq, D, generator=g).to(F16).cuda()
        self.k = torch.randn(nb, Hkv, 16, D, generator=g).to(F16).cuda()
        self.bt, self.L = bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.ws = _abi.alloc_weights_workspace(len(lens), Hq, Hkv, bound, 1, "cuda")
        self.shape = (len(lens), Hkv, bound)

    def right(self):
        w = torch.full(self.shape, -7., device="cuda")
        _abi.pa_attention_weights(w, self.q, self.k, self.bt, self.L, self.bound, .125, self.ws, decay=0.)
        assert _abi.pa_get_status() == (0, 0)
        return w

    def with_silent(self, warp):
        """The weights, the status and the seconds of a call whose warp says nothing."""
        w = torch.full(self.shape, -7., device="cuda")
        torch.cuda.synchronize()
        t = time.perf_counter()
        _abi.pa_test_weights_timeout(w, self.q, self.k, self.bt, self.L, self.bound, .125, self.ws,
                                     silent_warp=warp, limit_ns=LIMIT_NS)
        status = _abi.pa_get_status()
        return w, status, time.perf_counter() - t

    def timed_out(self, warp):
        w, status, seconds = self.with_silent(warp)
        assert status == (_abi.PA_ERR_TIMEOUT, _abi.PA_STATUS_TIMEOUT)
        assert seconds < 1.0                        # gave up after its limit, not the 2 s default
        assert _abi.pa_get_status() == (0, 0)       # the read cleared it
        return w


def test_a_unit_of_few_parts():
    """Units of 10, 3 and 13 pages, one a warp: warps wait for at most 16 others each by
    itself.  Only the unit with the silent warp stays unwritten."""
    c = Case([160, 40, 200], 4, 1, 64, 1)
    right = c.right()
    for warp, seq in ((0, 0), (9, 0), (10, 1), (12, 1), (13, 2), (25, 2)):
        got = c.timed_out(warp)
        for b, n in enumerate(c.lens):
            want = torch.full_like(right[b], -7.) if b == seq else right[b]
            assert torch.equal(got[b], want), (warp, b)
        c.ws.zero_()
        assert torch.equal(c.right(), right)


def test_a_unit_of_many_parts():
    """A context whose 300 pages go to 300 warps, joined by whole CTAs: none of it is
    written; the sequence after it, in CTAs of its own but for one, is right or unwritten."""
    c = Case([4800, 100], 7, 1, 128, 2)
    right = c.right()
    for warp in (0, 150, 299):
        got = c.timed_out(warp)
        assert got[0].eq(-7).all()
        at = torch.arange(7, device="cuda") * 16    # a page of the second sequence is whole or not there
        for page in at.tolist():
            a, b = got[1, 0, page:page + 16], right[1, 0, page:page + 16]
            assert torch.equal(a, b) or a.eq(-7).all()
        assert got[1, 0, 96:100].eq(right[1, 0, 96:100]).all()     # pages from 306 on: another CTA's
        c.ws.zero_()
        assert torch.equal(c.right(), right)


def test_warps_with_several_pages_and_units():
    """More pages than warps: what is written is right, the silent warp's unit is not, and
    the first unit of the line, far from it, is."""
    lens = [5000, 700] * 8
    c = Case(lens, 2, 2, 64, 3, bound=5008)
    right = c.right()
    got = c.timed_out(500)
    unwritten = got.eq(-7) & right.ne(-7)
    assert torch.equal(got[~unwritten], right[~unwritten])
    assert unwritten.any() and not unwritten[0, 0].any()
    assert unwritten.any(-1).sum() < len(lens) * 2 // 2
    c.ws.zero_()
    assert torch.equal(c.right(), right)


def test_a_warp_behind_the_last_changes_nothing():
    c = Case([160, 40], 4, 1, 64, 4)
    right = c.right()
    got, status, _ = c.with_silent(13)
    assert status == (0, 0) and torch.equal(got, right)
