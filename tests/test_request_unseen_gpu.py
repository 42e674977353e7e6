"""pa_prefill and what none of a call's queries sees, or not the one at hand: pages before every
window, and the scales of pages that other queries see."""
import pytest
import torch

from test_request_gpu import BF16, F16, Prompts, ok

pytestmark = pytest.mark.gpu

# context, new tokens, window: the first query's window begins inside a tile, its pages before
# (L - n - window + 1) // 16 are behind every window
BEHIND = [(1300, 20, 532), (1300, 20, 600), (700, 1, 100), (2600, 300, 1000), (300, 3, 40)]


@pytest.mark.parametrize("G,D,dtype", [(1, 64, F16), (4, 128, BF16), (7, 128, F16), (8, 64, BF16)])
@pytest.mark.parametrize("L,n,window", BEHIND)
@pytest.mark.parametrize("fp8", [False, True])
def test_pages_behind_every_window_are_not_looked_at(L, n, window, G, D, dtype, fp8):
    """Their ids may be anything (a page that was given back), and what stands in one."""
    gone = (L - n - window + 1) // 16
    for bad in (-1, 10 ** 6):
        p = Prompts([L], [n], 2 * G, 2, D, dtype, fp8, window)
        p.tables[0, :gone] = bad
        out = p.run()
        ok()
        p.check(out)
    p = Prompts([L], [n], 2 * G, 2, D, dtype, fp8, window)
    clean = Prompts([L], [n], 2 * G, 2, D, dtype, fp8, window)
    ids = p.tables[0, :gone].long()
    if fp8:
        p.ks[ids], p.vs[ids] = float("nan"), 1e30
        p.kc[ids] = p.vc[ids] = 0x7f
    else:
        p.kc[ids], p.vc[ids] = float("nan"), float("inf")
    out = p.run()
    ok()
    clean.check(out)


@pytest.mark.parametrize("factor", [2. ** 40, float("nan")])
@pytest.mark.parametrize("G,D,dtype", [(1, 64, F16), (4, 128, BF16), (7, 128, F16), (8, 64, BF16)])
@pytest.mark.parametrize("window", [0, 100])
def test_scales_of_pages_that_a_query_does_not_see(window, G, D, dtype, factor):
    """A page's scales reach the queries that see it.  Those before it (and, with a window,
    those past it) get what they would get from any other page in its place."""
    for at in (5, 11, 20):
        case = ([500, 64], [500, 64], 2 * G, 2, D, dtype, True, window)
        p, clean = Prompts(*case), Prompts(*case)
        for s in (p.ks, p.vs):
            s[int(p.tables[0, at])] *= factor
        got, want = p.run(), clean.run()
        ok()
        pos = torch.arange(500, device="cuda")
        sees = pos >= 16 * at
        if window:
            sees &= pos - window + 1 < 16 * (at + 1)
        sees = torch.cat([sees, torch.zeros(64, dtype=torch.bool, device="cuda")])
        clean.check(torch.where(sees[:, None, None], want, got))
