"""pa_prefill where some rows of a tile of queries see nothing of the first keys that the tile
sees: windows that begin on a tile's border, and contexts whose first pages are not there."""
import pytest
import torch

from paged_kv_cache_179_gb300 import _abi
from test_request_gpu import BF16, F16, Prompts, ok, status

pytestmark = pytest.mark.gpu

# heads of a group, head_dim, type
FORMS = [(1, 64, F16), (1, 128, BF16), (4, 64, BF16), (4, 128, F16), (7, 128, BF16), (8, 64, F16), (8, 128, F16)]
# (context, new tokens, window): the last query's window begins on a tile's border
WINDOWS = [(1536, 1536, 512), (1300, 20, 532), (8192, 512, 4096)]


def far_below(p):
    """Every score far below 0 (about -220, with a spread of a few units)."""
    if p.fp8:
        p.kc[..., 0] = 0xFE                 # -448
        p.ks[:] = .02
        p.q[..., 0] = 200 * p.D ** .5 / 8
    else:
        p.kc[..., 0] = -60
        p.q[..., 0] = 30 * p.D ** .5 / 8
    for b, L in enumerate(p.lens):          # (the rows behind each context are NaN again)
        if L % 16:
            p.kc[int(p.tables[b, L // 16]), :, L % 16:] = 0x7f if p.fp8 else float("nan")


@pytest.mark.parametrize("G,D,dtype", FORMS)
@pytest.mark.parametrize("L,n,window", WINDOWS)
@pytest.mark.parametrize("fp8", [False, True])
def test_windows_that_begin_on_a_tile(L, n, window, G, D, dtype, fp8):
    p = Prompts([L], [n], G, 1, D, dtype, fp8, window)
    out = p.run()
    ok()
    p.check(out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [256, 384, 512, 1024])
def test_windows_of_several_prompts(window, fp8):
    """Prompts and chunks in one call, of two kv heads."""
    p = Prompts([1152, 700, 1100], [1152, 60, 1], 8, 2, 64, F16, fp8, window)
    out = p.run()
    ok()
    p.check(out)


@pytest.mark.parametrize("G,D,dtype", [(1, 64, F16), (4, 128, BF16), (7, 128, F16), (8, 64, BF16)])
@pytest.mark.parametrize("L,bad", [(700, 8), (900, 16), (2600, 8), (2600, 24)])
@pytest.mark.parametrize("fp8", [False, True])
def test_first_tiles_without_a_valid_page(L, bad, G, D, dtype, fp8):
    """Whole tiles of invalid pages in front, nothing else; items that are cut, too."""
    p = Prompts([L, 130], [40, 3], G, 1, D, dtype, fp8)
    p.tables[0, :bad] = -1
    out = p.run()
    status(_abi.PA_STATUS_BAD_BLOCK)
    p.check(out)


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("fp8", [False, True])
def test_scores_far_below_zero(D, dtype, fp8):
    """An offset of 0 in place of a row's own would leave no weight above 0."""
    p = Prompts([1300, 900], [20, 300], 4, 1, D, dtype, fp8, 532)
    far_below(p)
    out = p.run()
    ok()
    p.check(out)
    assert bool((out.float().abs().amax(-1) > 0).all())
    p = Prompts([1300], [20], 4, 1, D, dtype, fp8)
    far_below(p)
    p.tables[0, :8] = -1
    out = p.run()
    status(_abi.PA_STATUS_BAD_BLOCK)
    p.check(out)


def test_rows_without_a_number_in_sight():
    """Keys whose scores are -inf for a whole tile, then numbers: the numbers alone count."""
    p = Prompts([900], [30], 4, 1, 64, F16)
    p.q[..., 0] = 1.
    for j in range(8):
        p.kc[int(p.tables[0, j]), 0, :, 0] = float("-inf")
    clean = Prompts([900], [30], 4, 1, 64, F16)
    clean.q[..., 0] = 1.
    clean.tables[0, :8] = -1
    out = p.run()
    ok()
    clean.check(out)
