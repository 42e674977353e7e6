"""The bounded waits of pa_prefill, run out on purpose: a copy of keys that never comes.  The
kernel gives up, the status word reports PA_STATUS_TIMEOUT, and the next call, with the
same workspace, gives what it gave before.  Nothing here faults, traps or waits without
bound."""
import time

import pytest
import torch

import _serving_ref as R
from paged_kv_cache_179_gb300 import _abi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype,drop", [(128, torch.bfloat16, 0), (64, torch.float16, 0), (128, torch.float16, 5)])
def test_prefill_waits_run_out(D, dtype, drop):
    g = torch.Generator().manual_seed(D)
    lens, news, Hq, Hkv = [1300, 700, 1200], [300, 700, 1200], 8, 2
    tables, nb = R.tables_for(lens, 82, g)
    q = torch.randn(sum(news), Hq, D, generator=g).to(dtype).cuda()
    kc, vc = (torch.randn(nb, Hkv, 16, D, generator=g).to(dtype).cuda() for _ in "kv")
    starts = torch.tensor([0, 300, 1000, 2200], dtype=torch.int32, device="cuda")
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = _abi.alloc_prefill_workspace(3, 2200, Hq, Hkv, D, "cuda")
    args = (q, kc, vc, tables.cuda(), L, 82 * 16, starts, .125, ws)
    want, out = torch.empty_like(q), torch.empty_like(q)
    _abi.pa_prefill(want, *args)
    assert _abi.pa_get_status() == (0, 0)
    t = time.perf_counter()
    _abi.pa_test_prefill_timeout(out, *args, drop_tile=drop, limit_ns=20_000_000)
    assert _abi.pa_get_status() == (_abi.PA_ERR_TIMEOUT, _abi.PA_STATUS_TIMEOUT)
    assert time.perf_counter() - t < 4.             # 20 ms, and 2 s for the copy that never comes
    assert _abi.pa_get_status() == (0, 0)           # the read cleared it
    _abi.pa_prefill(out, *args)
    assert _abi.pa_get_status() == (0, 0)
    assert torch.equal(out, want)
