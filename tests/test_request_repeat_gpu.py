"""pa_process_logits gives the same bits each time it is called, whatever order its threads run in."""
import pytest
import torch

from paged_kv_cache_179_gb300 import _abi
from test_request_gpu import BF16, F16, F32, gen, logits_case, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("B,n,V,H,bias,dtype", [(2, 1, 30000, 900, 40, BF16), (40, 3, 4000, 3000, 50, F32),
                                                (160, 0, 4000, 50, 3, F32), (152, 0, 32000, 5500, 300, F16),
                                                (100, 1, 128000, 4096, 64, BF16)])
def test_logits_repeat_themselves(B, n, V, H, bias, dtype, probs):
    """Few rows and many, tables that are nearly full, so that tokens collide there."""
    g = gen(V + B)
    x = (torch.randn(B, n + 1, V, generator=g) * 3).to(dtype).cuda()
    spec = logits_case(g, B, n, V, H, bias, True)
    spec["temperature"].clamp_(min=.3)      # (no row is greedy)
    ls = _abi.LogitsSpec(**{k: None if v is None else v.cuda() for k, v in spec.items()})
    first = torch.zeros(B, n + 1, V, dtype=F32 if probs else dtype, device="cuda")
    out = torch.zeros_like(first)
    _abi.pa_process_logits(first, x, ls, probs=probs)
    for _ in range(40):
        _abi.pa_process_logits(out, x, ls, probs=probs)
        assert torch.equal(out, first)
    ok()
