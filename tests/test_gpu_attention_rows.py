"""paged_attention over caches that end with the last key: nothing lies behind the last row."""
import pytest
import torch

from test_gpu_paged_attention import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("D", [136, 152, 184, 200, 232, 248, 256])
def test_cache_ends_with_its_last_row(D, heads_first, page):
    n = 4 * page
    q, kc, vc, table, lengths = make(1, 4, 2, D, [n], page, torch.bfloat16, seed=D, heads_first=heads_first, extra=0)
    assert kc.shape[0] * page == n
    # keys and values as the end of one allocation each, value elements told apart by their size
    caches = []
    for c in (kc, vc):
        t = c.transpose(1, 2) if heads_first else c
        whole = torch.empty((8 + t.numel(),), dtype=t.dtype, device=t.device)
        part = whole[8:].view(t.shape)
        part.copy_(t * torch.linspace(0.5, 4.0, D, device=t.device).to(t.dtype) if c is vc else t)
        caches.append(part.transpose(1, 2) if heads_first else part)
    case = (q, *caches, table, lengths)
    check(*case, *run(case))
