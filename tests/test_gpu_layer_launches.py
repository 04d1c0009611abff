"""Attention of so many sequences and heads that their chunks pass what a launch holds."""
import pytest
import torch

import tensor_core_matrix_amd as tcm
from test_gpu_paged_attention import check

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_chunks_that_pass_a_launch():
    """65535 sequences of 64 heads and five chunks of 1024 keys are 2^24.3 workgroups: four of 1280
    are taken.  Most sequences are short; those that are not are looked at."""
    B, H, D, page, n = 65535, 64, 8, 512, 5000
    g = torch.Generator(device=DEV).manual_seed(1)
    normal = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    kc, vc, q = normal(20, page, H, D), normal(20, page, H, D), normal(B, H, D)
    table = torch.randint(0, 20, (B, -(-n // page)), generator=g, device=DEV).to(torch.int32)
    lengths = torch.randint(0, 3, (B,), generator=g, device=DEV).to(torch.int32)
    seen = [0, 1, 777, 40000, B - 2, B - 1]
    lengths[seen] = torch.tensor([n, 1280, 1281, 3840, 3841, 2560], dtype=torch.int32, device=DEV)
    out = tcm.paged_attention(q, kc, vc, table, lengths, max_len=n)
    seen += [2, 3, 60000]
    check(q[seen], kc, vc, table[seen], lengths[seen], out[seen], None)
