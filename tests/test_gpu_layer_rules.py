"""The choices that the layer operators make by their sizes: both sides of each rule give
the oracle's result."""
import pytest
import torch

from test_gpu_paged_attention import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hk,n", [(4, 261120), (4, 261121), (8, 130048), (8, 130049), (8, 131072)])
def test_attention_a_head_a_wave(Hk, n):
    """Few sequences with much work: four key-value heads a workgroup from 256 chunks on;
    just below it and above, the last chunk full and of one key."""
    case = make(1, 2 * Hk, Hk, 16, [n], 64, torch.bfloat16, seed=n)
    check(*case, *run(case))


@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_attention_a_head_a_wave_ragged(kind):
    """The same with sequences that end early, one empty, groups of more than 16 heads, holes
    and pages that end inside tiles."""
    case = make(4, 80, 4, 32, [66000, 0, 1000, 31], 56, torch.float16, kind, seed=1)
    case[3][0, 10:400] = -1
    check(*case, *run(case))
