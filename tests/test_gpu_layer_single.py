"""Strides of dimensions of one element step to nowhere: any are taken."""
import pytest
import torch

import tensor_core_matrix_amd as tcm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def normal(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("stride", [1, 3, 68, (1 << 21) + 8, 1 << 33])
def test_one_row(stride):
    x, w, a, b = normal(1, 64), normal(32, 64, seed=1), normal(2, 16, 64, seed=2), normal(2, 32, 16, seed=3)
    rows = torch.ones(1, dtype=torch.int32, device=DEV)
    want = tcm.lora_gemm_tn(x, w, a, b, rows)
    out = torch.empty((1, 32), dtype=torch.bfloat16, device=DEV).as_strided((1, 32), (stride, 1))
    tcm.lora_gemm_tn(x.as_strided((1, 64), (stride, 1)), w, a, b, rows, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("stride", [1, 3, 68, 1 << 42])
def test_one_token_and_one_head(stride):
    pos, f = torch.full((1,), 7, dtype=torch.int32, device=DEV), tcm.rope_frequencies(64, device=DEV)[0]
    q, k = normal(1, 4, 64), normal(1, 1, 64, seed=1)
    want = tcm.qk_norm_rope(q, k, pos, f)
    odd = lambda t: t.as_strided(t.shape, (stride, t.stride(1) if t.shape[1] > 1 else stride, 1))  # noqa: E731
    got = tcm.qk_norm_rope(odd(q), odd(k), pos, f, q_out=odd(torch.empty_like(q)), k_out=odd(torch.empty_like(k)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    grads = tcm.qk_norm_rope_bwd(q, k, q, k, pos, f)
    got = tcm.qk_norm_rope_bwd(odd(q), odd(k), odd(q), odd(k), pos, f, dq=odd(torch.empty_like(q)))
    assert all(torch.equal(a, b) for a, b in zip(got[:2], grads[:2]))


@pytest.mark.parametrize("stride", [1, 3, 68, 1 << 42])
def test_a_cache_of_one_page_one_place_one_head(stride):
    q, kc, vc = normal(1, 4, 64), normal(1, 1, 1, 64, seed=1), normal(1, 1, 1, 64, seed=2)
    table, n = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    odd = lambda t: t.as_strided(t.shape, (stride,) * (t.dim() - 1) + (1,))  # noqa: E731
    out = tcm.paged_attention(q.as_strided(q.shape, (stride, 64, 1)), odd(kc), odd(vc), table, n)
    assert torch.equal(out, vc.view(1, 1, 64).expand(1, 4, 64))
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    pos = torch.zeros(1, dtype=torch.int32, device=DEV)
    tcm.qk_norm_rope_cache(q, odd(kc[0]), odd(vc[0]), pos, None, odd(k2), odd(v2), pos, norm=False)
    assert torch.equal(k2, kc) and torch.equal(v2, vc)
