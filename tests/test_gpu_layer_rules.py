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


def lora_case(M, N, K, R, L, dt, odt, seed, each):
    from test_gpu_lora import check as lora_check
    from test_gpu_lora import draw

    import tensor_core_matrix_amd as tcm

    x, w, a, b, rows, scales = draw(M, N, K, L, R, dt, seed)
    if not each:
        rows = torch.tensor([i * 3 // M - 1 for i in range(M)], dtype=torch.int32, device="cuda")
    out = tcm.lora_gemm_tn(x, w, a, b, rows, scales=scales, out_dtype=odt)
    lora_check(out, x, w, a, b, rows, scales)


# rows x columns on both sides of each choice of the adapters' product for 256 compute units: 16 and
# 32 columns a workgroup (8160, 8161 columns, from 17 rows on), rows and tiles (64, 65), 64 x 64
# and 128 x 64 tiles (191 and 192 of the latter), 128 x 128 (255 and 256) and 256 x 256
@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("M,N", [(16, 8161), (17, 8160), (17, 8161), (64, 8161), (64, 100), (65, 100), (128, 12224),
                                 (128, 12225), (128, 32640), (128, 32641), (256, 65281)])
def test_adapters_by_size(M, N, each):
    for dt, odt in ((torch.bfloat16, torch.float32), (torch.float16, torch.float16)):
        lora_case(M, N, 72, 40, 5, dt, odt, M + N, each)


@pytest.mark.parametrize("M", [1, 15, 16, 256, 257])
@pytest.mark.parametrize("K", [1016, 2048, 8192, 8200])
def test_adapters_parts_of_k(M, K):
    """One, two, four and eight parts of K, the last one short; a workgroup an adapter and a
    workgroup a block of rows."""
    lora_case(M, 40, K, 24, 3, torch.bfloat16, torch.bfloat16, M + K, True)
    lora_case(M, 40, K, 128, 3, torch.float16, torch.float32, M + K, True)


@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 1, 1, 16, 16), (513, 1, 1, 64, 64), (2047, 3, 1, 128, 128),
                                           (2048, 3, 1, 128, 128), (9000, 2, 1, 64, 16), (70, 40, 1, 240, 224)])
def test_rotation_tokens_a_workgroup(T, Hq, Hk, D, rot):
    """One token a workgroup and several, heads spread over workgroups, one head of a kind."""
    import numpy as np

    import tensor_core_matrix_amd as tcm
    from oracle import layer as ol
    from test_gpu_rope import close, f64, freqs, gen, normal, tolerance

    g = gen(T)
    qkv = normal((T, Hq + Hk, D), g, torch.bfloat16)
    q, k = qkv.split([Hq, Hk], 1)
    w, f = normal((D,), g, torch.bfloat16, 0.2, 1.0), freqs(rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37
    qo, ko = tcm.qk_norm_rope(q, k, pos, f, w, w)
    at = np.unique(np.linspace(0, T - 1, 40).astype(int))  # (the oracle goes token by token)
    for x, o in ((q, qo), (k, ko)):
        xs, p = f64(x)[at], pos.cpu().numpy()[at]
        ref = ol.norm_rope(xs, p, f64(f), f64(w))
        close(o[torch.from_numpy(at)], ref, tolerance(ref, xs, f64(f), "half", 1.0, f64(w)), "bf16")
