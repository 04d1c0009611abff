"""A workspace taken once for the largest batch serves every smaller one (CPU: the calls' own
checks of its size, before a device is touched)."""
import pytest

import tensor_core_matrix_amd as tcm
from test_layer_abi import NULLP, PASSED, WORKSPACE, _device_visible, attn, heads, lora

pytestmark = pytest.mark.skipif(_device_visible(), reason="stand-in pointers must not reach a device")


@pytest.mark.parametrize("R", [8, 128])
@pytest.mark.parametrize("K", [8, 1016, 2048, 4096, 8192, 9216, 1 << 20])
@pytest.mark.parametrize("M", [1, 5, 15, 16, 17, 64, 300, 4096, 4097, 5000, 5456, 5457, 8192, 8193, 20000])
def test_adapters(M, K, R):
    """Every smaller number of rows about the steps of the parts of K, and smaller K and R."""
    need = tcm.lora_workspace(M, K, R)
    for m in sorted({1, 2, 14, 15, 16, 17, 63, 255, 256, 257, 340, 4080, 4096, 4097, 5456, 5457, 8191, 8192, 8193, M}):
        for k in sorted({8, 2040, 2048, 3000, 4096, 5120, 8192, 9216, K}):
            if m > M or k > K:
                continue
            for r in {8, R}:
                assert lora(M=m, K=k, ldx=k, R=r, nb=need) in PASSED, (m, k, r)
                assert tcm.lora_workspace(m, k, r) <= need
    if M >= 16 and K >= 4096:  # (and the size is looked at)
        assert lora(M=M, K=K, ldx=K, R=R, nb=M * R * 4 - 16) == WORKSPACE


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (32, 8), (64, 1), (40, 1), (8, 8), (128, 128), (1, 1), (64, 4)])
@pytest.mark.parametrize("most", [1, 256, 257, 700, 1024, 1025, 4096, 40000, 262144, 262145, 1 << 20])
def test_attention(most, Hq, Hk):
    """Every smaller batch (all up to 150, some beyond), shorter bounds and windows."""
    D = 16
    view = dict(q=heads(ts=Hq * D, hs=D), out=heads(0x30000, ts=Hq * D, hs=D), Hq=Hq, Hk=Hk, D=D, ts=1 << 17, ws=0x90000)
    for B in (1, 2, 5, 33, 64, 127, 128, 150, 1000, 4000):
        need = tcm.paged_attention_workspace(B, Hq, Hk, D, most)
        for b in sorted({*range(1, min(B, 150) + 1), 255, 256, 257, 511, 512, 1000, B}):
            if b > B:
                continue
            for span in {1, 600, 1025, most // 2, most}:
                if span > most:
                    continue
                for window in (0, 300):
                    assert attn(B=b, most=span, window=window, nb=need, **view) in PASSED, (B, b, span, window)
        assert need <= 4 * (D + 2) * Hq * max(2 * 1024, B * 256)
    small = tcm.paged_attention_workspace(1, Hq, Hk, D, 256)
    assert small == 0  # one chunk: no parts to join


def test_attention_without_a_workspace_where_parts_need_one():
    view = dict(q=heads(ts=128, hs=16), out=heads(0x30000, ts=128, hs=16), D=16, ts=1 << 17)
    assert attn(B=1, most=5000, **view) == NULLP and attn(B=1, most=5000, ws=0x90000, nb=16, **view) == WORKSPACE
