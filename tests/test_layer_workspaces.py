"""A workspace taken once for the largest batch serves every smaller one (CPU: the calls' own
checks of its size, before a device is touched)."""
import pytest

import tensor_core_matrix_amd as tcm
from test_layer_abi import PASSED, WORKSPACE, _device_visible, lora

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
