"""Refusals of a drafting step's operators that no other test reaches (CPU: before a device is touched)."""
import pytest
import torch

import tensor_core_matrix_amd as tcm
from test_layer_abi import PASSED, UNSUP_SHAPE, P, _device_visible, cache, heads
from test_step_abi import tree

pytestmark = pytest.mark.skipif(_device_visible(), reason="stand-in pointers must not reach a device")


def test_blocks_of_rows_of_all_heads_and_sequences():
    """B * Hk blocks of rows at most 2^30, whatever a block's size."""
    wide = dict(D=8, c=cache(ks=(16 * 65535 * 8, 65535 * 8, 8), vs=(16 * 65535 * 8, 65535 * 8, 8)),
                q=heads(ts=65535 * 8, hs=8), out=heads(P[7], ts=65535 * 8, hs=8), Hq=65535, Hk=65535)
    assert tree(B=16384, nodes=1, **wide) in PASSED
    assert tree(B=16385, nodes=1, **wide) == UNSUP_SHAPE
    assert tree(B=16384, nodes=17, **wide) in PASSED and tree(B=16385, nodes=17, **wide) == UNSUP_SHAPE
    assert tree(B=8192, nodes=256, words=4, **wide) in PASSED and tree(B=8193, nodes=256, words=4, **wide) == UNSUP_SHAPE
