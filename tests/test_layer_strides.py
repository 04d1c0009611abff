"""Strides of dimensions of one element are not looked at (CPU: the checks of the C ABI)."""
import pytest

import tensor_core_matrix_amd as tcm
from test_layer_abi import (BADSHAPE, MISALIGNED, PASSED, P, _device_visible, attn, bwd, cache, fwd, heads, into, lora,
                            rope)

pytestmark = pytest.mark.skipif(_device_visible(), reason="stand-in pointers must not reach a device")
ODD = [-8, 0, 1, 3, 68, (1 << 41) + 8, (1 << 62) + 1, -(1 << 63)]


@pytest.mark.parametrize("odd", ODD)
def test_one_of_a_dimension(odd):
    assert lora(M=1, ldx=odd, ldo=odd) in PASSED
    one = [heads(p, ts=odd) for p in P[:6]]
    assert fwd(*one[:4], T=1) in PASSED and bwd(*one, T=1) in PASSED
    assert into(v=one[0], T=1) in PASSED
    assert attn(q=one[0], out=one[1], B=1) in PASSED
    single = [heads(p, hs=odd) for p in P[:4]]
    assert fwd(k=single[1], ko=single[3], Hk=1) in PASSED
    assert fwd(*single, Hq=1, Hk=1) in PASSED
    c = cache(pages=1, page_size=1, ks=(odd, odd, odd), vs=(odd, odd, odd))
    assert into(c, Hk=1) in PASSED and attn(c=c, Hk=1, B=1) in PASSED


def test_two_of_a_dimension():
    assert lora(M=2, ldx=56) == BADSHAPE and lora(M=2, ldx=68) == MISALIGNED and lora(M=0, ldx=56) == BADSHAPE
    assert fwd(q=heads(ts=516), T=2) == MISALIGNED and fwd(q=heads(ts=-512), T=2) == BADSHAPE
    assert fwd(q=heads(hs=68), T=1) == MISALIGNED
    for i in range(3):
        ks = [2048, 128, 64]
        ks[i] = 68
        assert into(cache(ks=tuple(ks))) == MISALIGNED and attn(c=cache(vs=tuple(ks))) == MISALIGNED
