"""Calls with more workgroups than a launch holds take longer chunks, or are refused before the device
is asked where even one chunk a sequence and head is too many (CPU)."""
import pytest

from test_layer_abi import PASSED, UNSUP_SHAPE, _device_visible, attn, cache, heads

pytestmark = pytest.mark.skipif(_device_visible(), reason="stand-in pointers must not reach a device")


def test_attention():
    """256 threads a workgroup, a workgroup a sequence and head and chunk: 2^32 threads are one too many."""
    def call(B, H, most):
        view = dict(q=heads(ts=H * 8, hs=8), out=heads(0x30000, ts=H * 8, hs=8))
        return attn(B=B, Hq=H, Hk=H, D=8, most=most, ts=1 << 16, c=cache(ks=(H * 128, H * 8, 8), vs=(H * 128, H * 8, 8)),
                    ws=0x90000, nb=1 << 50, **view)

    assert call(32768, 511, 1024) in PASSED
    assert call(32768, 512, 1024) == UNSUP_SHAPE
    assert call(32768, 256, 1024) in PASSED and call(32768, 256, 1025) in PASSED and call(65535, 200, 1 << 20) in PASSED
    assert call(65535, 256, 1024) in PASSED and call(65535, 257, 1024) == UNSUP_SHAPE
