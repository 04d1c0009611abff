"""add_rms_norm onto its own operands, where the sum is asked for nowhere else: the sum that it returns."""
import pytest
import torch

import tensor_core_matrix_amd as tcm
from test_gpu_norm import BF, DEV, F32, HF, check, rand, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("T,D", [(1, 8), (3, 512), (7, 4096), (2, 8200)])
def test_result_onto_x_without_a_residual(T, D, dt):
    x, w = rand((T, D), 1, dt), weight("f32", D, dt)
    a = x.clone()
    y, s = tcm.add_rms_norm(a, w, out=a)
    assert y is a and torch.equal(s, x)
    check(x, None, w, y, s)
    # the gradients that begin with that sum are those of a call that kept x
    dy = rand((T, D), 2, dt)
    for got, want in zip(tcm.add_rms_norm_bwd(dy, s, w), tcm.add_rms_norm_bwd(dy, x, w)):
        assert torch.equal(got, want)


def test_rows_of_a_wider_tensor():
    wide = rand((5, 3 * 64), 3, BF)
    keep = wide.clone()
    x = wide[:, 64:128]
    y, s = tcm.add_rms_norm(x, out=x)
    assert torch.equal(s, keep[:, 64:128]) and torch.equal(wide[:, :64], keep[:, :64]) and torch.equal(wide[:, 128:], keep[:, 128:])
    check(keep[:, 64:128], None, None, y, s)


def test_another_view_of_x():
    """The same memory through another tensor."""
    x = rand((4, 128), 4, HF)
    a = x.clone()
    y, s = tcm.add_rms_norm(a, out=a.view(2, 2, 128).view(4, 128))
    assert torch.equal(s, x)
    check(x, None, None, a, s)


def test_a_sum_that_is_given_and_one_that_is_x():
    x = rand((4, 128), 5, BF)
    a, into = x.clone(), torch.zeros_like(x)
    y, s = tcm.add_rms_norm(a, out=a, sum_out=into)
    assert s is into and torch.equal(s, x)
    y, s = tcm.add_rms_norm(x)
    assert s is x  # nothing is copied where x stays
    y, s = tcm.add_rms_norm(x, out_dtype=F32)
    assert s is x


def test_no_rows():
    x = torch.empty((0, 64), dtype=BF, device=DEV)
    assert tcm.add_rms_norm(x)[1] is x and tcm.add_rms_norm(x, out=x)[1] is x
