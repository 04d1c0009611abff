"""The rotation's angles at the largest positions."""
import math

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_angles_of_large_positions(layout):
    """(1, 0) turned by an angle near a whole number of half turns: its sine is small, so fp16 holds
    it to far below the angle's error.  The angle is fp32 after its reduction, at most half an ulp
    of one half turn off (2^-25 pi = 9.4e-8), and the sine of so small a remainder as exact as its
    argument."""
    g = np.random.default_rng(1)
    T, D = 64, 64
    pos = np.concatenate([g.integers(2**30, 2**31 - 1, T // 2), g.integers(1, 2**31 - 1, T // 2)])
    pos[0] = 2**31 - 1
    # frequency j turns position j into k half turns and a remainder of up to 6e-5 (as near as a
    # double comes), for the tokens t with t % 32 == j
    delta = g.uniform(-6e-5, 6e-5, 32)
    pi = np.longdouble("3.14159265358979323846264338327950288")
    freq = np.array([(np.longdouble(np.floor(g.uniform(0.1, 0.3) * pos[j])) * pi + np.longdouble(delta[j])) /
                     np.longdouble(int(pos[j])) for j in range(32)]).astype(np.float64)
    x = torch.zeros((T, 1, D), dtype=torch.float16)
    lo = torch.arange(32) if layout == "half" else 2 * torch.arange(32)
    hi = lo + 32 if layout == "half" else lo + 1
    x[..., lo] = 1.0
    xd = x.to(DEV)
    y, _ = tcm.qk_norm_rope(xd, xd, torch.from_numpy(pos.astype(np.int32)).to(DEV), torch.from_numpy(freq).to(DEV),
                            layout=layout, norm=False)
    y = y.double().cpu().numpy()[:, 0]
    seen = 0
    for t in range(T):
        for j in range(32):
            angle = np.longdouble(int(pos[t])) * np.longdouble(freq[j])
            rest = float(angle - pi * np.rint(angle / pi))
            if abs(rest) > 1.2e-4:
                continue  # (fp16's own rounding hides it)
            seen += 1
            sign = -1.0 if int(np.rint(angle / pi)) % 2 else 1.0
            want = sign * math.sin(rest)
            # half an fp16 ulp below 2^-13 (2^-25) beside the angle's error (2^-64 of a long double's
            # 4e8 radians is 2e-11)
            assert abs(y[t, hi[j]] - want) <= 1e-7 + 2.0 ** -25 + 1e-9, (t, j, pos[t], y[t, hi[j]] - want)
            assert abs(y[t, lo[j]] - sign) <= 2.0 ** -11
    assert seen >= 32
