"""The float64 oracle of the layer operators against other forms of their definitions."""
import math

import numpy as np
import pytest
import torch

import tensor_core_matrix_amd as tcm
from oracle import layer as ol


def rng(seed):
    return np.random.default_rng(seed)


def test_lora_rows_against_merged_weights():
    """A row with an adapter is a product with W + s B A; one without, with W."""
    g = rng(1)
    M, N, K, L, R = 6, 7, 16, 3, 8
    x, w = g.normal(size=(M, K)), g.normal(size=(N, K))
    a, b = g.normal(size=(L, R, K)), g.normal(size=(L, N, R))
    rows, scales, ranks = [0, 2, -1, 1, 7, 2], g.normal(size=L), [8, 3, 0]
    out, s = ol.lora(x, w, a, b, rows, scales, ranks)
    for i, r in enumerate(rows):
        wm = w.copy()
        if 0 <= r < L:
            wm += scales[r] * b[r, :, :ranks[r]] @ a[r, :ranks[r]]
        np.testing.assert_allclose(out[i], wm @ x[i], rtol=1e-12, atol=1e-12)
    assert (s >= np.abs(out) - 1e-12).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_one_of_the_plane(layout):
    """A pair turns as a complex number; lengths stay; position 0 and the rest of the
    head stay; back undoes it."""
    g = rng(2)
    T, H, D, rot = 4, 3, 24, 16
    n = g.normal(size=(T, H, D))
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    pos = [0, 1, 12345, 2**31 - 1]
    y = ol.rotate(n, pos, f, layout)
    lo, hi = ol._pairs(rot, layout)
    z = (n[..., lo] + 1j * n[..., hi]) * np.exp(1j * np.outer([0, 1, 12345, 0], f))[:, None]
    np.testing.assert_allclose(y[:3][..., lo], z[:3].real, atol=1e-11)
    np.testing.assert_allclose(y[:3][..., hi], z[:3].imag, atol=1e-11)
    np.testing.assert_allclose(y[..., lo] ** 2 + y[..., hi] ** 2, n[..., lo] ** 2 + n[..., hi] ** 2, rtol=1e-12)
    assert (y[0] == n[0]).all() and (y[..., rot:] == n[..., rot:]).all()
    np.testing.assert_allclose(ol.rotate(y, pos, f, layout, back=True), n, atol=1e-12)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_gradients_against_differences(layout, norm):
    """norm_rope_bwd against central differences of norm_rope."""
    g = rng(3)
    T, H, D, rot = 2, 2, 16, 8
    x, dy = g.normal(size=(T, H, D)), g.normal(size=(T, H, D))
    w = 1 + 0.2 * g.normal(size=D) if norm else None
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    pos = [3, 100]
    args = dict(eps=1e-3, layout=layout, factor=1.3, norm=norm)
    loss = lambda x, w: (dy * ol.norm_rope(x, pos, f, w, **args)).sum()  # noqa: E731
    dx, dw, _, _ = ol.norm_rope_bwd(dy, x, pos, f, w, **args)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for d in range(D if norm else 0):
        e = np.zeros(D)
        e[d] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[d]) < 1e-7


def test_attention_against_torch_softmax():
    """A sequence whose pages lie in order is softmax attention over its keys."""
    g = rng(4)
    Hq, Hk, D, ps, n = 4, 2, 8, 4, 11
    k, v = g.normal(size=(3, ps, Hk, D)), g.normal(size=(3, ps, Hk, D))
    q = g.normal(size=(1, Hq, D))
    out, lse, mag, _ = ol.paged_attention(q, k, v, np.array([[0, 1, 2]]), [n], ps, 0.3)
    kk, vv = (torch.from_numpy(t.reshape(-1, Hk, D)[:n]) for t in (k, v))
    for h in range(Hq):
        s = 0.3 * (kk[:, h // 2] @ torch.from_numpy(q[0, h]))
        np.testing.assert_allclose(out[0, h], (torch.softmax(s, 0) @ vv[:, h // 2]).numpy(), rtol=1e-12)
        assert abs(lse[0, h] - float(torch.logsumexp(s, 0))) < 1e-12
    assert (mag >= np.abs(out) - 1e-12).all()


def test_attention_windows_holes_and_empty_rows():
    g = rng(5)
    k, v = g.normal(size=(4, 2, 1, 8)), g.normal(size=(4, 2, 1, 8))
    q = g.normal(size=(4, 1, 8))
    table = np.array([[0, 1, 2], [3, -1, 0], [1, 2, 9], [-1, -1, -1]])
    out, lse, _, _ = ol.paged_attention(q, k, v, table, [6, 6, 0, 6], 2, 1.0, window=3)
    # row 0: keys 3, 4, 5 = the second of page 1 and page 2
    kk = np.concatenate([k[1, 1:, 0], k[2, :, 0]])
    vv = np.concatenate([v[1, 1:, 0], v[2, :, 0]])
    p = np.exp(kk @ q[0, 0])
    np.testing.assert_allclose(out[0, 0], p @ vv / p.sum(), rtol=1e-12)
    # row 1: key 3 lies in a hole; rows 2 and 3 have no key
    p = np.exp(k[0, :, 0] @ q[1, 0])
    np.testing.assert_allclose(out[1, 0], p @ v[0, :, 0] / p.sum(), rtol=1e-12)
    assert (out[2:] == 0).all() and np.isneginf(lse[2:]).all()


def test_half_ulp():
    for name, dt in (("bf16", torch.bfloat16), ("f16", torch.float16)):
        x = torch.tensor([1.0, 1.5, 3.0, 1e-3, 100.0], dtype=dt)
        up = torch.nextafter(x, torch.full_like(x, math.inf)) if name == "f16" else \
            (x.view(torch.int16) + 1).view(dt)
        np.testing.assert_allclose(ol.half_ulp(x.double().numpy(), name),
                                   (up.double() - x.double()).numpy() / 2, rtol=0)
    assert ol.half_ulp(np.array([1.0, 1e-9]), "e4m3").tolist() == [2.0**-4, 2.0**-10]


# ---- frequencies ----------------------------------------------------------------------

def test_frequencies_plain_and_linear():
    f, factor = tcm.rope_frequencies(8, base=100.0)
    assert f.dtype == torch.float64 and factor == 1.0
    np.testing.assert_allclose(f.numpy(), [1.0, 100 ** -0.25, 0.1, 100 ** -0.75], rtol=1e-15)
    g, factor = tcm.rope_frequencies(8, base=100.0, scaling="linear", ratio=4.0)
    np.testing.assert_allclose(g.numpy(), f.numpy() / 4, rtol=1e-15)
    assert factor == 1.0


def test_frequencies_ntk_keeps_the_highest_and_divides_the_lowest():
    f, _ = tcm.rope_frequencies(64)
    g, factor = tcm.rope_frequencies(64, scaling="ntk", ratio=8.0)
    assert g[0] == f[0] and factor == 1.0
    np.testing.assert_allclose(g[-1], f[-1] / 8, rtol=1e-12)


@pytest.mark.parametrize("scaling", ["yarn", "bands"])
def test_frequencies_by_parts(scaling):
    """Many turns over the trained context: kept; less than one: divided; between: between,
    and monotonous."""
    kw = dict(ratio=16.0, trained=4096, low=1.0, high=32.0)
    f, _ = tcm.rope_frequencies(128)
    g, factor = tcm.rope_frequencies(128, scaling=scaling, **kw)
    turns = 4096 * f / (2 * math.pi)
    share = (g / f - 1 / 16) / (1 - 1 / 16)
    assert torch.allclose(share[turns > 40], torch.ones(1, dtype=torch.float64), atol=1e-12)
    assert torch.allclose(share[turns < 0.8], torch.zeros(1, dtype=torch.float64), atol=1e-12)
    assert (share[1:] <= share[:-1] + 1e-12).all() and 0 < share[(turns > 4) & (turns < 8)].mean() < 1
    assert factor == (0.1 * math.log(16.0) + 1.0 if scaling == "yarn" else 1.0)
    one, factor = tcm.rope_frequencies(128, scaling=scaling, **{**kw, "ratio": 1.0})
    assert torch.allclose(one, f, rtol=1e-15) and factor == 1.0


def test_frequencies_refuse():
    for args in (dict(rot_dim=7), dict(rot_dim=8, scaling="no"), dict(rot_dim=2, scaling="ntk", ratio=2.0),
                 dict(rot_dim=8, scaling="yarn", ratio=2.0),
                 dict(rot_dim=8, scaling="bands", ratio=2.0, trained=64, low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            tcm.rope_frequencies(**args)
    assert tcm.rope_frequencies(0)[0].shape == (0,)
