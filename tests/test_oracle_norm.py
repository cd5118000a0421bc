"""Pins of the norm's float64 reference against something other than its own formula."""
import numpy as np
import pytest

import oracle.norm_oracle as no
from oracle import bf16_round


def inputs(T=5, H=24, seed=0):
    g = np.random.default_rng(seed)
    return (bf16_round(g.normal(size=(T, H)) * 2), bf16_round(g.normal(size=(T, H))), 1 + 0.3 * g.normal(size=H),
            g.normal(size=(T, H)), g.normal(size=(T, H)))


def test_forward_has_unit_rms_and_keeps_the_stream():
    x, r, w, _, _ = inputs()
    y, z, rstd = no.norm_forward(x, None, r, eps=1e-300)
    np.testing.assert_allclose((y ** 2).mean(1), 1, rtol=1e-14)
    np.testing.assert_allclose(y / rstd[:, None], z, rtol=1e-14)
    assert (np.abs(z - (x + r)) <= 2.0 ** -8 * np.abs(x + r)).all() and (bf16_round(z) == z).all()
    # the norm of the stored stream is the same one; scaling the input changes nothing but rstd
    np.testing.assert_array_equal(no.norm_forward(z, None, None, eps=1e-300)[0], y)
    np.testing.assert_allclose(no.norm_forward(8 * z, w, None, eps=1e-300)[0], no.norm_forward(z, w, None, 1e-300)[0],
                               rtol=1e-14)
    np.testing.assert_allclose(no.norm_forward(z, w, None, 0.5)[0],
                               w * z / np.sqrt((z ** 2).sum(1, keepdims=True) / 24 + 0.5), rtol=1e-14)


@pytest.mark.parametrize("with_w", [True, False])
def test_backward_against_differences(with_w):
    x, _, w, dy, d_sum = inputs()
    w = w if with_w else None
    _, z, rstd = no.norm_forward(x, w)
    dx, dw = no.norm_backward(dy, z, rstd, w, d_sum)
    # <dy, y> + <d_sum, z>, whose gradient in z is dx
    f = lambda zz, ww: (dy * no.norm_forward(zz, ww)[0]).sum() + (d_sum * zz).sum()  # noqa: E731
    h = 1e-6
    for t in range(z.shape[0]):
        for c in range(z.shape[1]):
            d = np.zeros_like(z)
            d[t, c] = h
            np.testing.assert_allclose((f(z + d, w) - f(z - d, w)) / (2 * h), dx[t, c], rtol=1e-6, atol=1e-7)
    if with_w:
        for c in range(z.shape[1]):
            d = np.zeros_like(w)
            d[c] = h
            np.testing.assert_allclose((f(z, w + d) - f(z, w - d)) / (2 * h), dw[c], rtol=1e-6, atol=1e-7)


def test_gradient_is_orthogonal_to_the_row():
    """Scaling a row does not change its norm (eps aside), so dx of a unit weight has no part along it."""
    x, _, w, dy, _ = inputs(seed=3)
    _, z, rstd = no.norm_forward(x, w, None, eps=1e-300)
    dx, _ = no.norm_backward(dy, z, rstd, w)
    assert (np.abs((dx * z).sum(1)) < 1e-12 * np.abs(dx * z).sum(1)).all()
