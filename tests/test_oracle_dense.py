"""Pins of the dense block's and MXFP4's references (oracle/dense_oracle.py)."""
import numpy as np
import pytest
import torch

import oracle.dense_oracle as do


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gate_matches_torch_and_differences(kind):
    a = np.linspace(-12, 12, 2001)
    f, df = do.act(a, kind)
    t = torch.from_numpy(a).requires_grad_()
    y = torch.nn.functional.silu(t) if kind == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    y.sum().backward()
    np.testing.assert_allclose(f, y.detach().numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(df, t.grad.numpy(), rtol=1e-10, atol=1e-13)
    e = 1e-6
    np.testing.assert_allclose(df, (do.act(a + e, kind)[0] - do.act(a - e, kind)[0]) / (2 * e), atol=1e-8)
    # what the bounds of the kernels' tests use
    assert np.abs(df).max() <= 1.13 and np.abs(np.diff(df) / np.diff(a)).max() <= 1.13


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward_matches_differences(kind):
    g = np.random.default_rng(3)
    T, H, I = 5, 6, 4
    p = {"x": g.normal(size=(T, H)), "wg": g.normal(size=(I, H)), "wu": g.normal(size=(I, H)),
         "wd": g.normal(size=(H, I))}
    dy = g.normal(size=(T, H))
    r = do.ffn_forward(p["x"], p["wg"], p["wu"], p["wd"], kind)
    b = do.ffn_backward(p["x"], r["a"], r["b"], p["wg"], p["wu"], p["wd"], dy, kind)
    for n in p:
        for i in np.ndindex(p[n].shape):
            v = []
            for s in (1e-6, -1e-6):
                q = {k: a.copy() for k, a in p.items()}
                q[n][i] += s
                v.append((dy * do.ffn_forward(q["x"], q["wg"], q["wu"], q["wd"], kind)["y"]).sum())
            assert abs(b["d" + n][i] - (v[0] - v[1]) / 2e-6) < 1e-7 * max(1, abs(b["d" + n][i])), (n, i)


def test_mxfp4_worked_values():
    v = np.zeros((1, 64))
    # amax 6 -> scale 127 (2^0): every value and midpoint of the grid, ties to the even code
    v[0, :16] = [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0]
    v[0, 16:20] = [-0.25, -0.26, 5.01, -6]
    v[0, 32] = 7.9                                   # floor(log2) = 2: saturates at 6
    c, s = do.mxfp4_quantize(v)
    assert s.tolist() == [[127, 127]]
    assert c[0, :20].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 0, 2, 2, 4, 4, 6, 6, 8, 8, 9, 7, 15]
    assert c[0, 32] == 7
    np.testing.assert_array_equal(do.unpack(do.pack(c)), c)
    assert do.mxfp4_values(do.pack(c), s)[0, 32] == 6
    v[0, 5] = np.nan
    v[0, 40] = np.inf
    c, s = do.mxfp4_quantize(v)
    assert s.tolist() == [[255, 255]] and not c.any()
    assert np.isnan(do.mxfp4_values(do.pack(c), s)).all()
    z = do.mxfp4_quantize(np.zeros((2, 32)))
    assert not z[0].any() and not z[1].any()


def test_mxfp4_scales_over_the_range():
    for e in range(-133, 128):
        v = np.full((1, 32), 2.0 ** e)
        c, s = do.mxfp4_quantize(v)
        assert s[0, 0] == max(0, e - 2 + 127)
        got = do.mxfp4_values(do.pack(c), s)
        if e - 2 >= -127:
            np.testing.assert_array_equal(got, v)
        else:                                        # below the smallest scale: the grid of 2^-128
            assert np.abs(got - v).max() <= 2.0 ** -129
