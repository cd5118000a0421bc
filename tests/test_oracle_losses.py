"""Pins of the router losses' float64 reference against something other than its own formula."""
import numpy as np
import pytest

import oracle
import oracle.losses_oracle as lo


def inputs(T=9, E=7, k=3, seed=0):
    g = np.random.default_rng(seed)
    logits = g.normal(size=(T, E)) * 2
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    mask = g.random(T) < 0.7
    return logits, ids, mask, g


def test_losses_by_loops():
    import math
    logits, ids, mask, _ = inputs()
    for m in (None, mask):
        r = lo.losses(logits, ids, m)
        keep = range(9) if m is None else np.nonzero(m)[0]
        count, prob, z = [0] * 7, [0.0] * 7, 0.0
        for t in keep:
            den = math.fsum(math.exp(v) for v in logits[t])
            z += math.log(den) ** 2
            for e in range(7):
                prob[e] += math.exp(logits[t, e]) / den
                count[e] += int((ids[t] == e).sum())
        n = len(keep)
        share = [c / (3 * n) for c in count]
        assert r["counts"].tolist() == count and r["n"] == n
        np.testing.assert_allclose(r["prob_sum"], prob, rtol=1e-13)
        np.testing.assert_allclose(r["losses"], [7 * sum(a * b / n for a, b in zip(share, prob)), z / n], rtol=1e-13)


def test_even_loads_give_one():
    """Every expert picked equally often: the balance loss is 1 whatever the probabilities; all on one expert with
    probability 1: E / k of it."""
    logits, _, _, g = inputs(T=14)
    ids = (np.arange(42) % 7).reshape(14, 3)
    np.testing.assert_allclose(lo.losses(logits, ids)["losses"][0], 1, rtol=1e-14)
    one = np.full((5, 7), -np.inf)
    one[:, 2] = 3.0
    r = lo.losses(one, np.full((5, 1), 2))
    np.testing.assert_allclose(r["losses"], [7, 9], rtol=1e-14)


@pytest.mark.parametrize("masked", [False, True])
def test_backward_against_differences(masked):
    logits, ids, mask, g = inputs()
    mask = mask if masked else None
    dl = np.array([0.7, -0.3])
    w, gw = g.random((9, 3)), g.normal(size=(9, 3))
    sel0 = np.take_along_axis(logits, ids.astype(np.int64), 1)
    w = np.exp(sel0) / np.exp(sel0).sum(1, keepdims=True)

    def f(v):
        sel = np.take_along_axis(v, ids.astype(np.int64), 1)
        ww = np.exp(sel) / np.exp(sel).sum(1, keepdims=True)
        return (dl * lo.losses(v, ids, mask)["losses"]).sum() + (gw * ww).sum()

    d = lo.losses_backward(lo.losses(logits, ids, mask), ids, dl, w, gw)
    for t in range(9):
        for e in range(7):
            h = np.zeros_like(logits)
            h[t, e] = 1e-6
            np.testing.assert_allclose((f(logits + h) - f(logits - h)) / 2e-6, d[t, e], rtol=1e-6, atol=1e-9)


def test_selection_part_is_the_routers():
    """Without the losses the gradient is the router oracle's, and through the products its dx and dWr."""
    logits, ids, _, g = inputs()
    x, wr = g.normal(size=(9, 16)), g.normal(size=(7, 16))
    w, gw = g.random((9, 3)), g.normal(size=(9, 3))
    d = lo.losses_backward(lo.losses(logits, ids), ids, (0, 0), w, gw)
    _, dl, dwr, dx = oracle.router_backward(x, wr, ids, w, gw)
    np.testing.assert_allclose(d, dl, rtol=1e-14, atol=1e-16)
    a, b = lo.logits_backward(x, wr, d)
    np.testing.assert_allclose(a, dx, rtol=1e-13, atol=1e-15)
    np.testing.assert_allclose(b, dwr, rtol=1e-13, atol=1e-15)
    np.testing.assert_array_equal(lo.logits_backward(x, wr, d, x)[0], a + x)


def test_nothing_left():
    logits, ids, _, _ = inputs()
    r = lo.losses(logits, ids, np.zeros(9))
    assert (r["losses"] == 0).all() and r["n"] == 0 and (r["counts"] == 0).all()
    assert (lo.losses_backward(r, ids, (1.0, 1.0)) == 0).all()
    logits[4] = -np.inf
    r = lo.losses(logits, ids)
    assert (r["p"][4] == 0).all() and r["lse"][4] == 0 and (lo.losses_backward(r, ids, (1.0, 1.0))[4] == 0).all()
