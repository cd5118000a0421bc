"""The router's losses and its dense backward on the GPU against their float64
references, and a whole step around the layer.

Bounds, from the arithmetic (u = 2^-24; a rounding of fp32 is at most u of the
value). exp: the argument's rounding (|v - top| u) and 2 ulp, so a probability is
within (|v - top| + 40) u of itself: its own exponential, the sum of a lane's 8
and a butterfly's 6 additions, the same errors of the other terms in the
denominator (weighted by themselves, where |x| e^x <= 0.37 bounds theirs), a
reciprocal and a product. lse: the denominator's relative error (20 u), the
logarithm and the addition: (|lse| + 40) u. Sums over tokens: a lane adds at
most 2 + T / 2048 of them, then 6 + 4 + 64 + 8 partial sums."""
import numpy as np
import pytest

import mixture_experts_layer_30_amd as mok
import oracle
import oracle.losses_oracle as lo
import oracle.norm_oracle as no
from ffn_testlib import F32, HALF, assert_within, dot
from mixture_experts_layer_30_amd import functional as F
from oracle import bf16_round
from test_gpu_mxfp4 import bf, f64

pytestmark = pytest.mark.gpu


def f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def routing(T, E, k, seed=0, scale=2.0):
    g = np.random.default_rng(seed + 31 * T + 7 * E + k)
    logits = (g.normal(size=(T, E)) * scale + g.normal(size=E)).astype(np.float32).astype(np.float64)
    ids = np.argsort(-logits, 1)[:, :k].astype(np.int32)
    sel = np.take_along_axis(logits, ids.astype(np.int64), 1)
    w = np.exp(sel - sel.max(1, keepdims=True))
    w = (w / w.sum(1, keepdims=True)).astype(np.float32).astype(np.float64)
    gw = g.normal(size=(T, k)).astype(np.float32).astype(np.float64)
    return logits, ids, w, gw, g.random(T) < 0.7


def bounds(logits, ids, r, dl, w, g):
    """{name: largest error} of the sums and of d_logits."""
    T, E = logits.shape
    k, n = ids.shape[1], max(r["n"], 1)
    p, lse = r["p"], r["lse"]
    v = np.where(r["m"][:, None], logits, 0.0)
    top = v.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        far = np.where(np.isfinite(v), np.abs(v - top), 0.0)
    ep = p * (far + 40) * F32 + 1e-38
    el = (np.abs(lse) + 40) * F32
    chain = (100 + T / 2048) * F32
    eP = ep[r["m"]].sum(0) + chain * r["prob_sum"] + 1e-37
    c = r["counts"].astype(np.float64)
    z2 = (lse[r["m"]] ** 2).sum()
    losses = np.array([E / (k * n * n) * (c * eP).sum() + 4 * F32 * r["losses"][0],
                       ((2 * np.abs(lse) * el + el ** 2)[r["m"]].sum() + chain * z2) / n + 4 * F32 * r["losses"][1]])
    a = (E * c - k * n) / (k * n * n)              # counts from their mean, as the kernel takes them
    s = (p * a).sum(1, keepdims=True)
    es = (ep * np.abs(a)).sum(1, keepdims=True) + 16 * F32 * (p * np.abs(a)).sum(1, keepdims=True)
    gb, gz = abs(dl[0]), abs(dl[1]) * 2 / n
    d = gb * ((ep + 3 * F32 * p) * (np.abs(a - s) + es) + p * (es + 2 * F32 * (np.abs(a) + np.abs(s)))) \
        + gz * (ep * np.abs(lse)[:, None] + (p + ep) * (el + 4 * F32 * np.abs(lse))[:, None])
    d = np.where(r["m"][:, None], d, 0.0)
    if w is not None:
        sw = (w * g).sum(1, keepdims=True)
        e = np.abs(w) * ((k + 8) * F32 * np.abs(w * g).sum(1, keepdims=True) + 3 * F32 * (np.abs(g) + np.abs(sw)))
        hits = np.zeros_like(d)
        for t in range(T):
            for j in range(k):
                if 0 <= ids[t, j] < E:
                    d[t, ids[t, j]] += e[t, j]
                    hits[t, ids[t, j]] += np.abs(w * (g - sw))[t, j]
        d = d + (k + 1) * F32 * hits
    ref = lo.losses_backward(r, ids, dl, w, g)
    return {"losses": losses + 1e-38, "prob_sum": eP, "d_logits": d + 2 * F32 * np.abs(ref) + 1e-37}, ref


def check(T, E, k, mask=False, sel=True, dl=(0.5, -0.25), seed=0, data=None, inplace=False):
    import torch
    logits, ids, w, g, m = data or routing(T, E, k, seed)
    m = m if mask else None
    if not sel:
        w = g = None
    ws = F.get_router_workspace(T, 128, E, k)
    L, I = f32(logits), i32(ids)
    M = None if m is None else torch.from_numpy(np.asarray(m)).cuda()
    W, G = (None, None) if w is None else (f32(w), f32(g))
    D = f32(np.array(dl))
    o = F.run_router_losses(ws, L, I, mask=M)
    d = F.run_router_losses_backward(ws, L, I, o, D, topk_w=W, d_topk_w=G, mask=M)
    o2 = F.run_router_losses(ws, L, I, mask=M)
    d2 = torch.empty_like(L).copy_(L) if inplace else torch.full_like(L, 7.0)
    mok.router_losses_backward(ws.problem, d2 if inplace else L, I, o.counts, o.n_tokens, D, d2, W, G, mask=M)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, o2)) and torch.equal(d, d2)
    r = lo.losses(logits, ids, m)
    np.testing.assert_array_equal(o.counts.cpu().numpy(), r["counts"])
    assert int(o.n_tokens) == r["n"]
    b, ref = bounds(logits, ids, r, dl, w, g)
    assert_within(f64(o.prob_sum), r["prob_sum"], b["prob_sum"], "prob_sum")
    assert_within(f64(o.losses), r["losses"], b["losses"], "losses")
    assert_within(f64(d), ref, b["d_logits"], "d_logits")
    return o, d


# every number of experts at which another number of lanes, or of loads, begins
EXPERTS = [1, 2, 3, 4, 5, 8, 9, 12, 16, 17, 32, 33, 37, 60, 64, 65, 100, 127, 128, 129, 130, 256, 257, 300, 511, 512]


@pytest.mark.parametrize("E", EXPERTS)
def test_losses_experts(E):
    check(203, E, min(E, 3), mask=E % 2 == 0, inplace=E % 3 == 0)
    check(5, E, min(E, 8), mask=E % 2 == 1, sel=E % 3 != 0)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 64, 1000, 4099, 20000])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 6), (512, 8)])
def test_losses_tokens(T, E, k):
    check(T, E, k, mask=T % 2 == 1)


def test_z_loss_of_large_and_small_rows():
    """Squares of 2^24 and then of 1, which fp32 loses beside them. With one expert lse is the logit itself, its square is exact
    in 64 bits and so are the sums of a workgroup, each rounded once to fp32; with the loss's own rounding that is 2 u."""
    import torch
    T = 1 << 20
    L = torch.ones((T, 1), device="cuda")
    L[:T // 8] = 4096.0
    ws = F.get_router_workspace(T, 128, 1, 1)
    o = F.run_router_losses(ws, L, torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    z = (T // 8 * 2.0 ** 24 + T // 8 * 7) / T
    assert abs(float(o.losses[1]) - z) <= 2.0 * F32 * (1 + F32) * z
    assert float(o.losses[0]) == 1.0 and float(o.prob_sum) == T and int(o.n_tokens) == T


@pytest.mark.parametrize("E", [7, 8, 128, 512])
@pytest.mark.parametrize("dl", [(np.inf, 0.0), (0.0, np.nan)])
def test_losses_backward_of_overflowed_gradients(E, dl):
    """A token that the mask leaves out keeps the gradient through its combine weights, whatever d_losses holds."""
    import torch
    logits, ids, w, g, m = routing(50, E, 2)
    ws = F.get_router_workspace(50, 128, E, 2)
    L, I, W, G, M = f32(logits), i32(ids), f32(w), f32(g), torch.from_numpy(m).cuda()
    o = F.run_router_losses(ws, L, I, mask=M)
    for sel in ((None, None), (W, G)):
        a, b = (F.run_router_losses_backward(ws, L, I, o, f32(np.array(v)), *sel, mask=M) for v in (dl, (0.0, 0.0)))
        assert torch.equal(a[~M], b[~M])
        assert not torch.isfinite(a[M]).all(1).any()


@pytest.mark.parametrize("E,k", [(4, 4), (8, 8), (12, 12), (100, 100), (512, 65)])
def test_losses_many_picks(E, k):
    check(37, E, k)


def test_losses_of_large_logits():
    """Logits far apart, and all far from zero: exponentials are taken from the largest."""
    for shift, scale in ((1e4, 1.0), (-1e4, 1.0), (0.0, 60.0)):
        logits, ids, w, g, m = routing(50, 33, 4, scale=scale)
        logits = (logits + shift).astype(np.float32).astype(np.float64)
        check(50, 33, 4, data=(logits, ids, w, g, m))


def test_small_probabilities_keep_their_bits():
    """One token with logits of 0 and down to -80: every probability within 25 u of itself. Its exponential is within 4 u (2 u of
    the instruction, 1 of the correction's addition), the denominator within those 4 u and 14 additions, its reciprocal within 2
    and the product within 1. (The difference from the largest logit, 0, is exact.)"""
    import torch
    for E in (8, 100, 512):
        ws = F.get_router_workspace(1, 128, E, 1)
        l = np.concatenate([[0.0], -80 * np.random.default_rng(E).random(E - 1)]).astype(np.float32)
        o = F.run_router_losses(ws, f32(l[None]), torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        p = np.exp(l.astype(np.float64))
        p /= p.sum()
        assert_within(f64(o.prob_sum), p, 25 * F32 * p, "prob_sum")


def test_losses_masks_and_holes():
    import torch
    T, E, k = 40, 20, 3
    logits, ids, w, g, m = routing(T, E, k)
    data = lambda **kw: tuple({"logits": logits, "ids": ids, "w": w, "g": g, "m": m, **kw}.values())  # noqa: E731
    o, d = check(T, E, k, mask=True, data=data(m=np.zeros(T, bool)))     # no token is left
    assert (o.losses == 0).all() and int(o.n_tokens) == 0 and (o.prob_sum == 0).all()
    one = np.zeros(T, bool)
    one[17] = True
    check(T, E, k, mask=True, data=data(m=one))
    # what a left-out token holds does not matter to the others
    bad = logits.copy()
    bad[~m] = np.nan
    bad[np.nonzero(~m)[0][0]] = np.inf
    ws = F.get_router_workspace(T, 128, E, k)
    M, D = torch.from_numpy(m).cuda(), f32(np.array([1.0, 1.0]))
    a, b = (F.run_router_losses(ws, f32(v), i32(ids), mask=M) for v in (logits, bad))
    da, db = (F.run_router_losses_backward(ws, f32(v), i32(ids), a, D, mask=M) for v in (logits, bad))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(da, db) and (da[~M] == 0).all()
    # a mask of bytes other than 0 and 1
    c = F.run_router_losses(ws, f32(logits), i32(ids), mask=(M.to(torch.uint8) * 200))
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    # experts that cannot be chosen, and a token without any
    hole = logits.copy()
    hole[:, 3:7] = -np.inf
    hole[11] = -np.inf
    o, d = check(T, E, k, data=data(logits=hole), sel=False)
    assert (d[:, 3:7] == 0).all() and (d[11] == 0).all() and (o.prob_sum[3:7] == 0).all()
    # a NaN stays in its own row's gradient, and reaches the sums
    nan = logits.copy()
    nan[5, 2] = np.nan
    o = F.run_router_losses(ws, f32(nan), i32(ids))
    d = F.run_router_losses_backward(ws, f32(nan), i32(ids), a, D)
    torch.cuda.synchronize()
    assert torch.isnan(o.losses).all() and torch.isnan(d[5]).all() and torch.isfinite(d[:5]).all() and torch.isfinite(d[6:]).all()


def test_losses_ids_out_of_range_and_picked_twice():
    T, E, k = 30, 12, 4
    logits, ids, w, g, m = routing(T, E, k)
    ids[3] = [-1, 12, 1 << 30, -(1 << 31)]
    ids[4] = [5, 5, 5, 5]
    ids[5] = [7, 2, 7, 2]
    check(T, E, k, data=(logits, ids, w, g, m))


@pytest.mark.parametrize("E", [8, 60, 130])
def test_logits_backward_of_no_tokens_and_no_operands(E):
    """Without tokens every input may be NULL; d_w_router is set to zeros."""
    import ctypes
    import torch
    p = mok.make_problem(0, 1024, 128, E, 2)
    dwr = torch.full((E, 1024), 7.0, device="cuda")
    st = mok.lib().mok_router_logits_backward(ctypes.byref(p), None, None, None, None, None, dwr.data_ptr(), None, 0,
                                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == mok.MOK_OK and (dwr == 0).all()


def test_losses_of_no_tokens():
    import torch
    ws = F.get_router_workspace(0, 128, 9, 2)
    L, I = torch.empty((0, 9), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    o = F.run_router_losses(ws, L, I)
    d = F.run_router_losses_backward(ws, L, I, o, torch.ones(2, device="cuda"))
    dx, dwr = F.run_router_logits_backward(ws, torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),
                                           torch.ones((9, 128), device="cuda"), L)
    torch.cuda.synchronize()
    assert (o.losses == 0).all() and (o.counts == 0).all() and (o.prob_sum == 0).all() and int(o.n_tokens) == 0
    assert d.shape == (0, 9) and dx.shape == (0, 128) and (dwr == 0).all()


def test_losses_over_two_ranks():
    """Two halves of the tokens with their sums added up: the gradients of the whole batch, bit for bit."""
    import torch
    T, E, k = 600, 64, 4
    logits, ids, w, g, m = routing(T, E, k)
    ws, half = F.get_router_workspace(T, 128, E, k), F.get_router_workspace(T // 2, 128, E, k)
    L, I, M, D = f32(logits), i32(ids), torch.from_numpy(m).cuda(), f32(np.array([1.0, 0.5]))
    whole = F.run_router_losses(ws, L, I, mask=M)
    d = F.run_router_losses_backward(ws, L, I, whole, D, mask=M)
    a, b = (F.run_router_losses(half, L[s], I[s], mask=M[s]) for s in (slice(0, 300), slice(300, 600)))
    s = F.RouterLosses(a.losses, a.counts + b.counts, a.prob_sum + b.prob_sum, a.n_tokens + b.n_tokens)
    torch.cuda.synchronize()
    assert torch.equal(s.counts, whole.counts) and torch.equal(s.n_tokens, whole.n_tokens)
    for p in (slice(0, 300), slice(300, 600)):
        assert torch.equal(F.run_router_losses_backward(half, L[p], I[p], s, D, mask=M[p]), d[p])


@pytest.mark.parametrize("E", [1, 7, 37, 130, 511])
def test_slices_of_tokens(E):
    """Rows of the middle of a batch, at whatever place they start: the bits of the same rows in memory of their own."""
    import torch
    T, H, k, a, b = 90, 256, min(E, 3), 11, 74
    logits, ids, w, g, m = routing(T, E, k)
    L, I, W, G, M, D = f32(logits), i32(ids), f32(w), f32(g), torch.from_numpy(m).cuda(), f32(np.array([1.0, 0.5]))
    rng = np.random.default_rng(0)
    x, wr = bf(rng.normal(size=(b - a, H))), f32(rng.normal(size=(E, H)))
    ws = F.get_router_workspace(b - a, H, E, k)
    out = torch.full_like(L, 7.0)
    got = []
    for own in (False, True):
        v = [t[a:b].clone() if own else t[a:b] for t in (L, I, W, G, M)]
        o = F.run_router_losses(ws, v[0], v[1], mask=v[4])
        d = torch.empty_like(v[0]) if own else out[a:b]
        mok.router_losses_backward(ws.problem, v[0], v[1], o.counts, o.n_tokens, D, d, v[2], v[3], mask=v[4])
        got.append((*o, d, *F.run_router_logits_backward(ws, x, wr, d)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*got)) and (out[:a] == 7).all() and (out[b:] == 7).all()


def test_losses_leave_what_lies_behind():
    import torch
    T, E, k = 33, 21, 3
    logits, ids, *_ = routing(T, E, k)
    p = mok.make_problem(T, 128, 128, E, k)
    n = mok.router_workspace(p)
    ws = torch.full((n + 64,), 7, dtype=torch.uint8, device="cuda")
    c, q = torch.full((E + 16,), 7, dtype=torch.int32, device="cuda"), torch.full((E + 16,), 7.0, device="cuda")
    v, t = torch.full((8,), 7.0, device="cuda"), torch.full((8,), 7, dtype=torch.int32, device="cuda")
    d = torch.full((T * E + 16,), 7.0, device="cuda")
    mok.router_losses(p, f32(logits), i32(ids), v[:2], c[:E], q[:E], t[:1], ws[:n])
    mok.router_losses_backward(p, f32(logits), i32(ids), c[:E], t[:1], v[:2], d[:T * E].view(T, E))
    torch.cuda.synchronize()
    assert (ws[n:] == 7).all() and (c[E:] == 7).all() and (q[E:] == 7).all() and (v[2:] == 7).all() and (t[1:] == 7).all()
    assert (d[T * E:] == 7).all()


# ------------------------------------------------------------------ forward that keeps the logits
@pytest.mark.parametrize("T,H,E,k", [(1, 128, 8, 2), (100, 256, 37, 5), (300, 384, 130, 8), (16384, 128, 64, 4),
                                     (16500, 128, 100, 4)])
def test_forward_logits(T, H, E, k):
    import torch
    g = np.random.default_rng(T + E)
    x, wr = bf16_round(g.normal(size=(T, H))), (g.normal(size=(E, H)) * H ** -0.5).astype(np.float32)
    bias = g.normal(size=E).astype(np.float32)
    ws = F.get_router_workspace(T, H, E, k)
    ids, tw = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    mok.router_forward(ws.problem, bf(x), f32(wr), f32(bias), ids, tw)
    a, b, logits = F.run_router_forward(ws, bf(x), f32(wr), f32(bias))
    torch.cuda.synchronize()
    assert torch.equal(a, ids) and torch.equal(b, tw)
    w64 = wr.astype(np.float64)
    assert_within(f64(logits), x @ w64.T, dot(3 * H) * (np.abs(x) @ np.abs(w64).T) + 1e-37, "logits")


# ------------------------------------------------------------------ dense backward
def check_grad(T, H, E, residual=True, seed=0, inplace=False):
    import torch
    g = np.random.default_rng(seed + T + 13 * H + E)
    x = bf16_round(g.normal(size=(T, H)))
    wr = (g.normal(size=(E, H)) * H ** -0.5).astype(np.float32).astype(np.float64)
    dl = (g.normal(size=(T, E)) * np.exp(2 * g.normal(size=(T, 1)))).astype(np.float32).astype(np.float64)
    res = bf16_round(g.normal(size=(T, H))) if residual else None
    ws = F.get_router_workspace(T, H, E, 1)
    X, W, D = bf(x), f32(wr), f32(dl)
    R = None if res is None else bf(res)
    dx, dwr = F.run_router_logits_backward(ws, X, W, D, residual=R)
    buf = R.clone() if inplace else torch.full_like(X, 7.0)
    dx2, dwr2 = F.run_router_logits_backward(ws, X, W, D, residual=buf if inplace else R, dx=buf)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dwr, dwr2)
    rx, rw = lo.logits_backward(x, wr, dl, res)
    # dx: three products of each pair, each factor and their product short of 2^-16 of itself; the residual's addition
    a = np.abs(dl) @ np.abs(wr)
    e = (3 * 2.0 ** -16 + dot(3 * (E + 16))) * a + (0 if res is None else F32 * (np.abs(res) + np.abs(rx)))
    assert_within(f64(dx), rx, e + HALF * (np.abs(rx) + e) + 1e-37, "dx")
    # dWr: the products are exact; 3 T of them are added in fp32
    assert_within(f64(dwr), rw, dot(3 * T + 64) * (np.abs(dl).T @ np.abs(x)) + 1e-37, "dwr")
    # in the mean square the roundings of 3 T additions of terms of either sign are within u sqrt(3 T) of the root of
    # the terms' summed squares; twice that
    q = np.sqrt(((dl ** 2).T @ (x ** 2)).sum())
    assert np.linalg.norm(f64(dwr) - rw) <= 2 * F32 * np.sqrt(3 * T) * q


@pytest.mark.parametrize("E", [1, 2, 5, 15, 16, 17, 32, 33, 60, 64, 65, 100, 127, 128, 129, 200, 256, 257, 300, 512])
def test_grad_experts(E):
    check_grad(70, 384, E, residual=E % 2 == 0, inplace=E % 4 == 0)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 500, 4099])
@pytest.mark.parametrize("H,E", [(128, 8), (640, 60), (2048, 128), (256, 200)])
def test_grad_tokens(T, H, E):
    check_grad(T, H, E, residual=T % 2 == 1)


@pytest.mark.parametrize("E", [7, 32, 33, 64])
def test_grad_of_much_data(E):
    """More than 2^24 values of x: both results come from one kernel."""
    check_grad(4105, 4224, E, residual=E % 2 == 0, inplace=E == 64)


@pytest.mark.parametrize("T,H,E", [(700, 7168, 100), (300, 1024, 70), (580, 896, 40), (97, 1152, 9)])
def test_grad_of_odd_launches(T, H, E):
    """Numbers of workgroups that are no multiple of 8 (252, 20, 36, 10)."""
    check_grad(T, H, E)


def test_grad_of_the_wide_layer():
    check_grad(3000, 7168, 32)


def test_grad_products_are_exact():
    """One token of each column and one expert of each row different from zero: d_w_router is the value itself, all 24
    bits, and dx is Wr to 16 bits, rounded once."""
    import torch
    T, H, E = 96, 256, 130
    g = np.random.default_rng(0)
    dl = (g.normal(size=(T, E)) * np.exp2(g.integers(-60, 60, size=(T, E)))).astype(np.float32)
    tok = g.integers(0, T, size=H)
    x = np.zeros((T, H))
    x[tok, np.arange(H)] = np.where(g.random(H) < 0.5, 1.0, -2.0)
    ws = F.get_router_workspace(T, H, E, 1)
    wr = (g.normal(size=(E, H)) * np.exp2(g.integers(-60, 60, size=(E, H)))).astype(np.float32)
    _, dwr = F.run_router_logits_backward(ws, bf(x), f32(wr), f32(dl))
    np.testing.assert_array_equal(f64(dwr), dl[tok].T.astype(np.float64) * x[tok, np.arange(H)])
    one = np.zeros((T, E), np.float32)
    pick = g.integers(0, E, size=T)
    one[np.arange(T), pick] = 1.0
    dx, _ = F.run_router_logits_backward(ws, bf(x), f32(wr), f32(one))
    torch.cuda.synchronize()
    want = wr[pick].astype(np.float64)
    assert_within(f64(dx), want, (HALF + 2.0 ** -15) * np.abs(want), "dx")


def test_grad_leaves_what_lies_behind():
    import torch
    T, H, E = 33, 128, 37
    p = mok.make_problem(T, H, 128, E, 1)
    n = mok.router_workspace(p)
    ws = torch.full((n + 64,), 7, dtype=torch.uint8, device="cuda")
    dx, dw = torch.full((T * H + 64,), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((E * H + 64,), 7.0, device="cuda")
    g = np.random.default_rng(0)
    mok.router_logits_backward(p, bf(g.normal(size=(T, H))), f32(g.normal(size=(E, H))), f32(g.normal(size=(T, E))),
                               dx[:T * H].view(T, H), dw[:E * H].view(E, H), ws[:n])
    torch.cuda.synchronize()
    assert (ws[n:] == 7).all() and (dx[T * H:] == 7).all() and (dw[E * H:] == 7).all()


def test_grad_against_the_selected_ones():
    """With the selection's gradient alone, the dense backward gives what router_backward gives."""
    import torch
    T, H, E, k = 300, 256, 16, 3
    logits, ids, w, g, _ = routing(T, E, k)
    rng = np.random.default_rng(1)
    x, wr = bf(rng.normal(size=(T, H))), f32(rng.normal(size=(E, H)) * H ** -0.5)
    ws = F.get_router_workspace(T, H, E, k)
    lw = F.get_workspace(T, H, 128, E, k)
    I, W, G = i32(ids), f32(w), f32(g)
    F.run_schedule(lw, I)
    d_sel, dx, dwr = torch.empty_like(W), torch.empty_like(x), torch.empty_like(wr)
    mok.router_backward(lw.problem, lw.schedule, x, wr, I, W, G, d_sel, dx, dwr, lw.config)
    L = f32(logits)
    o = F.run_router_losses(ws, L, I)
    d = F.run_router_losses_backward(ws, L, I, o, torch.zeros(2, device="cuda"), topk_w=W, d_topk_w=G)
    dx2, dwr2 = F.run_router_logits_backward(ws, x, wr, d)
    torch.cuda.synchronize()
    sel = f64(d_sel)
    a = np.zeros((T, E))
    np.put_along_axis(a, ids.astype(np.int64), np.abs(sel), 1)
    W64, X64 = np.abs(f64(wr)), np.abs(f64(x))
    # two roundings of dx, and d_sel's own few u
    assert (np.abs(f64(dx2) - f64(dx)) <= (2.01 * HALF + 2.0 ** -13) * (a @ W64)).all()
    assert (np.abs(f64(dwr2) - f64(dwr)) <= (2 * dot(3 * T + 64) + 2.0 ** -18) * (a.T @ X64) + 1e-37).all()


# ------------------------------------------------------------------ the step around the layer
def step_inputs(T, H, E, I, k, seed=0):
    g = np.random.default_rng(seed)
    n = lambda *s, std=1.0: bf16_round(g.normal(size=s) * std)  # noqa: E731
    return {"x": n(T, H), "res": n(T, H), "wn": bf16_round(1 + 0.2 * g.normal(size=H)),
            "wr": (g.normal(size=(E, H)) * H ** -0.5).astype(np.float32).astype(np.float64), "wg": n(E, I, H, std=H ** -0.5),
            "wu": n(E, I, H, std=H ** -0.5), "wd": n(E, H, I, std=I ** -0.5), "dy": n(T, H), "d_sum": n(T, H)}


class Step:
    """norm -> router -> losses -> layer, and back."""

    def __init__(self, T, H, E, I, k):
        import torch
        self.nw = F.get_norm_workspace(T, H)
        self.rw = F.get_router_workspace(T, H, E, k)
        self.lw = F.get_workspace(T, H, I, E, k)
        self.d_losses = torch.tensor([0.02, 0.001], device="cuda")

    def __call__(self, s):
        n = F.run_norm_forward(self.nw, s["x"], s["wn"], s["res"])
        ids, tw, logits = F.run_router_forward(self.rw, n.y, s["wr"])
        aux = F.run_router_losses(self.rw, logits, ids)
        F.run_schedule(self.lw, ids)
        weights = (s["wg"], s["wu"], s["wd"])
        y = F.run_forward(self.lw, n.y, tw, weights)
        dx, dwg, dwu, dwd, dtw = F.run_backward(self.lw, n.y, tw, weights, s["dy"])
        d = F.run_router_losses_backward(self.rw, logits, ids, aux, self.d_losses, topk_w=tw, d_topk_w=dtw)
        dyn, dwr = F.run_router_logits_backward(self.rw, n.y, s["wr"], d, residual=dx, dx=dx)
        dz, dwn = F.run_norm_backward(self.nw, n.sum, n.rstd, s["wn"], dyn, d_sum=s["d_sum"])
        return {"sum": n.sum, "ids": ids, "y": y, "losses": aux.losses, "counts": aux.counts, "dz": dz, "dwn": dwn, "dwr": dwr,
                "dwg": dwg, "dwu": dwu, "dwd": dwd}


def on_gpu(s):
    return {k: f32(v) if k == "wr" else bf(v) for k, v in s.items()}


def test_step_around_the_layer():
    import torch
    T, H, E, I, k = 200, 256, 8, 128, 2
    s = step_inputs(T, H, E, I, k)
    o = Step(T, H, E, I, k)(on_gpu(s))
    torch.cuda.synchronize()
    ids = o["ids"].cpu().numpy()
    y, z, rstd = no.norm_forward(s["x"], s["wn"], s["res"])
    yb = bf16_round(y)
    logits = yb @ s["wr"].T
    sel = np.take_along_axis(logits, ids.astype(np.int64), 1)
    tw = np.exp(sel) / np.exp(sel).sum(1, keepdims=True)
    experts = list(zip(s["wg"], s["wu"], s["wd"]))
    ref = oracle.backward(yb, ids, tw, experts, s["dy"])
    aux = lo.losses(logits, ids)
    d = lo.losses_backward(aux, ids, (0.02, 0.001), tw, ref["dw"])
    dyn, dwr = lo.logits_backward(yb, s["wr"], d, ref["dx"])
    dz, dwn = no.norm_backward(dyn, z, rstd, s["wn"], s["d_sum"])
    want = {"sum": z, "y": ref["y"], "losses": aux["losses"], "counts": aux["counts"], "dz": dz, "dwn": dwn, "dwr": dwr,
            "dwg": ref["dWg"], "dwu": ref["dWu"], "dwd": ref["dWd"]}
    for name, v in want.items():
        got = f64(o[name])
        # every tensor passed on is rounded to bf16, 2^-8 at most each, in a chain of at most five (y, h, obuf, dx, dyn)
        # that add up as independent errors do: the layer's own bar of 1e-2
        assert np.linalg.norm(got - v) <= 1e-2 * np.linalg.norm(v), (name, np.linalg.norm(got - v) / np.linalg.norm(v))


def test_step_in_a_graph_and_on_two_streams():
    """The step captured and replayed on other inputs between eager steps, then two steps with their own buffers on two
    streams at once: the eager bits each time."""
    import torch
    dims = (200, 256, 8, 128, 2)
    sets = [on_gpu(step_inputs(*dims, seed=k)) for k in range(3)]
    eager = Step(*dims)
    refs = [eager(s) for s in sets]
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(a[k], b[k]) for k in b)  # noqa: E731
    static = {k: v.clone() for k, v in sets[0].items()}
    st = Step(*dims)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = st(static)
    for k in (1, 2, 0, 1):
        for n in static:
            static[n].copy_(sets[k][n])
        g.replay()
        torch.cuda.synchronize()
        assert same(out, refs[k]), k
        assert same(eager(sets[k]), refs[k])
        torch.cuda.synchronize()
    two = [Step(*dims) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append(two[i](sets[i + 1]))
        torch.cuda.synchronize()
        assert same(got[0], refs[1]) and same(got[1], refs[2])


def test_logits_past_32_bits():
    """More than 2^32 bytes of logits: the last rows are what they are alone."""
    import torch
    T, E, k = 2_200_000, 512, 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    ws = F.get_router_workspace(T, 128, E, k)
    tail, ids = routing(64, E, k)[:2]
    L = torch.zeros((T, E), device="cuda")
    L[-64:] = f32(tail)
    I = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    I[-64:] = i32(ids)
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-64:] = True
    D = torch.ones(2, device="cuda")
    o = F.run_router_losses(ws, L, I, mask=mask)
    d = F.run_router_losses_backward(ws, L, I, o, D, mask=mask)
    small = F.get_router_workspace(64, 128, E, k)
    o2 = F.run_router_losses(small, f32(tail), i32(ids))
    d2 = F.run_router_losses_backward(small, f32(tail), i32(ids), o2, D)
    torch.cuda.synchronize()
    assert torch.equal(o.counts, o2.counts) and int(o.n_tokens) == 64 and torch.equal(d[-64:], d2) and not d[:-64].any()
    np.testing.assert_allclose(f64(o.losses), f64(o2.losses), rtol=2e-6)
