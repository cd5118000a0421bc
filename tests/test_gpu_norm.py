"""The norm on the GPU, forward and backward, against its float64 reference, and
the reading back of MXFP8 rows.

Bounds, from the arithmetic (u = 2^-24). A row's sum runs over at most 32 terms
in a thread, 6 steps of a butterfly and 15 wavefronts, each an fp32 addition: it
is within 64 u of the sum of the terms' magnitudes (products included). With the
mean (2 u), the square root of a relative error (half of it) and a square root
and a division of at most 2 u each, rstd is within (64 + 2) / 2 + 4 < 40 u of
itself, and y before its rounding within 44 u. A rounding to bf16 adds at most
2^-8 of the value (finfo.eps / 2), or half the smallest subnormal."""
import numpy as np
import pytest

import mixture_experts_layer_30_amd as mok
import oracle.dense_oracle as do
import oracle.norm_oracle as no
from ffn_testlib import F32, HALF, assert_within
from mixture_experts_layer_30_amd import functional as F
from oracle import bf16_round, e4m3_decode, e4m3_encode
from test_gpu_mxfp4 import bf, f64, u8

pytestmark = pytest.mark.gpu

SUM, RSTD, Y = 64 * F32, 40 * F32, 44 * F32
TINY = 2.0 ** -134               # half the smallest bf16 subnormal


def rnd(v, e):
    return e + HALF * (np.abs(v) + e) + TINY


def make(T, H, seed=0, wf32=False, residual=True):
    g = np.random.default_rng(seed + 1000 * T + H)
    ch = np.exp(0.7 * g.normal(size=H))
    rows = lambda: bf16_round(g.normal(size=(T, H)) * ch * np.exp(g.normal(size=(T, 1))))  # noqa: E731
    w = 1 + 0.3 * g.normal(size=H)
    w = w.astype(np.float32).astype(np.float64) if wf32 else bf16_round(w)
    return rows(), rows() if residual else None, w


def dev_w(w, wf32):
    import torch
    if w is None:
        return None
    return torch.from_numpy(w.astype(np.float32)).cuda() if wf32 else bf(w)


def workspace(T, H, wf32=False, eps=1e-6, training=True):
    import torch
    return F.get_norm_workspace(T, H, eps=eps, weight_dtype=torch.float32 if wf32 else torch.bfloat16, training=training)


def check_mx(q, s, y, err):
    """Codes and scales are those of some rows within err of y, block by block."""
    q, s = q.cpu().numpy(), s.cpu().numpy().astype(int)
    rows, K = q.shape
    lo, hi = (np.sign(y) * np.maximum(np.abs(y) + k * err, 0) for k in (-1, 1))
    blk = lambda v: np.abs(v).reshape(rows, K // 32, 32).max(-1)  # noqa: E731
    byte = lambda a: np.where(a > 0, np.clip(np.frexp(a)[1] - 1 - 8 + 127, 0, 254), 0)  # noqa: E731
    assert ((byte(blk(lo)) <= s) & (s <= byte(blk(hi)))).all(), "scales"
    x = np.exp2(127.0 - s).repeat(32, -1)
    got = e4m3_decode(q)
    a, b = (e4m3_decode(e4m3_encode(v * x)) for v in (lo, hi))
    assert ((np.minimum(a, b) <= got) & (got <= np.maximum(a, b))).all(), "codes"


def check_forward(T, H, wf32=False, residual=True, out="bf16", weight=True, eps=1e-6, seed=0):
    import torch
    x, r, w = make(T, H, seed, wf32, residual)
    if not weight:
        w = None
    ws = workspace(T, H, wf32, eps)
    o = F.run_norm_forward(ws, bf(x), dev_w(w, wf32), None if r is None else bf(r), out=out)
    torch.cuda.synchronize()
    y, z, rstd = no.norm_forward(x, w, r, eps)
    np.testing.assert_array_equal(f64(o.sum), z)
    assert_within(f64(o.rstd), rstd, RSTD * rstd, "rstd")
    if out != "mxfp8":
        assert_within(f64(o.y), y, rnd(y, Y * np.abs(y)), "y")
    if out != "bf16":
        check_mx(o.q, o.scales, y, Y * np.abs(y))
    assert (o.y is None) == (out == "mxfp8") and (o.q is None) == (out == "bf16")
    return o


# every width at which another number of threads or chunks begins, and the column before it
WIDTHS = [8, 16, 24, 64, 72, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 7168, 8192, 8200,
          16384, 16392, 32768]


@pytest.mark.parametrize("H", WIDTHS)
def test_forward_widths(H):
    check_forward(5, H)
    check_forward(3, H, wf32=True, residual=False, weight=H % 16 == 0)


@pytest.mark.parametrize("H", [32, 64, 96, 128, 288, 512, 544, 1024, 1056, 2080, 4096, 7168, 8224, 16416, 32768])
@pytest.mark.parametrize("out", ["mxfp8", "both"])
def test_forward_mxfp8(H, out):
    check_forward(7, H, out=out, wf32=out == "both")


@pytest.mark.parametrize("T,H", [(2000, 96), (1500, 4096), (400, 7168), (60, 32768)])
def test_forward_sums_in_64_bits(T, H):
    """rstd is its value rounded once: the sum (of exact products), the mean and a Newton step from a value within 4 u, which
    leaves 1.5 (4 u)^2 < 2^-43, are in 64 bits. MXFP8 rows are those of values within one fp32 rounding of y."""
    import torch
    x, r, w = make(T, H, 11)
    o = F.run_norm_forward(workspace(T, H, eps=2.0 ** -20), bf(x), bf(w), bf(r), out="both")
    torch.cuda.synchronize()
    y, z, rstd = no.norm_forward(x, w, r, 2.0 ** -20)
    one = F32 * (1 + 2.0 ** -16)
    assert_within(f64(o.rstd), rstd, one * rstd, "rstd")
    check_mx(o.q, o.scales, y, one * np.abs(y))
    assert_within(f64(o.y), y, rnd(y, 4 * F32 * np.abs(y)), "y")


@pytest.mark.parametrize("T", [1, 2, 31, 33, 1000, 4099])
@pytest.mark.parametrize("H", [32, 640, 4096])
def test_forward_rows(T, H):
    check_forward(T, H, out="both", residual=T % 2 == 1)


@pytest.mark.parametrize("eps", [1.2e-38, 1e-12, 1e-5, 0.5, 1e30])
def test_forward_eps(eps):
    check_forward(3, 96, eps=eps)


def test_rows_do_not_depend_on_the_rows_beside_them():
    """A row alone gives the bits it gives among 3000 others (more than one pass of the grid for H = 8192), and a call on the
    stored stream the bits of the call that stored it."""
    import torch
    for H in (64, 1000, 2048, 8192):
        x, r, w = make(3000, H, 5)
        x, r, w = bf(x), bf(r), bf(w)
        o = F.run_norm_forward(workspace(3000, H), x, w, r)
        for t in (0, 1, 1777, 2999):
            p = F.run_norm_forward(workspace(1, H), x[t:t + 1], w, r[t:t + 1])
            assert torch.equal(p.y[0], o.y[t]) and torch.equal(p.rstd[0], o.rstd[t])
        again = F.run_norm_forward(workspace(3000, H), o.sum, w)
        assert torch.equal(again.y, o.y) and torch.equal(again.rstd, o.rstd) and again.sum is o.sum


def test_forward_strides_and_places():
    """Windows of wider matrices at every operand, outputs in place, and nothing written beside them."""
    import torch
    T, H = 37, 1000
    x, r, w = make(T, H, 3)
    wb = bf(w)
    ref = F.run_norm_forward(workspace(T, H), bf(x), wb, bf(r))
    X, R = (torch.full((T, P), 7.0, dtype=torch.bfloat16, device="cuda") for P in (1016, 2048))
    X[:, 8:1008], R[:, 1000:2000] = bf(x), bf(r)
    S, Yb = torch.full_like(R, 5.0), torch.full((T, 1200), 5.0, dtype=torch.bfloat16, device="cuda")
    o = F.run_norm_forward(workspace(T, H), X[:, 8:1008], wb, R[:, 1000:2000], y=Yb[:, 16:1016], sum_out=S[:, :1000])
    torch.cuda.synchronize()
    assert torch.equal(o.y, ref.y) and torch.equal(o.sum, ref.sum)
    assert (S[:, 1000:] == 5).all() and (Yb[:, :16] == 5).all() and (Yb[:, 1016:] == 5).all()
    # in place: the stream over the residual, y over x; and the other way round
    for swap in (False, True):
        a, b = bf(x), bf(r)
        o = F.run_norm_forward(workspace(T, H), a, wb, b, y=b if swap else a, sum_out=a if swap else b)
        torch.cuda.synchronize()
        assert torch.equal(o.y, ref.y) and torch.equal(o.sum, ref.sum)
    # sum beside x in one matrix of the pitch of both
    M = torch.zeros((T, 2000), dtype=torch.bfloat16, device="cuda")
    M[:, :1000] = bf(x)
    o = F.run_norm_forward(workspace(T, H), M[:, :1000], wb, y=M[:, 1000:])
    torch.cuda.synchronize()
    assert torch.equal(M[:, :1000], bf(x))
    assert torch.equal(o.y, F.run_norm_forward(workspace(T, H), bf(x), wb).y)


@pytest.mark.parametrize("H", [96, 1056, 8224])
def test_forward_mxfp8_strides_and_places(H):
    """MXFP8 rows from windows of wider matrices, the stream beside them, in place over the residual, and over x."""
    import torch
    T, P, Q = 19, H + 40, 2 * H + 8
    x, r, w = make(T, H, 6)
    wb, ws = bf(w), workspace(T, H)
    ref = F.run_norm_forward(ws, bf(x), wb, bf(r), out="both")
    same = lambda o: torch.equal(o.q, ref.q) and torch.equal(o.scales, ref.scales) and torch.equal(o.sum, ref.sum)  # noqa: E731
    for out in ("mxfp8", "both"):
        X, R = (torch.full((T, n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (P, Q))
        X[:, 8:8 + H], R[:, H:2 * H] = bf(x), bf(r)
        o = F.run_norm_forward(ws, X[:, 8:8 + H], wb, R[:, H:2 * H], out=out)
        assert same(o) and torch.equal(X[:, 8:8 + H], bf(x)) and torch.equal(R[:, H:2 * H], bf(r))
        assert out == "mxfp8" or torch.equal(o.y, ref.y)
        o = F.run_norm_forward(ws, X[:, 8:8 + H], wb, R[:, H:2 * H], out=out, sum_out=R[:, H:2 * H])
        assert same(o) and (R[:, :H] == 7).all() and (R[:, 2 * H:] == 7).all() and (X[:, :8] == 7).all()
        a, b = bf(x), bf(r)
        assert same(F.run_norm_forward(ws, a, wb, b, out=out, sum_out=a)) and torch.equal(a, ref.sum)
        if out == "both":
            a, b = bf(x), bf(r)
            o = F.run_norm_forward(ws, a, wb, b, out=out, y=a, sum_out=b)
            assert same(o) and torch.equal(a, ref.y)
    torch.cuda.synchronize()


def test_forward_more_rows_than_a_launch_holds():
    """A launch holds 2^22 rows of this width: workgroups that go round three times give every row the bits it has among fewer."""
    import torch
    T, H, N = (2 << 22) + 5, 544, 1 << 20
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = bf(make(1, H)[2])
    o = F.run_norm_forward(workspace(T, H), x, w, out="both")
    for a in range(0, T, N):
        n = min(N, T - a)
        p = F.run_norm_forward(workspace(n, H), x[a:a + n], w, out="both")
        assert torch.equal(p.y, o.y[a:a + n]) and torch.equal(p.rstd, o.rstd[a:a + n])
        assert torch.equal(p.q, o.q[a:a + n]) and torch.equal(p.scales, o.scales[a:a + n])


def test_forward_names_no_stream_that_y_lies_over():
    """Without a residual the stream is x itself, and where y was written over it there is none left to name."""
    import torch
    x, r, w = (bf(a) for a in make(6, 96, 1))
    ws = workspace(6, 96)
    a = x.clone()
    o = F.run_norm_forward(ws, a, w, y=a)
    assert o.sum is None and o.y is a
    with pytest.raises(ValueError):
        F.run_norm_backward(ws, o.sum, o.rstd, w, x)
    # the window of a wider matrix, and y elsewhere in it
    m = torch.zeros((6, 192), dtype=torch.bfloat16, device="cuda")
    m[:, :96] = x
    o = F.run_norm_forward(ws, m[:, :96], w, y=m[:, 96:])
    assert o.sum.data_ptr() == m.data_ptr() and torch.equal(o.sum, x)
    assert F.run_norm_forward(ws, m[:, :96], w, y=m[:, :96]).sum is None
    # with a residual the stream is what the call wrote
    a, ref = x.clone(), F.run_norm_forward(ws, x, w, r)
    o = F.run_norm_forward(ws, a, w, r, y=a)
    assert torch.equal(o.sum, ref.sum) and torch.equal(a, ref.y)
    e = torch.empty((0, 96), dtype=torch.bfloat16, device="cuda")
    assert F.run_norm_forward(workspace(0, 96), e, w, y=torch.empty_like(e)).sum is e


def test_forward_leaves_what_lies_behind():
    import torch
    T, H = 5, 96
    x, r, w = make(T, H)
    y = torch.full((T * H + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    q, s = (torch.full((n + 64,), 7, dtype=torch.uint8, device="cuda") for n in (T * H, T * H // 32))
    rstd = torch.full((T + 64,), 3.0, device="cuda")
    p = mok.make_norm_problem(T, H)
    mok.norm_forward(p, bf(x), bf(w), y=y[:T * H].view(T, H), rstd=rstd[:T], q=q[:T * H].view(T, H),
                     scales=s[:T * H // 32].view(T, H // 32))
    torch.cuda.synchronize()
    assert (y[T * H:] == 3).all() and (q[T * H:] == 7).all() and (s[T * H // 32:] == 7).all() and (rstd[T:] == 3).all()


def test_forward_zeros_infinities_and_nans():
    import torch
    T, H = 6, 96
    x, _, w = make(T, H)
    x[0] = 0
    x[1, 5] = np.inf
    x[2, 40] = np.nan
    x[3] = 1e-30                                  # squares below fp32: eps alone is left
    x[4] = 3e38                                   # their sum passes fp32
    o = F.run_norm_forward(workspace(T, H), bf(x), bf(w), out="both")
    v = f64(F.mxfp8_dequantize(o.q, o.scales))
    torch.cuda.synchronize()
    y = f64(o.y)
    assert (y[0] == 0).all() and (v[0] == 0).all()
    assert np.isnan(y[1, 5]) and (np.delete(y[1], 5) == 0).all()
    assert np.isnan(v[1, :32]).all() and (v[1, 32:] == 0).all()
    assert np.isnan(y[2]).all() and np.isnan(v[2]).all()
    assert (y[4] == 0).all()
    ref = no.norm_forward(f64(bf(x))[[3, 5]], w)[0]
    assert_within(y[[3, 5]], ref, rnd(ref, Y * np.abs(ref)), "rows beside them")


def test_empty():
    import torch
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    ws = workspace(0, 64, True)
    o = F.run_norm_forward(ws, x, w, out="both")
    dx, dw = F.run_norm_backward(ws, o.sum, o.rstd, w, x)
    torch.cuda.synchronize()
    assert o.y.shape == (0, 64) and o.q.shape == (0, 64) and dx.shape == (0, 64) and (dw == 0).all()
    assert F.mxfp8_dequantize(o.q, o.scales).shape == (0, 64)


# ------------------------------------------------------------------ backward
def check_backward(T, H, wf32=False, d_sum=True, weight=True, seed=0):
    import torch
    z, ds, w = make(T, H, seed, wf32)
    g = np.random.default_rng(seed + 1)
    dy = bf16_round(g.normal(size=(T, H)))
    if not weight:
        w = None
    if not d_sum:
        ds = None
    ws = workspace(T, H, wf32)
    rs = F.run_norm_forward(ws, bf(z), dev_w(w, wf32)).rstd
    dx, dw = F.run_norm_backward(ws, bf(z), rs, dev_w(w, wf32), bf(dy), d_sum=None if ds is None else bf(ds))
    dx2, dw2 = F.run_norm_backward(ws, bf(z), rs, dev_w(w, wf32), bf(dy), d_sum=None if ds is None else bf(ds))
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and (dw is None or torch.equal(dw, dw2))
    r = f64(rs)[:, None]
    rx, rw = no.norm_backward(dy, z, r[:, 0], w, ds)
    # s = mean(g xh): the row's sum, its products and the mean within 64 + 4 u of the terms' magnitudes; then
    # rstd (g - xh s) + d_sum: at most 6 roundings of the terms
    xh, gw = np.abs(z * r), np.abs(dy if w is None else dy * w)
    es = (SUM + 4 * F32) * (gw * xh).mean(1, keepdims=True)
    s = np.abs((dy * (1 if w is None else w) * z * r).mean(1, keepdims=True))
    e = r * (xh * es + 6 * F32 * (gw + xh * (s + es))) + (0 if ds is None else F32 * (np.abs(ds) + np.abs(rx)))
    assert_within(f64(dx), rx, rnd(rx, e), "dx")
    if w is None:
        assert dw is None
        return
    # dw: T terms of two roundings each, added in some fixed order
    e = (T + 8) * F32 * np.abs(dy * z * r).sum(0) + 1e-38
    assert dw.dtype == (torch.float32 if wf32 else torch.bfloat16)
    assert_within(f64(dw), rw, e if wf32 else rnd(rw, e), "dw")


@pytest.mark.parametrize("H", WIDTHS)
def test_backward_widths(H):
    check_backward(5, H)
    check_backward(3, H, wf32=True, d_sum=False)


@pytest.mark.parametrize("T", [1, 2, 31, 257, 1000, 4099])
@pytest.mark.parametrize("H", [40, 640, 4096])
def test_backward_rows(T, H):
    check_backward(T, H, wf32=T % 2 == 0, d_sum=T % 2 == 1)


def test_backward_without_a_weight():
    check_backward(33, 1000, weight=False)


def test_backward_against_differences_of_the_forward():
    """Along random directions, on values that bf16 holds with room: the forward's own fp32 rstd and y are too coarse for
    differences, so the directions are steps of the stored stream and the reference is the 64-bit forward."""
    import torch
    T, H = 4, 64
    g = np.random.default_rng(9)
    z = bf16_round(g.normal(size=(T, H)))
    w, dy = bf16_round(1 + 0.3 * g.normal(size=H)), bf16_round(g.normal(size=(T, H)))
    ws = workspace(T, H)
    o = F.run_norm_forward(ws, bf(z), bf(w))
    dx, dw = F.run_norm_backward(ws, bf(z), o.rstd, bf(w), bf(dy))
    torch.cuda.synchronize()
    f = lambda zz, ww: (dy * no.norm_forward(zz, ww)[0]).sum()  # noqa: E731
    for i in range(8):
        d, dwv, h = g.normal(size=(T, H)), g.normal(size=H), 1e-5
        num = (f(z + h * d, w) - f(z - h * d, w)) / (2 * h)
        # the gradient's roundings to bf16, and the curvature of the difference (h^2)
        assert abs(num - (f64(dx) * d).sum()) <= HALF * 1.01 * (np.abs(f64(dx)) * np.abs(d)).sum() + 1e-6
        num = (f(z, w + h * dwv) - f(z, w - h * dwv)) / (2 * h)
        assert abs(num - (f64(dw) * dwv).sum()) <= HALF * 1.01 * (np.abs(f64(dw)) * np.abs(dwv)).sum() + 1e-6


@pytest.mark.parametrize("T,H", [(70, 16640), (300, 32768)])
def test_backward_of_wide_rows_in_strides_and_places(T, H):
    """Beyond 16384 columns the sums of dw lie in LDS."""
    import torch
    z, ds, w = make(T, H, 1)
    dy = bf16_round(np.random.default_rng(2).normal(size=(T, H)))
    ws, wb = workspace(T, H), bf(w)
    rs = F.run_norm_forward(ws, bf(z), wb).rstd
    ref = F.run_norm_backward(ws, bf(z), rs, wb, bf(dy), d_sum=bf(ds))
    Z, D, G = (torch.full((T, H + n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (24, 40, 8))
    Z[:, 16:16 + H], D[:, 8:8 + H], G[:, :H] = bf(z), bf(ds), bf(dy)
    O = torch.full_like(D, 5.0)
    for dx in (O[:, 32:32 + H], D[:, 8:8 + H]):
        got = F.run_norm_backward(ws, Z[:, 16:16 + H], rs, wb, G[:, :H], d_sum=D[:, 8:8 + H], dx=dx)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert (O[:, :32] == 5).all() and (O[:, 32 + H:] == 5).all() and (D[:, :8] == 7).all() and (D[:, 8 + H:] == 7).all()
    a = bf(dy)
    got = F.run_norm_backward(ws, bf(z), rs, wb, a, d_sum=bf(ds), dx=a)
    torch.cuda.synchronize()
    assert torch.equal(a, ref[0]) and torch.equal(got[1], ref[1])


def test_backward_strides_and_places():
    import torch
    T, H = 300, 520
    z, ds, w = make(T, H, 1)
    dy = bf16_round(np.random.default_rng(2).normal(size=(T, H)))
    ws = workspace(T, H)
    wb = bf(w)
    rs = F.run_norm_forward(ws, bf(z), wb).rstd
    ref = F.run_norm_backward(ws, bf(z), rs, wb, bf(dy), d_sum=bf(ds))
    Z, D, G = (torch.full((T, P), 7.0, dtype=torch.bfloat16, device="cuda") for P in (1040, 536, 528))
    Z[:, 512:1032], D[:, 8:528], G[:, :520] = bf(z), bf(ds), bf(dy)
    O = torch.full_like(D, 5.0)
    dx, dw = F.run_norm_backward(ws, Z[:, 512:1032], rs, wb, G[:, :520], d_sum=D[:, 8:528], dx=O[:, 16:])
    torch.cuda.synchronize()
    assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1]) and (O[:, :16] == 5).all()
    dx, dw = F.run_norm_backward(ws, Z[:, 512:1032], rs, wb, G[:, :520], d_sum=D[:, 8:528], dx=D[:, 8:528])
    torch.cuda.synchronize()
    assert torch.equal(D[:, 8:528], ref[0]) and torch.equal(dw, ref[1]) and (D[:, :8] == 7).all() and (D[:, 528:] == 7).all()
    a = bf(dy)
    dx, _ = F.run_norm_backward(ws, bf(z), rs, wb, a, d_sum=bf(ds), dx=a)
    torch.cuda.synchronize()
    assert torch.equal(a, ref[0])


def test_offsets_past_32_bits():
    import torch
    T, H, P = 3, 64, (1 << 31) - 64
    x, r, w = make(T, H, 4)
    big = torch.empty((T - 1) * P + H, dtype=torch.bfloat16, device="cuda").as_strided((T, H), (P, 1))
    big.copy_(bf(x))
    ws = workspace(T, H)
    o, ref = F.run_norm_forward(ws, big, bf(w), y=big), F.run_norm_forward(ws, bf(x), bf(w))
    torch.cuda.synchronize()
    assert torch.equal(big, ref.y) and torch.equal(o.rstd, ref.rstd)
    big.copy_(bf(x))
    dy = bf(r)
    d, dref = F.run_norm_backward(ws, big, o.rstd, bf(w), dy), F.run_norm_backward(ws, bf(x), o.rstd, bf(w), dy)
    torch.cuda.synchronize()
    assert torch.equal(d[0], dref[0]) and torch.equal(d[1], dref[1])


def test_other_stream_and_graph():
    """On a side stream, and captured with both directions and replayed on new inputs between eager calls of its own shapes."""
    import torch
    T, H = 700, 1024
    ws = workspace(T, H)
    wb = bf(make(T, H)[2])
    sets = [[bf(a) for a in (*make(T, H, k)[:2], bf16_round(np.random.default_rng(k).normal(size=(T, H))))] for k in range(3)]

    def step(x, r, dy):
        o = F.run_norm_forward(ws, x, wb, r, out="both")
        return (*o, *F.run_norm_backward(ws, o.sum, o.rstd, wb, dy, d_sum=r))

    refs = [step(*s) for s in sets]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = step(*sets[1])
    st.synchronize()
    for a, b in zip(got, refs[1]):
        assert torch.equal(a, b)
    static = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(*static)
    for k in (1, 2, 0, 1):
        for a, b in zip(static, sets[k]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, refs[k]):
            assert torch.equal(a, b), k
        for a, b in zip(step(*sets[k]), refs[k]):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


# ------------------------------------------------------------------ reading MXFP8 rows back
def test_dequantize_every_code_and_scale():
    import torch
    q = np.tile(np.arange(256, dtype=np.uint8).reshape(8, 32), (256, 1))
    s = np.arange(256, dtype=np.uint8).repeat(8).reshape(-1, 1)
    got = f64(F.mxfp8_dequantize(u8(q), u8(s)))
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        want = bf16_round(do.mxfp8_values(q, s))
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("rows,K", [(1, 32), (37, 96), (129, 1056), (1000, 7168)])
def test_dequantize_returns_the_quantizers_values(rows, K):
    import torch
    g = np.random.default_rng(rows)
    v = bf16_round(g.normal(size=(rows, K)) * np.exp2(g.integers(-130, 100, size=(rows, K // 32)).repeat(32, 1)))
    q = torch.empty((rows, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
    mok.mxfp8_quantize(bf(v), q, s)
    out = torch.full((rows * K + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    mok.mxfp8_dequantize(q, s, out[:rows * K].view(rows, K))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(out[:rows * K]).reshape(rows, K), do.mxfp8_round(v))
    assert (out[rows * K:] == 3).all()


def test_dequantize_past_32_bits():
    """More than 2^32 codes, 2^33 bytes of values: the first and last rows are what they are alone."""
    import torch
    rows, K = (1 << 20) + 3, 4128
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB")
    g = torch.Generator("cuda").manual_seed(2)
    q = torch.zeros((rows, K), dtype=torch.uint8, device="cuda")
    s = torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")
    for a in (slice(0, 64), slice(rows - 64, rows)):
        q[a] = torch.randint(0, 127, (64, K), generator=g, device="cuda", dtype=torch.uint8)
        s[a] = torch.randint(100, 150, (64, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    v = F.mxfp8_dequantize(q, s)
    for a in (slice(0, 64), slice(rows - 64, rows)):
        assert torch.equal(v[a], F.mxfp8_dequantize(q[a], s[a])) and v[a].any()
    assert not v[64:rows - 64].any()


def test_norm_into_an_mxfp4_product():
    """The MXFP8 rows are what the product with an MXFP4 matrix takes: the same bits as from the read-back values quantized again
    (a second quantization of MXFP8 values changes nothing)."""
    import torch
    T, H, N = 50, 512, 384
    x, r, w = make(T, H, 8)
    b, sb = F.mxfp4_quantize(bf(np.random.default_rng(0).normal(size=(N, H)) * H ** -0.5))
    o = F.run_norm_forward(workspace(T, H, training=False), bf(x), bf(w), bf(r), out="mxfp8")
    assert o.rstd is None
    mm = F.get_mx_matmul_workspace(T, N, H, mok.MOK_MXFP8)
    d = F.run_mx_matmul(mm, o.q, o.scales, b, sb)
    v = F.mxfp8_dequantize(o.q, o.scales)
    q, s = torch.empty_like(o.q), torch.empty_like(o.scales)
    mok.mxfp8_quantize(v, q, s)
    d2 = F.run_mx_matmul(mm, q, s, b, sb)
    torch.cuda.synchronize()
    assert torch.equal(d, d2)
