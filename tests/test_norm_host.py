"""Host-side tests of the norm's calls and the MXFP8 read-back (no GPU needed):
sizes, and every argument error found before anything touches a device."""
import ctypes

import pytest
import torch

import mixture_experts_layer_30_amd as mok
from mixture_experts_layer_30_amd import functional as F

INV, UNS, SMALL = mok.MOK_ERR_INVALID_ARG, mok.MOK_ERR_UNSUPPORTED, mok.MOK_ERR_BUFFER_TOO_SMALL
# what a call answers here once its arguments pass: there is no device
GONE = mok.MOK_ERR_DEVICE
V = ctypes.c_void_p

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="passes pointers to no memory: not where a GPU is")


def fwd(T=8, H=64, x=1 << 32, res=None, w=2 << 32, y=3 << 32, total=None, rstd=4 << 32, q=None, s=None, **kw):
    p = mok.make_norm_problem(T, H, **kw)
    return mok.lib().mok_norm_forward(ctypes.byref(p), *(V(a) for a in (x, res, w, y, total, rstd, q, s)), None)


def bwd(T=8, H=64, dy=1 << 32, z=2 << 32, ld_z=0, rstd=3 << 32, w=4 << 32, d_sum=None, dx=5 << 32, dw=6 << 32,
        ws=7 << 32, n=1 << 30, **kw):
    p = mok.make_norm_problem(T, H, **kw)
    return mok.lib().mok_norm_backward(ctypes.byref(p), V(dy), V(z), ld_z, V(rstd), V(w), V(d_sum), V(dx), V(dw), V(ws),
                                       n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(H=-8), INV), (dict(H=12), UNS), (dict(H=32776), UNS),
    (dict(T=(1 << 30) + 1), UNS), (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(eps=1e-40), INV), (dict(weight_f32=2), INV), (dict(ld_x=56), INV),
    (dict(ld_s=68), INV), (dict(ld_y=60), INV), (dict(ld_x=(1 << 31) + 8), UNS), (dict(ld_s=(1 << 31) + 8), UNS),
    (dict(ld_y=(1 << 31) + 8), UNS),
])
def test_problems_refused(kw, status):
    p = dict(T=8, H=64)
    p.update(kw)
    with pytest.raises(mok.MokError) as e:
        mok.norm_workspace(mok.make_norm_problem(**p))
    assert e.value.status == status
    assert fwd(**p) == status and bwd(**p) == status


def test_workspace():
    for T in (0, 1, 2, 777, 16384, 1 << 30):
        for H in (8, 64, 1000, 7168, 32768):
            assert mok.norm_workspace(mok.make_norm_problem(T, H)) <= 1024 * H * 4
    assert mok.norm_workspace(mok.make_norm_problem(1, 7168)) == 0
    assert mok.norm_workspace(mok.make_norm_problem(16384, 7168)) > 0


def test_forward_refuses():
    assert fwd() == GONE and fwd(w=None) == GONE and fwd(rstd=None) == GONE
    assert fwd(res=8 << 32, total=9 << 32) == GONE and fwd(y=None, q=8 << 32, s=9 << 32) == GONE
    assert fwd(x=None) == INV and fwd(y=None) == INV
    assert fwd(res=8 << 32) == INV and fwd(total=8 << 32) == INV and fwd(q=8 << 32) == INV and fwd(s=8 << 32) == INV
    assert fwd(H=72, q=8 << 32, s=9 << 32) == UNS and fwd(H=72) == GONE
    for k in ("x", "w", "y", "q"):
        kw = {k: (10 << 32) + 8}
        if k == "q":
            kw["s"] = 9 << 32
        assert fwd(**kw) == INV, k
    assert fwd(res=(8 << 32) + 8, total=9 << 32) == INV and fwd(res=8 << 32, total=(9 << 32) + 8) == INV
    assert fwd(rstd=(4 << 32) + 2) == INV
    assert fwd(T=0, x=None, y=None, rstd=None) == GONE


def test_forward_overlaps():
    x, r, t, y = 1 << 32, 8 << 32, 9 << 32, 3 << 32
    full = dict(res=r, total=t, q=11 << 32, s=12 << 32)
    n = 8 * 64
    assert fwd(**full) == GONE
    # exactly over x or the residual: allowed
    for kw in (dict(total=r), dict(total=x), dict(y=x), dict(y=r), dict(total=r, y=x), dict(total=x, y=r)):
        assert fwd(**{**full, **kw}) == GONE, kw
    assert fwd(**{**full, "total": r, "y": r}) == INV and fwd(**{**full, "y": t}) == INV
    for off in (16, -16, 2 * n - 16, -(2 * n - 16)):
        for a in (x, r):
            assert fwd(**{**full, "total": a + off}) == INV and fwd(**{**full, "y": a + off}) == INV
        assert fwd(**{**full, "y": t + off}) == INV
    for off in (2 * n, -2 * n):
        assert fwd(**{**full, "total": x + off}) == GONE and fwd(**{**full, "y": r + off}) == GONE
    # over x with another pitch
    assert fwd(y=x, ld_y=72) == INV and fwd(y=x, ld_y=72, ld_x=72) == GONE
    # side by side in one matrix of pitch 160
    assert [fwd(y=x + 2 * c, ld_y=160, ld_x=160) for c in (56, 64, 96, 104)] == [INV, GONE, GONE, INV]
    for k, at in (("rstd", x), ("rstd", r + 2 * n - 4), ("rstd", y), ("rstd", t), ("q", x), ("q", y), ("q", t), ("q", r),
                  ("s", x), ("s", y), ("s", 11 << 32), ("s", (11 << 32) + n - 1), ("q", (4 << 32) + 16), ("w", y),
                  ("w", t), ("w", 4 << 32), ("w", 11 << 32), ("w", 12 << 32)):
        assert fwd(**{**full, k: at}) == INV, (k, at)
    assert fwd(w=y, weight_f32=1) == INV and fwd(w=y - 4 * 64, weight_f32=1) == GONE
    assert fwd(w=y - 4 * 64 + 16, weight_f32=1) == INV


def test_backward_refuses():
    assert bwd() == GONE and bwd(d_sum=8 << 32) == GONE and bwd(w=None, dw=None) == GONE and bwd(dw=None) == GONE
    for k in ("dy", "z", "rstd", "dx"):
        assert bwd(**{k: None}) == INV, k
    assert bwd(w=None) == INV
    for k in ("dy", "z", "w", "dx", "dw", "d_sum", "ws"):
        assert bwd(**{k: (10 << 32) + 8}) == INV, k
    assert bwd(rstd=(3 << 32) + 2) == INV and bwd(ld_z=56) == INV and bwd(ld_z=68) == INV
    assert bwd(ld_z=(1 << 31) + 8) == UNS
    need = mok.norm_workspace(mok.make_norm_problem(16384, 7168))
    assert bwd(T=16384, H=7168, n=need) == GONE and bwd(T=16384, H=7168, n=need - 1) == SMALL
    assert bwd(T=16384, H=7168, ws=None) == SMALL and bwd(T=16384, H=7168, ws=None, dw=None) == GONE
    assert bwd(T=0, dy=None, z=None, rstd=None, dx=None) == GONE


def test_backward_overlaps():
    T, H, n = 16384, 64, 16384 * 64
    a = dict(T=T, H=H, d_sum=8 << 32, n=mok.norm_workspace(mok.make_norm_problem(T, H)))
    assert bwd(**a) == GONE
    assert bwd(**{**a, "dx": 8 << 32}) == GONE and bwd(**{**a, "dx": 1 << 32}) == GONE
    assert bwd(**{**a, "dx": 2 << 32}) == INV                     # over z
    for base in (1, 2, 8):
        for off in (16, -16, 2 * n - 16, -(2 * n - 16)):
            assert bwd(**{**a, "dx": (base << 32) + off}) == INV, (base, off)
        for off in (2 * n, -2 * n):
            assert bwd(**{**a, "dx": (base << 32) + off}) == GONE, (base, off)
    assert bwd(**{**a, "dx": 1 << 32, "ld_y": 72}) == INV and bwd(**{**a, "dx": 1 << 32, "ld_y": 72, "ld_s": 72}) == GONE
    for k in ("dw", "ws"):
        for at in (1, 2, 3, 4, 5, 8):
            assert bwd(**{**a, k: at << 32}) == INV, (k, at)
    assert bwd(**{**a, "ws": 6 << 32}) == INV and bwd(**{**a, "dx": 3 << 32}) == INV and bwd(**{**a, "dx": 4 << 32}) == INV


def test_mxfp8_dequantize_refuses():
    f = lambda q=1 << 32, s=2 << 32, r=4, K=64, d=3 << 32: mok.lib().mok_mxfp8_dequantize(V(q), V(s), r, K, V(d), None)  # noqa: E731
    assert f() == GONE and f(r=0, q=None, s=None, d=None) == GONE
    assert f(r=-1) == INV and f(K=0) == INV and f(K=48) == INV and f(q=None) == INV and f(s=None) == INV
    assert f(d=None) == INV and f(q=(1 << 32) + 8) == INV and f(d=(3 << 32) + 8) == INV
    assert f(K=1 << 39) == UNS and f(r=(1 << 33) + 1, K=32) == UNS
    assert f(d=1 << 32) == INV and f(d=(1 << 32) - 2 * 256 + 16) == INV and f(d=(1 << 32) - 2 * 256) == GONE
    assert f(s=(3 << 32) + 511) == INV and f(s=(3 << 32) + 512) == GONE


def test_python_refuses_other_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = F.get_norm_workspace(4, 64, device="cpu")
    with pytest.raises(mok.MokError):                            # not on a GPU
        F.run_norm_forward(w, x, torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        F.run_norm_forward(w, x, None, out="fp8")
    with pytest.raises(ValueError):
        F.run_norm_forward(w, x, None, out="mxfp8", y=x)
    with pytest.raises(ValueError):
        F.get_norm_workspace(4, 64, weight_dtype=torch.float16)
    with pytest.raises(ValueError):
        F.run_norm_backward(F.get_norm_workspace(4, 64, device="cpu", training=False), x, x, None, x)


def test_python_refuses_a_stream_that_was_overwritten():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.run_norm_backward(F.get_norm_workspace(4, 64, device="cpu"), None, torch.zeros(4), None, x)
