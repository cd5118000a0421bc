"""Host-side tests of the router's losses and its dense backward (no GPU needed):
sizes, and every argument error found before anything touches a device."""
import ctypes

import pytest
import torch

import mixture_experts_layer_30_amd as mok
from mixture_experts_layer_30_amd import functional as F

INV, UNS, SMALL, GONE = mok.MOK_ERR_INVALID_ARG, mok.MOK_ERR_UNSUPPORTED, mok.MOK_ERR_BUFFER_TOO_SMALL, mok.MOK_ERR_DEVICE
V = ctypes.c_void_p
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="passes pointers to no memory: not where a GPU is")

T, H, E, K = 64, 256, 40, 4


def P(**kw):
    a = dict(T=T, H=H, I=128, E=E, topk=K)
    a.update(kw)
    return mok.make_problem(**a)


def call(fn, at, tail=(), p=None, **kw):
    a = dict(at)
    a.update(kw)
    return fn(ctypes.byref(p or P()), *(V(a[k]) for k in at), *tail, None)


def places(*names):
    return {n: (i + 1) << 32 for i, n in enumerate(names)}


FWD = places("x", "wr", "bias", "ids", "w", "logits")
LOSS = places("logits", "ids", "mask", "losses", "counts", "prob", "n", "ws")
BACK = places("logits", "ids", "mask", "counts", "n", "dl", "w", "g", "out")
GRAD = places("x", "wr", "dl", "res", "dx", "dwr", "ws")


def fwd(p=None, **kw):
    return call(mok.lib().mok_router_forward_logits, FWD, p=p, **kw)


def loss(p=None, size=1 << 30, **kw):
    return call(mok.lib().mok_router_losses, LOSS, (size,), p=p, **kw)


def back(p=None, **kw):
    return call(mok.lib().mok_router_losses_backward, BACK, p=p, **kw)


def grad(p=None, size=1 << 30, **kw):
    return call(mok.lib().mok_router_logits_backward, GRAD, (size,), p=p, **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(E=0), INV), (dict(topk=0), INV), (dict(topk=41), INV),
    (dict(dtype=mok.MOK_MXFP4), INV), (dict(E=513), UNS), (dict(H=200), UNS), (dict(H=(1 << 20) + 128), UNS),
    (dict(T=(1 << 30) + 1, topk=1), UNS),
])
def test_problems_refused(kw, status):
    with pytest.raises(mok.MokError) as e:
        mok.router_workspace(P(**kw))
    assert e.value.status == status
    assert all(f(p=P(**kw)) == status for f in (fwd, loss, back, grad))


def test_workspace():
    for t in (0, 1, 33, 1037, 16384, 1 << 30):
        for h in (128, 7168):
            for e in (1, 37, 128, 512):
                n = mok.router_workspace(P(T=t, H=h, E=e, topk=1))
                # at most 512 partial sums of the losses, and 512 of 128 x 128 of d_w_router
                assert n <= max(512 * (2 * e + 2) * 4 + 4, 512 * 128 * 128 * 4 * ((e + 127) // 128))


def test_calls_refuse():
    assert fwd() == loss() == back() == grad() == GONE
    assert fwd(bias=None) == loss(mask=None) == back(mask=None) == back(w=None, g=None) == grad(res=None) == GONE
    for f, at, free in ((fwd, FWD, ("bias",)), (loss, LOSS, ("mask", "ws")), (back, BACK, ("mask",)), (grad, GRAD, ("res", "ws"))):
        for k in at:
            if k not in free:
                assert f(**{k: None}) == INV, (f.__name__, k)
    for f, at in ((loss, LOSS), (fwd, FWD), (back, BACK), (grad, GRAD)):
        for k in at:
            if k == "mask":
                continue
            assert f(**{k: at[k] + 2}) == INV, (f.__name__, k)
            wide = k in {"loss": ("logits", "ws"), "fwd": ("x", "wr"), "back": ("logits", "out"), "grad": GRAD}[f.__name__]
            assert (f(**{k: at[k] + 8}) == INV) == wide, (f.__name__, k)
    assert loss(mask=LOSS["mask"] + 1) == GONE
    assert fwd(p=P(E=128, topk=65)) == UNS and loss(p=P(E=128, topk=65)) == GONE and back(p=P(E=128, topk=65)) == GONE
    big = P(T=16384)
    a, b = (mok.router_workspace(P(T=16384, H=h)) for h in (128, 7168))
    assert loss(p=big, size=a) == GONE and loss(p=big, ws=None) == SMALL and loss(p=big, size=1000) == SMALL
    assert grad(p=P(T=16384, H=7168), size=b) == GONE and grad(p=P(T=16384, H=7168), size=b - 4) == SMALL
    assert grad(p=P(T=16384, H=7168), ws=None) == SMALL
    none = P(T=0)
    assert fwd(p=none, **dict.fromkeys(FWD)) == GONE
    assert loss(p=none, logits=None, ids=None, mask=None, ws=None) == GONE and loss(p=none, counts=None) == INV
    assert back(p=none, logits=None, ids=None, out=None, w=None, g=None) == GONE
    assert grad(p=none, x=None, wr=None, dl=None, res=None, dx=None, ws=None) == GONE and grad(p=none, dwr=None) == INV


def test_overlaps():
    sizes = {"fwd": dict(x=T * H * 2, wr=E * H * 4, bias=E * 4, ids=T * K * 4, w=T * K * 4, logits=T * E * 4),
            "loss": dict(logits=T * E * 4, ids=T * K * 4, mask=T, losses=8, counts=E * 4, prob=E * 4, n=4),
            "back": dict(logits=T * E * 4, ids=T * K * 4, mask=T, counts=E * 4, n=4, dl=8, w=T * K * 4, g=T * K * 4, out=T * E * 4),
            "grad": dict(x=T * H * 2, wr=E * H * 4, dl=T * E * 4, res=T * H * 2, dx=T * H * 2, dwr=E * H * 4)}
    outs = {"fwd": ("ids", "w", "logits"), "loss": ("losses", "counts", "prob", "n"), "back": ("out",), "grad": ("dx", "dwr")}
    for f, at in ((fwd, FWD), (loss, LOSS), (back, BACK), (grad, GRAD)):
        z = sizes[f.__name__]
        for o in outs[f.__name__]:
            for i in z:
                if i == o:
                    continue
                exact = (f.__name__, o, i) in (("back", "out", "logits"), ("grad", "dx", "res"))
                end = (z[i] + 15) // 16 * 16 - 16       # the last 16-byte place that touches i
                assert f(**{o: at[i]}) == (GONE if exact else INV), (f.__name__, o, i)
                if end > 0:
                    assert f(**{o: at[i] + end}) == INV, (f.__name__, o, i)
                assert f(**{o: at[i] + end + 16}) == GONE, (f.__name__, o, i)
    need = mok.router_workspace(P(T=16384))
    for f, at in ((loss, LOSS), (grad, GRAD)):
        for i in at:
            if i != "ws":
                assert f(p=P(T=16384), size=need, ws=at[i]) == INV, (f.__name__, i)


def test_python_refuses_other_tensors():
    w = F.get_router_workspace(4, 128, 8, 2, device="cpu")
    with pytest.raises(mok.MokError):
        F.run_router_losses(w, torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(mok.MokError):
        F.run_router_forward(w, torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(8, 128))


def test_rows_that_start_at_any_value():
    """Where E is not a multiple of 4, a slice of the tokens starts wherever it does."""
    for e in (37, 38, 39):
        p = P(E=e)
        for k in (4, 8, 12, 4 * e):
            assert loss(p=p, logits=LOSS["logits"] + k) == GONE and grad(p=p, dl=GRAD["dl"] + k) == GONE
            assert back(p=p, logits=BACK["logits"] + k, out=BACK["out"] + 4) == GONE
        assert loss(p=p, logits=LOSS["logits"] + 2) == INV and grad(p=p, dl=GRAD["dl"] + 2) == INV
        assert back(p=p, logits=BACK["logits"] + 2) == INV and back(p=p, out=BACK["out"] + 2) == INV
    for k in (4, 8):
        assert loss(logits=LOSS["logits"] + k) == INV and grad(dl=GRAD["dl"] + k) == INV
        assert back(logits=BACK["logits"] + k) == INV and back(out=BACK["out"] + k) == INV


def test_workspace_limits():
    """At most 256 partial rows of the losses' 2 E + 2 words, and 256 tiles of 128 x 256 of d_w_router, whatever the problem."""
    for t in (0, 1, 33, 203, 1037, 4099, 16384, 65536, 1 << 30):
        for h in (128, 256, 384, 2048, 4096, 7168, 1 << 14):
            for e in (1, 2, 37, 60, 64, 128, 129, 256, 300, 512):
                n = mok.router_workspace(P(T=t, H=h, E=e, topk=1))
                assert n <= max(256 * (2 * e + 2) * 4, 256 * 128 * 256 * 4), (t, h, e)
    # one slice of the tokens needs none, and the losses of few tokens neither
    assert mok.router_workspace(P(T=64, H=4096, E=128)) == 0
    # 16 slices of [128][4096], 9 of [32][7168]
    assert mok.router_workspace(P(T=16384, H=4096, E=128)) == 16 * 128 * 4096 * 4
    assert mok.router_workspace(P(T=16384, H=7168, E=32)) == 9 * 32 * 7168 * 4
    # 256 workgroups of the losses, at an H that needs less for d_w_router
    assert mok.router_workspace(P(T=1 << 20, H=128, E=1, topk=1)) >= 256 * 4 * 4
