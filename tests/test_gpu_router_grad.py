"""The dense router backward on the GPU: what its operands' parts keep.

u = 2^-24. dl and Wr go into the products of dx as three bf16 parts each, together all 24 bits. A part is at most 2^-7 of what
the parts before it left, so of dl Wr the products that are left out (second with third part, third with third) are less than
2 * 2^-22 + 2^-30 of it; the other six are exact in fp32 and are added in fp32. With k values of a row of dl different from zero
there are 6 k terms: dx is within ((6 k + 8) u + 2^-21) sum |dl Wr| of its value before it is rounded to bf16."""
import numpy as np
import pytest

import mixture_experts_layer_30_amd as mok
from ffn_testlib import HALF, assert_within, dot
from mixture_experts_layer_30_amd import functional as F
from test_gpu_losses import check_grad, f32
from test_gpu_mxfp4 import bf, f64

pytestmark = pytest.mark.gpu


def check_cancelled(T, H, E):
    """Two experts of a token, of opposite gradients and nearly equal rows of Wr: dx is their small difference, so that its own
    rounding hides nothing."""
    import torch
    g = np.random.default_rng(T + E)
    wr = (g.normal(size=H) * (1 + 2.0 ** -12 * g.normal(size=(E, H)))).astype(np.float32)
    a = g.integers(0, E, size=T)
    b = (a + g.integers(1, E, size=T)) % E
    v = g.normal(size=T).astype(np.float32)
    dl = np.zeros((T, E), np.float32)
    dl[np.arange(T), a], dl[np.arange(T), b] = v, -v
    ws = F.get_router_workspace(T, H, E, 1)
    dx, _ = F.run_router_logits_backward(ws, torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), f32(wr), f32(dl))
    torch.cuda.synchronize()
    w64, v64 = wr.astype(np.float64), v.astype(np.float64)[:, None]
    want = v64 * w64[a] - v64 * w64[b]
    e = (dot(12) + 2.0 ** -21) * (np.abs(v64 * w64[a]) + np.abs(v64 * w64[b]))
    assert_within(f64(dx), want, e + HALF * (np.abs(want) + e) + 1e-37, "dx")


@pytest.mark.parametrize("E", [2, 31, 33, 60, 64, 65, 128, 129, 200, 256, 257, 512])
def test_dx_keeps_all_bits(E):
    check_cancelled(203, 640, E)


@pytest.mark.parametrize("E", [32, 60, 100, 128])
def test_dx_keeps_all_bits_with_much_data(E):
    """More than 2^24 values of x: other launches than with less."""
    check_cancelled(4105, 4224, E)


@pytest.mark.parametrize("E", [30, 60, 100, 200, 300])
def test_grad_of_the_largest_and_smallest_values(E):
    """One token of each column and one expert of each row different from zero, at the ends of fp32: finite values stay finite,
    above bf16's largest too, and keep their 24 bits down to 2^-110. A value v below has a last bit of less than 2^(-110 - 23) =
    2^-133, bf16's smallest step, and its third part, cut to multiples of that, is short of it by less than 2^-133; the other two
    parts are multiples of at least 2^-126 where v is at least 2^-111."""
    import torch
    T, H = 64, 256
    g = np.random.default_rng(E)
    big = np.float32(np.finfo(np.float32).max)
    ends = np.concatenate([[big, -big], big * (1 - np.arange(1, 40) * 2.0 ** -10), 2.0 ** np.arange(-110, -90)]).astype(np.float32)
    ends = np.concatenate([ends, ends * np.float32(1 - 2.0 ** -9)])
    value = lambda *s: g.choice(ends, size=s) * (1 - g.integers(0, 2 ** 10, size=s) * 2.0 ** -24).astype(np.float32)  # noqa: E731
    ws = F.get_router_workspace(T, H, E, 1)
    # d_w_router: x = 2^-3 or 2^3 where the value is small, so that neither side leaves the range
    dl = value(T, E)
    tok = g.integers(0, T, size=H)
    for x in (2.0 ** -3, -2.0 ** 6):
        v = np.where((np.abs(dl) > 1) == (np.abs(x) < 1), dl, 0).astype(np.float32)
        X = np.zeros((T, H))
        X[tok, np.arange(H)] = x
        _, dwr = F.run_router_logits_backward(ws, bf(X), torch.zeros((E, H), device="cuda"), f32(v))
        torch.cuda.synchronize()
        want = v[tok].T.astype(np.float64) * x
        with np.errstate(invalid="ignore"):            # (0 / 0 in its message)
            assert_within(f64(dwr), want, np.where(np.abs(v[tok].T) < 2.0 ** -110, 2.0 ** -133 * abs(x), 0), "dwr")
    # dx = 2^-20 w and 2^20 w: one product of each part, then rounded
    wr, pick = value(E, H), g.integers(0, E, size=T)
    for d in (2.0 ** -20, 2.0 ** 20):
        v = np.where((np.abs(wr) > 1) == (d < 1), wr, 0).astype(np.float32)
        one = np.zeros((T, E), np.float32)
        one[np.arange(T), pick] = d
        dx, _ = F.run_router_logits_backward(ws, torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), f32(v), f32(one))
        torch.cuda.synchronize()
        want = v[pick].astype(np.float64) * d
        lost = np.where(np.abs(v[pick]) < 2.0 ** -110, 2.0 ** -133 * d, 0)
        assert_within(f64(dx), want, lost + HALF * (np.abs(want) + lost), "dx")


@pytest.mark.parametrize("E", [70, 128])
def test_grad_of_much_data(E):
    check_grad(4105, 4224, E, residual=E % 4 == 0, inplace=E == 128)


@pytest.mark.parametrize("T,H,E,steps", [(4099, 4096, 130, 16), (4099, 4096, 200, 16), (4001, 4096, 257, 25), (4099, 4096, 512, 32),
                                         (2080, 2048, 256, 4), (2050, 640, 300, 2)])
def test_grad_of_many_steps(T, H, E, steps):
    """Above 128 experts with at least `steps` times 32 tokens for each workgroup that forms d_w_router, odd numbers of them among
    these. (Those that form dx go through 8 or 9 times 32 tokens at H = 4096 up to 256 experts and 16 or 17 beyond, 16 tokens a
    step.) The workspace holds one [E][H] for each slice of the tokens."""
    slices = mok.router_workspace(mok.make_problem(T, H, 128, E, 1)) // (4 * E * H)
    assert (T + 31) // 32 // max(slices, 1) >= steps
    check_grad(T, H, E, residual=E != 200, inplace=E in (130, 512))


@pytest.mark.parametrize("T,H,E,dwr,dx", [(300, 1024, 70, 20, 40), (97, 1152, 9, 10, 10), (333, 1408, 100, 36, 66),
                                          (1100, 896, 70, 72, 126), (2000, 1152, 33, 105, 105), (4099, 1664, 128, 119, 221)])
def test_grad_of_workgroups_of_either_kind(T, H, E, dwr, dx):
    """Numbers of workgroups that form d_w_router and dx in one launch which are no multiples of 8, or of each other."""
    slices = mok.router_workspace(mok.make_problem(T, H, 128, E, 1)) // (4 * E * H)
    assert (slices * ((H + 255) // 256), slices * ((H + 127) // 128 if E > 64 else (H + 255) // 256)) == (dwr, dx)
    check_grad(T, H, E, residual=E % 2 == 0)


@pytest.mark.parametrize("E", [8, 60, 100, 200, 300])
def test_grad_past_32_bits(E):
    """More than 2^31 values, 2^32 bytes, of x, dx and the residual: the last rows are what they are alone. All of x but the last
    32 rows, one step of one workgroup, is zero, and so d_w_router is that step's."""
    import torch
    T, H = 300_032, 7168
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    g = torch.Generator(device="cuda").manual_seed(E)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-32:] = rnd(32, H).bfloat16()
    res = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    res[-96:] = rnd(96, H).bfloat16()
    dl, wr = rnd(T, E), rnd(E, H)
    tail = res[-96:].clone()
    dx, dwr = F.run_router_logits_backward(F.get_router_workspace(T, H, E, 1), x, wr, dl, residual=res, dx=res)
    dx2, _ = F.run_router_logits_backward(F.get_router_workspace(96, H, E, 1), x[-96:], wr, dl[-96:], residual=tail)
    _, dwr2 = F.run_router_logits_backward(F.get_router_workspace(32, H, E, 1), x[-32:], wr, dl[-32:])
    first = F.run_router_logits_backward(F.get_router_workspace(96, H, E, 1), x[:96], wr, dl[:96])[0]
    torch.cuda.synchronize()
    assert torch.equal(dx[-96:], dx2) and torch.equal(dwr, dwr2) and torch.equal(dx[:96], first)
