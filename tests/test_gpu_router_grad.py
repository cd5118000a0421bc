"""The dense router backward on the GPU: what its operands' parts keep.

u = 2^-24. dl and Wr go into the products of dx as three bf16 parts each, together all 24 bits. A part is at most 2^-7 of what
the parts before it left, so of dl Wr the products that are left out (second with third part, third with third) are less than
2 * 2^-22 + 2^-30 of it; the other six are exact in fp32 and are added in fp32. With k values of a row of dl different from zero
there are 6 k terms: dx is within ((6 k + 8) u + 2^-21) sum |dl Wr| of its value before it is rounded to bf16."""
import numpy as np
import pytest

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


@pytest.mark.parametrize("E", [70, 128])
def test_grad_of_much_data(E):
    check_grad(4105, 4224, E, residual=E % 4 == 0, inplace=E == 128)
