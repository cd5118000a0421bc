"""float64 references of the dense gated feed-forward block and of the MXFP4
format, written from the definitions in include/mok.h (test infrastructure; no
code shared with the HIP path)."""
from __future__ import annotations

import numpy as np

from .moe_oracle import e4m3_decode, mxfp8_quantize

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------ MXFP4
def e2m1_codes(q):
    """Codes of the E2M1 values nearest to q (float64), ties to the even code,
    saturating at 6: by distance to each of the eight values."""
    a = np.minimum(np.abs(q), 6.0)
    d = np.abs(a[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    even = np.argmax((d == best) & (np.arange(8) % 2 == 0), -1)
    odd = np.argmax(d == best, -1)
    has_even = ((d == best) & (np.arange(8) % 2 == 0)).any(-1)
    return np.where(has_even, even, odd).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 3)


def mxfp4_quantize(v):
    """v [rows][K] float64 -> (codes [rows][K] one a byte, scale bytes [rows][K/32])."""
    rows, K = v.shape
    b = v.reshape(rows, K // 32, 32)
    fine = np.isfinite(b).all(-1)
    amax = np.where(fine[..., None], np.abs(b), 0.0).max(-1)
    e = np.frexp(amax)[1] - 1
    s = np.where(amax > 0, np.clip(e - 2 + 127, 0, 254), 0)
    q = np.where(fine[..., None], b, 0.0) * np.exp2(127.0 - s)[..., None]
    codes = np.where(fine[..., None], e2m1_codes(q), 0)
    return codes.reshape(rows, K).astype(np.uint8), np.where(fine, s, 255).astype(np.uint8)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(q):
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)


def mxfp4_values(q, scales):
    """float64 values of packed codes [rows][K/2] and scales [rows][K/32]."""
    c = unpack(q)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    x = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(x, 32, -1)


def mxfp8_values(q, scales):
    x = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return e4m3_decode(q) * np.repeat(x, 32, -1)


def mxfp8_round(v):
    """The MXFP8 values of the rows of v; a block that is not finite becomes NaN."""
    rows, K = v.shape
    b = v.reshape(rows, K // 32, 32)
    fine = np.isfinite(b).all(-1)
    q, s = mxfp8_quantize(np.where(fine[..., None], b, 0.0).reshape(rows, K))
    out = mxfp8_values(q, s).reshape(b.shape)
    return np.where(fine[..., None], out, np.nan).reshape(rows, K)


# ------------------------------------------------------------------ gates
def act(a, kind):
    """(act(a), act'(a)) of "silu" or "gelu" (tanh form)."""
    if kind == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * a))
        return a * s, s + a * s * (1 - s)
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * c * (1 + 3 * 0.044715 * a * a)


# ------------------------------------------------------------------ dense block
def ffn_forward(x, wg, wu, wd, kind, residual=None, mx=False):
    """dict of a, b, h (MXFP8-rounded with mx), y; with mx the weights are the values of MXFP4 codes."""
    xq = mxfp8_round(x) if mx else x
    a, b = xq @ wg.T, xq @ wu.T
    h = act(a, kind)[0] * b
    hq = mxfp8_round(h) if mx else h
    y = hq @ wd.T
    return {"x": xq, "a": a, "b": b, "h": h, "hq": hq, "y": y if residual is None else y + residual}


def ffn_backward(x, a, b, wg, wu, wd, dy, kind):
    """Gradients of <dy, y> given the saved pre-activations."""
    f, df = act(a, kind)
    dh = dy @ wd
    da, db, h = dh * b * df, dh * f, f * b
    return {"dh": dh, "da": da, "db": db, "h": h, "dx": da @ wg + db @ wu, "dwg": da.T @ x, "dwu": db.T @ x,
            "dwd": dy.T @ h}
