"""Calls of the dense gated feed-forward block and of the MXFP4 format, as they are used beside a
mixture-of-experts layer: the shared expert that every token passes (bf16 in training, 4-bit weights in
serving) and the 4-bit quantization and product below it.

Operators
  quantize   MXFP4 codes of bf16 rows (E2M1, one E8M0 scale per 32 along the row) and the values read back
  matmul     D = A . B^T with B in MXFP4 and A in MXFP4 or MXFP8, both blocked by 32 along K, D in bf16
  forward    y = (act(x Wg^T) * (x Wu^T)) Wd^T [+ residual]; in training also the pre-activations [a | b]
  backward   dx, dWg, dWu, dWd from dy and the saved pre-activations

`own` chooses between the plain form of each (torch, 32-bit) and the library's call.
"""
import math

import torch

own = False

BLOCK = 32
E2M1_MAX_EXP, E4M3_MAX_EXP = 2, 8


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the activations of a full training batch, hidden size 7168: what a memory-bound pass costs
        {"name": "quantize_16384x7168", "op": "quantize", "rows": 16384, "K": 7168},
        # one ragged decode batch of expert activations: a launch and little else
        {"name": "quantize_37x768", "op": "quantize", "rows": 37, "K": 768},
        # one decoded token against one expert's gate and up rows: the 4-bit weights are all the traffic
        {"name": "matmul_a8_1x4096x7168", "op": "matmul", "a": "mxfp8", "M": 1, "N": 4096, "K": 7168},
        # a ragged prompt, both sides in 4 bits, N not a multiple of any tile
        {"name": "matmul_a4_1037x1544x4096", "op": "matmul", "a": "mxfp4", "M": 1037, "N": 1544, "K": 4096},
        # the largest batch through a gate|up product, both sides in 4 bits
        {"name": "matmul_a4_16384x4096x7168", "op": "matmul", "a": "mxfp4", "M": 16384, "N": 4096, "K": 7168},
        # shared expert, one token, bf16: the three weight matrices are read once
        {"name": "forward_bf16_1", "op": "forward", "dtype": "bf16", "act": "silu", "train": False,
         "T": 1, "H": 7168, "I": 2048},
        # a ragged batch with sizes that fill no tile, GELU gate, in training
        {"name": "forward_bf16_777_odd", "op": "forward", "dtype": "bf16", "act": "gelu", "train": True,
         "T": 777, "H": 1000, "I": 712},
        # a training batch of the mid-size layer
        {"name": "forward_bf16_16384", "op": "forward", "dtype": "bf16", "act": "silu", "train": True,
         "T": 16384, "H": 4096, "I": 1536},
        # shared expert with 4-bit weights, a decode batch of 16
        {"name": "forward_mxfp4_16", "op": "forward", "dtype": "mxfp4", "act": "silu", "train": False,
         "T": 16, "H": 7168, "I": 2048},
        # shared expert with 4-bit weights, a prompt
        {"name": "forward_mxfp4_4096", "op": "forward", "dtype": "mxfp4", "act": "silu", "train": False,
         "T": 4096, "H": 4096, "I": 1536},
        # backward of a small layer, a ragged batch: few output tiles, long sums over the tokens
        {"name": "backward_4093_small", "op": "backward", "act": "gelu", "T": 4093, "H": 2048, "I": 768},
        # backward of the full-size layer, a full batch: the largest call
        {"name": "backward_16384", "op": "backward", "act": "silu", "T": 16384, "H": 7168, "I": 2048},
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step, max(-(-lo // step), round(v / step))) * step


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "forward", "forward", "backward"])
    if op == "quantize":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "K": _log_int(rng, 256, 7168, 32)}
    if op == "matmul":
        return {"op": op, "a": rng.choice(["mxfp8", "mxfp4"]), "M": _log_int(rng, 1, 16384),
                "N": _log_int(rng, 256, 7168), "K": _log_int(rng, 256, 7168, 128)}
    act = rng.choice(["silu", "gelu"])
    if op == "backward":
        return {"op": op, "act": act, "T": _log_int(rng, 64, 16384), "H": _log_int(rng, 256, 7168, 8),
                "I": _log_int(rng, 256, 2048, 8)}
    dtype = rng.choice(["bf16", "mxfp4"])
    step = 8 if dtype == "bf16" else 128
    return {"op": op, "dtype": dtype, "act": act, "train": dtype == "bf16" and rng.random() < 0.5,
            "T": _log_int(rng, 1, 16384), "H": _log_int(rng, 256, 7168, step),
            "I": _log_int(rng, 256, 2048, step)}


def work(case):
    mx = 0.5 + 1 / BLOCK                            # bytes of an MXFP4 value with its share of the scale
    if case["op"] == "quantize":
        n = case["rows"] * case["K"]
        return {"bytes": n * (2 + 2 + 2 * mx), "flops": 0}   # rows in, codes out; codes in, rows out
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        a = mx if case["a"] == "mxfp4" else 1 + 1 / BLOCK
        return {"bytes": M * K * a + N * K * mx + 2 * M * N, "flops": 2 * M * N * K}
    T, H, I = case["T"], case["H"], case["I"]
    if case["op"] == "backward":
        # x, dy, [a | b] and the weights in; dx and the weight gradients out
        return {"bytes": 2 * (3 * T * H + 2 * T * I + 6 * H * I), "flops": 12 * T * H * I}
    w = 3 * H * I * (2 if case["dtype"] == "bf16" else mx)
    extra = 2 * T * I if case["train"] else T * H   # [a | b] out, or the residual in
    return {"bytes": w + 2 * (2 * T * H + extra), "flops": 6 * T * H * I}


# ------------------------------------------------------------------ the formats, plain form
def _scale_exp(v, max_exp):
    """Block exponent of v [..., K/32, 32]: floor(log2 amax) - max_exp, held to E8M0; -127 for zeros."""
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax).exponent - 1 - max_exp
    return torch.where(amax > 0, e.clamp(-127, 127), torch.full_like(e, -127))


def _e2m1(q):
    """Nearest E2M1 value, ties to even, held to +-6."""
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6).copysign(q)


def _e4m3(q):
    """Nearest E4M3 value, ties to even, held to +-448."""
    a = q.abs()
    step = torch.ldexp(torch.ones_like(a), (torch.frexp(a).exponent - 1).clamp(min=-6) - 3)
    return (torch.round(a / step) * step).clamp(max=448).copysign(q)


def _mx(v, max_exp, grid):
    """(element values, block exponents) of the rows of v."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    e = _scale_exp(b, max_exp)
    half = e // 2                                   # two steps: 2^-e alone can pass the type's range
    q = grid(torch.ldexp(torch.ldexp(b, -half), half - e))
    return q, e


def _values(q, e):
    half = e // 2
    return torch.ldexp(torch.ldexp(q, half), e - half).flatten(-2)


def _quantized(v, max_exp, grid):
    return _values(*_mx(v, max_exp, grid))


def _pack_e2m1(q):
    """Packed codes of E2M1 values [..., K]: element 2i in the low nibble of byte i."""
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack_e2m1(packed):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float32, device=packed.device)
    table = torch.cat([table, -table])
    return table[torch.stack([packed & 15, packed >> 4], -1).flatten(-2).int()]


def _decode(codes, scales, fmt):
    v = _unpack_e2m1(codes) if fmt == "mxfp4" else codes.view(torch.float8_e4m3fn).float()
    return _values(v.reshape(*v.shape[:-1], -1, BLOCK), scales.int().unsqueeze(-1) - 127)


def _encode(v, fmt):
    """(codes, scales) of bf16 or fp32 rows, as a program that quantized them before holds them."""
    v = v.float()
    q, e = _mx(v, *((E2M1_MAX_EXP, _e2m1) if fmt == "mxfp4" else (E4M3_MAX_EXP, _e4m3)))
    codes = _pack_e2m1(q.flatten(-2)) if fmt == "mxfp4" else q.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e.squeeze(-1) + 127).to(torch.uint8)


# ------------------------------------------------------------------ inputs
def _inputs(case, seed):
    """The call's bf16 inputs (and codes) on the GPU: activations with channels of unequal size, as a
    residual stream has them; weights of standard deviation fan_in^-1/2."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    def rows(n, k):
        channel = torch.exp(0.7 * torch.randn(k, generator=g, device="cuda"))
        return (torch.randn(n, k, generator=g, device="cuda") * channel).bfloat16()

    if case["op"] == "quantize":
        return {"src": rows(case["rows"], case["K"])}
    if case["op"] == "matmul":
        a, sa = _encode(rows(case["M"], case["K"]), case["a"])
        b, sb = _encode(normal(case["N"], case["K"], std=case["K"] ** -0.5), "mxfp4")
        return {"a": a, "sa": sa, "b": b, "sb": sb}
    T, H, I = case["T"], case["H"], case["I"]
    s = {"x": normal(T, H), "wg": normal(I, H, std=H ** -0.5), "wu": normal(I, H, std=H ** -0.5),
         "wd": normal(H, I, std=I ** -0.5)}
    if case["op"] == "backward":
        s["dy"] = normal(T, H)
        s["ab"] = torch.cat([s["x"] @ s["wg"].t(), s["x"] @ s["wu"].t()], 1)
    elif not case["train"]:
        s["residual"] = normal(T, H)
    if case["op"] == "forward" and case["dtype"] == "mxfp4":
        for n in ("wg", "wu", "wd"):
            s[n], s["s" + n[1:]] = _encode(s[n], "mxfp4")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    s["buffers"] = {}                               # what the library's calls write into, made on the first one
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _buffers(s):
    """Workspace of the library's call, kept with the state as a program keeps it."""
    import mixture_experts_layer_30_amd as mok
    from mixture_experts_layer_30_amd import functional as F
    c, b = s["case"], s["buffers"]
    if c["op"] == "matmul":
        b["a_dtype"] = mok.MOK_MXFP4 if c["a"] == "mxfp4" else mok.MOK_MXFP8
        b["ws"] = F.get_mx_matmul_workspace(c["M"], c["N"], c["K"], b["a_dtype"])
    elif c["op"] in ("forward", "backward"):
        mx = c.get("dtype") == "mxfp4"
        b["ws"] = F.get_ffn_workspace(
            c["T"], c["H"], c["I"], dtype=mok.MOK_MXFP4 if mx else mok.MOK_BF16,
            activation=mok.ACT_SILU if c["act"] == "silu" else mok.ACT_GELU_TANH,
            training=c["op"] == "backward" or c["train"])
        b["weights"] = (s["wg"], s["wu"], s["wd"]) + ((s["sg"], s["su"], s["sd"]) if mx else ())
        if c["op"] == "backward":
            b["ws"].ctx = s["ab"]
    b["ready"] = True
    return F


def _run_own(s):
    b = s["buffers"]
    if "ready" not in b:
        b["F"] = _buffers(s)
    F, op = b["F"], s["case"]["op"]
    if op == "quantize":
        return F.mxfp4_dequantize(*F.mxfp4_quantize(s["src"]))
    if op == "matmul":
        return F.run_mx_matmul(b["ws"], s["a"], s["sa"], s["b"], s["sb"])
    if op == "backward":
        return F.run_ffn_backward(b["ws"], s["x"], b["weights"], s["dy"])
    if s["case"]["train"]:
        return F.run_ffn_forward(b["ws"], s["x"], b["weights"]), b["ws"].ctx
    return F.run_ffn_forward(b["ws"], s["x"], b["weights"], residual=s["residual"])


def _act(a, name):
    """(act(a), act'(a))"""
    if name == "silu":
        sg = 1 / (1 + torch.exp(-a))
        return a * sg, sg * (1 + a * (1 - sg))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (a + 0.044715 * a ** 3))
    return 0.5 * a * (1 + th), 0.5 * (1 + th) + 0.5 * a * (1 - th * th) * c * (1 + 3 * 0.044715 * a * a)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        return _quantized(s["src"].float(), E2M1_MAX_EXP, _e2m1).bfloat16()
    if case["op"] == "matmul":
        return (_decode(s["a"], s["sa"], case["a"]) @ _decode(s["b"], s["sb"], "mxfp4").t()).bfloat16()
    x = s["x"].float()
    if case["op"] == "backward":
        wg, wu, wd, dy = s["wg"].float(), s["wu"].float(), s["wd"].float(), s["dy"].float()
        a, b = s["ab"].float().chunk(2, 1)
        act, dact = _act(a, case["act"])
        dh = dy @ wd
        da, db = dh * b * dact, dh * act
        return ((da @ wg + db @ wu).bfloat16(), (da.t() @ x).bfloat16(), (db.t() @ x).bfloat16(),
                (dy.t() @ (act * b)).bfloat16())
    if case["dtype"] == "mxfp4":
        wg, wu, wd = (_decode(s["w" + n], s["s" + n], "mxfp4") for n in "gud")
        x = _quantized(x, E4M3_MAX_EXP, _e4m3)
    else:
        wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    a, b = x @ wg.t(), x @ wu.t()
    h = _act(a, case["act"])[0] * b
    if case["dtype"] == "mxfp4":
        h = _quantized(h, E4M3_MAX_EXP, _e4m3)
    y = h @ wd.t()
    if case["train"]:
        return y.bfloat16(), torch.cat([a, b], 1).bfloat16()
    return (y + s["residual"].float()).bfloat16()


# ------------------------------------------------------------------ the definition, 64 bits
def _exact_mx(v, top, mantissa, lowest):
    """Values of the MX blocks of v in float64: grid of `mantissa` bits from 2^lowest on, saturating at top."""
    b = v.double().reshape(*v.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax))
    e = torch.where(torch.exp2(e) > amax, e - 1, torch.where(torch.exp2(e + 1) <= amax, e + 1, e))
    x = torch.exp2((e - math.floor(math.log2(top))).clamp(-127, 127))
    x = torch.where(amax > 0, x, torch.ones_like(x))
    m = (b / x).abs()
    f = torch.floor(torch.log2(m.clamp(min=2.0 ** lowest)))
    f = torch.where(torch.exp2(f) > m, f - 1, torch.where(torch.exp2(f + 1) <= m, f + 1, f)).clamp(min=lowest)
    u = torch.exp2(f - mantissa)
    return (torch.sign(b) * torch.round(m / u).mul(u).clamp(max=top) * x).flatten(-2)


def _exact_codes(codes, scales, fmt):
    if fmt == "mxfp4":
        n = torch.stack([codes % 16, codes // 16], -1).flatten(-2).double()
        sign, n = 1 - 2 * torch.floor(n / 8), n % 8
        exp, man = torch.floor(n / 2), n % 2
        v = sign * torch.where(exp > 0, (1 + man / 2) * torch.exp2(exp - 1), man / 2)
    else:
        n = codes.double()
        sign, n = 1 - 2 * torch.floor(n / 128), n % 128
        exp, man = torch.floor(n / 8), n % 8
        v = sign * torch.where(exp > 0, (1 + man / 8) * torch.exp2(exp - 7), man / 8 * 2.0 ** -6)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def _exact_act(a, name):
    if name == "silu":
        return a * torch.special.expit(a)
    return a * torch.special.expit(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a))


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quantize":
        return _exact_mx(s["src"], 6.0, 1, 0)
    if case["op"] == "matmul":
        return _exact_codes(s["a"], s["sa"], case["a"]) @ _exact_codes(s["b"], s["sb"], "mxfp4").t()
    x = s["x"].double()
    if case["op"] == "backward":
        ab = s["ab"].double().requires_grad_()
        I = case["I"]
        with torch.enable_grad():
            h = _exact_act(ab[:, :I], case["act"]) * ab[:, I:]
        dy = s["dy"].double()
        (dab,) = torch.autograd.grad(h, ab, dy @ s["wd"].double())
        w = torch.cat([s["wg"], s["wu"]]).double()
        dw = dab.t() @ x
        return dab @ w, dw[:I], dw[I:], dy.t() @ h.detach()
    if case["dtype"] == "mxfp4":
        w = [_exact_codes(s["w" + n], s["s" + n], "mxfp4") for n in "gud"]
        x = _exact_mx(x, 448.0, 3, -6)
    else:
        w = [s["w" + n].double() for n in "gud"]
    a, b = x @ w[0].t(), x @ w[1].t()
    h = _exact_act(a, case["act"]) * b
    if case["dtype"] == "mxfp4":
        h = _exact_mx(h, 448.0, 3, -6)
    y = h @ w[2].t()
    if case["train"]:
        return y, torch.cat([a, b], 1)
    return y + s["residual"].double()
