"""The dense gated feed-forward block on the GPU against its float64 reference,
element by element within the bounds of its arithmetic (ffn_testlib)."""
import numpy as np
import pytest

import mixture_experts_layer_30_amd as mok
import oracle.dense_oracle as do
from ffn_testlib import assert_within, backward_bounds, forward_bounds
from mixture_experts_layer_30_amd import functional as F
from oracle import bf16_round

pytestmark = pytest.mark.gpu
ACT = {"silu": mok.ACT_SILU, "gelu": mok.ACT_GELU_TANH}


def bf(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def case(T, H, I, seed=0):
    g = np.random.default_rng(seed * 1000003 + T * 7919 + H * 31 + I)
    n = lambda *s, std=1.0: bf16_round(g.normal(size=s).astype(np.float32) * std).astype(np.float64)  # noqa: E731
    return {"x": n(T, H) * np.exp2(g.integers(-2, 3, size=H)), "wg": n(I, H, std=H ** -0.5),
            "wu": n(I, H, std=H ** -0.5), "wd": n(H, I, std=I ** -0.5), "dy": n(T, H), "res": n(T, H)}


# one token to a few thousand; sizes below a tile, of whole tiles, just past them, of a single 8; the
# products of the last rows run as 256 x 256 tiles (the weight gradients of the very last split along K),
# those of the others as 128 x 128, split along K or not
SHAPES = [(1, 8, 8), (1, 256, 512), (2, 1000, 712), (16, 2048, 768), (17, 264, 520), (32, 1024, 136), (33, 264, 520),
          (64, 7168, 256), (128, 128, 128), (129, 136, 72), (257, 8, 2048), (300, 2048, 768), (513, 4096, 8),
          (777, 1000, 712), (1031, 520, 264), (4100, 520, 2056), (2049, 2312, 1096), (4671, 3032, 64)]


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward_and_backward(T, H, I, kind):
    import torch
    c = case(T, H, I)
    d = {k: bf(v) for k, v in c.items()}
    w = (d["wg"], d["wu"], d["wd"])
    ws = F.get_ffn_workspace(T, H, I, activation=ACT[kind])
    y = F.run_ffn_forward(ws, d["x"], w, residual=d["res"])
    ctx = ws.ctx.clone()
    grads = F.run_ffn_backward(ws, d["x"], w, d["dy"])
    torch.cuda.synchronize()
    r = do.ffn_forward(c["x"], c["wg"], c["wu"], c["wd"], kind, c["res"])
    b = forward_bounds(r, c["x"], c["wg"], c["wu"], c["wd"], kind, c["res"])
    assert_within(f64(y), r["y"], b["y"], "y")
    assert_within(f64(ctx), np.concatenate([r["a"], r["b"]], 1), b["ab"], "ab")
    assert torch.equal(ctx, ws.ctx)                      # the backward only reads it
    sa, sb = f64(ctx)[:, :I], f64(ctx)[:, I:]
    r = do.ffn_backward(c["x"], sa, sb, c["wg"], c["wu"], c["wd"], c["dy"], kind)
    b = backward_bounds(r, c["x"], sa, sb, c["wg"], c["wu"], c["wd"], c["dy"], kind)
    for k, t in zip(("dx", "dwg", "dwu", "dwd"), grads):
        assert_within(f64(t), r[k], b[k], k)


def test_no_tokens():
    import torch
    ws = F.get_ffn_workspace(0, 264, 136)
    w = tuple(torch.randn(s, device="cuda").bfloat16() for s in ((136, 264), (136, 264), (264, 136)))
    x = torch.empty((0, 264), dtype=torch.bfloat16, device="cuda")
    assert F.run_ffn_forward(ws, x, w).shape == (0, 264)
    dx, *dw = F.run_ffn_backward(ws, x, w, x)
    torch.cuda.synchronize()
    assert dx.shape == (0, 264)
    for g, t in zip(dw, w):
        assert g.shape == t.shape and not g.any()


@pytest.mark.parametrize("T,H,I", [(5, 264, 136), (200, 264, 136), (4100, 520, 2056)])
def test_row_pitches_and_what_lies_around(T, H, I):
    """x, y, dy, dx as windows of wider matrices: the same bits as contiguous ones, and nothing outside the
    windows (columns, rows behind the last) is read into a result or written."""
    import torch
    c = {k: bf(v) for k, v in case(T, H, I, 1).items()}
    w = (c["wg"], c["wu"], c["wd"])
    ws = F.get_ffn_workspace(T, H, I)
    y0 = F.run_ffn_forward(ws, c["x"], w, residual=c["res"])
    g0 = F.run_ffn_backward(ws, c["x"], w, c["dy"])

    def window(t, extra):
        big = torch.full((T + 3, H + extra), float("nan"), dtype=torch.bfloat16, device="cuda")
        v = big[1:T + 1, 8:8 + H]
        if t is not None:
            v.copy_(t)
        return big, v

    bx, x = window(c["x"], 24)
    _, res = window(c["res"], 40)
    by, y = window(None, 40)
    _, dy = window(c["dy"], 16)
    bd, dx = window(None, 24)
    mok.ffn_forward(ws.problem, x, w, y, ws.workspace, residual=res, ctx=ws.ctx)
    dw = [torch.empty_like(t) for t in w]
    mok.ffn_backward(ws.problem, ws.ctx, x, w, dy, dx, *dw, ws.workspace)
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(dx, g0[0])
    for a, b in zip(dw, g0[1:]):
        assert torch.equal(a, b)
    for big, v in ((by, y), (bd, dx)):
        assert int(big.isnan().sum()) == big.numel() - v.numel()


@pytest.mark.parametrize("T,H", [(1, 1024), (40, 1024), (2500, 1024), (4111, 4104)])
def test_residual_in_place(T, H):
    import torch
    I = 520
    c = {k: bf(v) for k, v in case(T, H, I, 2).items()}
    w = (c["wg"], c["wu"], c["wd"])
    ws = F.get_ffn_workspace(T, H, I, training=False)
    want = F.run_ffn_forward(ws, c["x"], w, residual=c["res"])
    y = c["res"].clone()
    assert F.run_ffn_forward(ws, c["x"], w, residual=y, y=y) is y
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("T,H,I", [(3, 256, 136), (300, 264, 136), (4100, 520, 2056)])
def test_what_is_not_finite_stays_in_its_rows(T, H, I):
    """A NaN and an infinity in two tokens' x and dy: the other tokens' outputs keep their bits (the padding of
    tiles and of K never multiplies a neighbour's values)."""
    import torch
    c = {k: bf(v) for k, v in case(T, H, I, 3).items()}
    w = (c["wg"], c["wu"], c["wd"])
    ws = F.get_ffn_workspace(T, H, I)
    y0 = F.run_ffn_forward(ws, c["x"], w)
    dx0 = F.run_ffn_backward(ws, c["x"], w, c["dy"])[0]
    x, dy = c["x"].clone(), c["dy"].clone()
    x[T - 1, H - 1] = float("nan")
    x[0, 0] = float("inf")
    dy[T - 1, 0] = float("nan")
    y = F.run_ffn_forward(ws, x, w)
    dx = F.run_ffn_backward(ws, x, w, dy)[0]
    torch.cuda.synchronize()
    assert not y[T - 1].isfinite().any() and not y[0].isfinite().all()
    assert torch.equal(y[1:T - 1], y0[1:T - 1]) and torch.equal(dx[1:T - 1], dx0[1:T - 1])
    assert not dx[T - 1].isfinite().any()


@pytest.mark.parametrize("T,H,I", [(1, 2048, 768), (24, 2048, 768), (300, 2048, 768), (4100, 520, 2056)])
def test_bitwise_run_to_run_and_in_a_graph(T, H, I):
    """Ten eager runs and six replays of a captured forward + backward, with eager work between, bit for bit."""
    import torch
    c = {k: bf(v) for k, v in case(T, H, I, 4).items()}
    w = (c["wg"], c["wu"], c["wd"])
    ws = F.get_ffn_workspace(T, H, I)
    y, dx = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    dw = [torch.empty_like(t) for t in w]

    def step(ws):
        mok.ffn_forward(ws.problem, c["x"], w, y, ws.workspace, residual=c["res"], ctx=ws.ctx)
        mok.ffn_backward(ws.problem, ws.ctx, c["x"], w, c["dy"], dx, *dw, ws.workspace)

    step(ws)
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, *dw)]
    outs = (y, dx, *dw)
    for _ in range(10):
        for t in outs:
            t.zero_()
        step(ws)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    gws = F.get_ffn_workspace(T, H, I)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(gws)
    for k in range(6):
        for t in outs:
            t.zero_()
        gws.workspace.fill_(0xFF)                        # no state of a replay is used by the next
        if k % 2:
            step(ws)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k


def test_two_streams_at_once():
    import torch
    T, H, I = 70, 2048, 768
    c = {k: bf(v) for k, v in case(T, H, I, 5).items()}
    w = (c["wg"], c["wu"], c["wd"])
    ws = [F.get_ffn_workspace(T, H, I) for _ in range(2)]
    want = F.run_ffn_forward(ws[0], c["x"], w)
    xr = c["x"].flip(0).contiguous()
    want_r = F.run_ffn_forward(ws[0], xr, w)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    ys = [[], []]
    for _ in range(8):
        for k, x in enumerate((c["x"], xr)):
            with torch.cuda.stream(st[k]):
                ys[k].append(F.run_ffn_forward(ws[k], x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys[0]) and all(torch.equal(y, want_r) for y in ys[1])


def test_shared_expert_beside_the_routed_ones():
    """The routed layer and the shared expert as a model runs them: y = layer(x) + block(x), the block adding
    into the layer's output, and both backwards."""
    import torch
    T, H, I, E, k = 300, 256, 384, 6, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    x, dy = n(T, H), n(T, H)
    we = (n(E, I, H, std=H ** -0.5), n(E, I, H, std=H ** -0.5), n(E, H, I, std=I ** -0.5))
    wsh = (n(I, H, std=H ** -0.5), n(I, H, std=H ** -0.5), n(H, I, std=I ** -0.5))
    layer = F.get_workspace(T, H, I, E, k)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    tw = torch.empty((T, k), dtype=torch.float32, device="cuda")
    mok.router_forward(layer.problem, x, torch.randn(E, H, generator=g, device="cuda") * H ** -0.5, None, ids, tw)
    F.run_schedule(layer, ids)
    y = F.run_forward(layer, x, tw, we)
    routed = y.clone()
    block = F.get_ffn_workspace(T, H, I)
    F.run_ffn_forward(block, x, wsh, residual=y, y=y)
    dxl = F.run_backward(layer, x, tw, we, dy)[0]
    dxs, *dws = F.run_ffn_backward(block, x, wsh, dy)
    torch.cuda.synchronize()
    c = [f64(t) for t in (x, *wsh, dy)]
    r = do.ffn_forward(*c[:4], "silu", f64(routed))
    assert_within(f64(y), r["y"], forward_bounds(r, *c[:4], "silu", f64(routed))["y"], "y")
    a, b = f64(block.ctx)[:, :I], f64(block.ctx)[:, I:]
    r = do.ffn_backward(c[0], a, b, *c[1:], "silu")
    bound = backward_bounds(r, c[0], a, b, *c[1:], "silu")
    for name, t in zip(("dx", "dwg", "dwu", "dwd"), (dxs, *dws)):
        assert_within(f64(t), r[name], bound[name], name)
    # a layer of one expert that every token picks with weight 1 is the same block
    one = F.get_workspace(T, H, I, 1, 1)
    F.run_schedule(one, torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    y1 = F.run_forward(one, x, torch.ones((T, 1), device="cuda"), tuple(t.unsqueeze(0) for t in wsh))
    y2 = F.run_ffn_forward(block, x, wsh)
    torch.cuda.synchronize()
    r = do.ffn_forward(*c[:4], "silu")
    bound = forward_bounds(r, *c[:4], "silu")["y"]
    assert_within(f64(y1), f64(y2), 2 * bound, "one expert")
    assert torch.isfinite(dxl).all()


def test_binding_refuses():
    import torch
    T, H, I = 8, 256, 128
    ws = F.get_ffn_workspace(T, H, I)
    c = {k: bf(v) for k, v in case(T, H, I).items()}
    w = (c["wg"], c["wu"], c["wd"])
    wide = torch.zeros((T, 2 * H), dtype=torch.bfloat16, device="cuda")

    def refused(**kw):
        a = dict(x=c["x"], w=w, y=torch.empty_like(c["x"]), residual=None, ctx=None)
        a.update(kw)
        with pytest.raises(mok.MokError) as e:
            mok.ffn_forward(ws.problem, a["x"], a["w"], a["y"], ws.workspace, residual=a["residual"], ctx=a["ctx"])
        assert e.value.status == mok.MOK_ERR_INVALID_ARG

    refused(x=c["x"].float())
    refused(x=c["x"][:4])
    refused(x=c["x"][:1].expand(T, H))                   # rows that share memory
    refused(x=wide[:, ::2])                              # a step within a row
    refused(x=wide[:, 4:4 + H])                          # off a 16-byte boundary
    refused(x=c["x"].cpu())
    refused(y=wide[:, :H], residual=c["x"])              # two pitches for one
    refused(ctx=torch.empty((T, I), dtype=torch.bfloat16, device="cuda"))
    refused(w=(w[0], w[1], w[2].t()))
    refused(w=w[:2])


@pytest.mark.parametrize("T,H,I", [(3, 256, 128), (200, 256, 128), (2500, 2048, 768), (4100, 2048, 768)])
def test_outputs_in_place_of_inputs(T, H, I):
    """y over x (as residual too): the same bits as in a buffer of its own. dx beside x in the same rows is fine;
    any overlap with x or dy, which are read while it is written, is refused."""
    import torch
    c = {k: bf(v) for k, v in case(T, H, I).items()}
    w = (c["wg"], c["wu"], c["wd"])
    ws = F.get_ffn_workspace(T, H, I)
    y = F.run_ffn_forward(ws, c["x"], w, residual=c["x"])
    dx, *dw = F.run_ffn_backward(ws, c["x"], w, c["dy"])
    over = c["x"].clone()
    F.run_ffn_forward(ws, over, w, residual=over, y=over)
    assert torch.equal(over, y)

    def back(x, dy, dx):
        g = [torch.full_like(t, float("nan")) for t in dw]
        mok.ffn_backward(ws.problem, ws.ctx, x, w, dy, dx, *g, ws.workspace)
        return g

    for kw in (dict(x=c["x"], dy=c["dy"], dx=c["x"]), dict(x=c["x"], dy=c["dy"], dx=c["dy"])):
        with pytest.raises(mok.MokError) as e:
            back(**kw)
        assert e.value.status == mok.MOK_ERR_INVALID_ARG
    wide = torch.zeros((T, 2 * H), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = c["x"]
    g = back(wide[:, :H], c["dy"], wide[:, H:])
    assert torch.equal(wide[:, H:], dx) and all(torch.equal(p, q) for p, q in zip(g, dw))
    with pytest.raises(mok.MokError):
        back(wide[:, :H], c["dy"], wide[:, 8:H + 8])


def test_offsets_past_32_bits():
    """Two billion elements of x, y, dy and dx: the last tokens' outputs and the weight gradients, whose sums run
    over all tokens."""
    import torch
    T, H, I = 1_100_003, 2048, 16
    assert T * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    w = tuple((torch.randn(s, generator=g, device="cuda") * s[1] ** -0.5).bfloat16() for s in ((I, H), (I, H), (H, I)))
    ws = F.get_ffn_workspace(T, H, I)
    y = F.run_ffn_forward(ws, x, w)
    dx, dwg, dwu, dwd = F.run_ffn_backward(ws, x, w, dy)
    torch.cuda.synchronize()
    t = slice(T - 300, T)
    c = [f64(v) for v in (x[t], *w, dy[t])]
    r = do.ffn_forward(*c[:4], "silu")
    assert_within(f64(y[t]), r["y"], forward_bounds(r, *c[:4], "silu")["y"], "y")
    a, b = f64(ws.ctx[t])[:, :I], f64(ws.ctx[t])[:, I:]
    r = do.ffn_backward(c[0], a, b, *c[1:], "silu")
    assert_within(f64(dx[t]), r["dx"], backward_bounds(r, c[0], a, b, *c[1:], "silu")["dx"], "dx")
    # the sums over all tokens in double, by chunks, with their magnitudes for the bound: h, da, db are
    # rounded to bf16 (2^-8) after the gate (2^-15 of terms up to 1 + |a| / 4 of |dh b|), T terms in fp32
    ref = {k: torch.zeros(s, dtype=torch.float64, device="cuda") for k, s in
           (("dwg", (I, H)), ("dwu", (I, H)), ("dwd", (H, I)))}
    mag = {k: v.clone() for k, v in ref.items()}
    wd = w[2].double()
    for k in range(0, T, 1 << 17):
        q = slice(k, min(T, k + (1 << 17)))
        xc, dc, ab = x[q].double(), dy[q].double(), ws.ctx[q].double()
        a, b = ab[:, :I], ab[:, I:]
        s = torch.sigmoid(a)
        dh = dc @ wd
        da, db, h = dh * b * s * (1 + a * (1 - s)), dh * a * s, a * s * b
        for n, u, v, loose in (("dwg", da, xc, (dh * b).abs() * (1 + a.abs())), ("dwu", db, xc, db.abs()),
                               ("dwd", dc, h, None)):
            ref[n] += u.t() @ v
            mag[n] += (u.abs() + (2.0 ** -7 * loose if loose is not None else 0)).t() @ v.abs()
    for n, t in (("dwg", dwg), ("dwu", dwu), ("dwd", dwd)):
        allowed = (2.0 ** -7 + (T + 8) * 2.0 ** -24) * mag[n] + 2.0 ** -8 * ref[n].abs()
        assert bool(((t.double() - ref[n]).abs() <= allowed).all()), n
        # and far closer in the mean: errors of either sign over a million tokens
        assert float((t.double() - ref[n]).norm() / ref[n].norm()) < 2.0 ** -7, n


def test_another_current_device_is_not_touched():
    """The call runs on its tensors' device; tensors of two devices are refused (needs two GPUs to say more)."""
    import torch
    T, H, I = 4, 256, 128
    ws = F.get_ffn_workspace(T, H, I)
    c = {k: bf(v) for k, v in case(T, H, I).items()}
    before = torch.cuda.current_device()
    F.run_ffn_forward(ws, c["x"], (c["wg"], c["wu"], c["wd"]))
    assert torch.cuda.current_device() == before
    with pytest.raises(mok.MokError):
        mok.ffn_forward(ws.problem, c["x"], (c["wg"], c["wu"], c["wd"]), torch.empty_like(c["x"]),
                        ws.workspace.cpu())


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gates_far_out(kind):
    """Saved pre-activations up to bf16's largest: from |a| = 200 on both gates are a or 0 in fp32 and their
    derivatives 1 or 0. Identities for x, w_gate and w_down and powers of two elsewhere make dx, dw_gate and dw_up
    one product each without a rounding; dw_down, a sum of up to 64 terms of up to 0.5 * 0.5 * 3.3e38 and none
    below 0, may pass the largest number, and is no NaN."""
    import torch
    n = 64
    g = torch.Generator(device="cuda").manual_seed(11)
    eye = torch.eye(n, device="cuda").bfloat16()
    zero = torch.zeros_like(eye)
    dy = torch.exp2(-torch.randint(1, 5, (n, n), generator=g, device="cuda").float()).bfloat16()
    far = torch.tensor([200.0, 1e3, 1e10, 1.8e19, 2e19, 4e19, 6e19, 1e25, 1e38, 3.3e38], device="cuda").bfloat16()
    far = torch.cat([far, -far])
    a = far[torch.randint(0, far.numel(), (n, n), generator=g, device="cuda")]
    b = torch.full_like(a, 0.5)
    ws = F.get_ffn_workspace(n, n, n, activation=ACT[kind])
    ws.ctx = torch.cat([a, b], 1)
    dx, dwg, dwu, dwd = F.run_ffn_backward(ws, eye, (eye, zero, eye), dy)
    torch.cuda.synchronize()
    on = a > 0
    assert torch.equal(dwg.t(), torch.where(on, dy * b, zero)) and torch.equal(dx, torch.where(on, dy * b, zero))
    assert torch.equal(dwu.t(), torch.where(on, dy * a, zero))
    assert not dwd.isnan().any()


@pytest.mark.parametrize("T,H,I", [(3, 256, 128), (200, 256, 128), (4100, 2048, 768)])
def test_residual_beside_y(T, H, I):
    """The residual in the same rows as y, or right behind it, is no overlap: the bits of separate buffers. A
    window that shares columns with y is refused."""
    import torch
    c = {k: bf(v) for k, v in case(T, H, I, 6).items()}
    w = (c["wg"], c["wu"], c["wd"])
    ws = F.get_ffn_workspace(T, H, I, training=False)
    want = F.run_ffn_forward(ws, c["x"], w, residual=c["res"])
    wide = torch.zeros((T, 2 * H), dtype=torch.bfloat16, device="cuda")
    flat = torch.zeros((2 * T, H), dtype=torch.bfloat16, device="cuda")
    for y, res in ((wide[:, :H], wide[:, H:]), (wide[:, H:], wide[:, :H]), (flat[:T], flat[T:]), (flat[T:], flat[:T])):
        res.copy_(c["res"])
        F.run_ffn_forward(ws, c["x"], w, residual=res, y=y)
        assert torch.equal(y, want) and torch.equal(res, c["res"])
    with pytest.raises(mok.MokError) as e:
        F.run_ffn_forward(ws, c["x"], w, residual=wide[:, 8:H + 8], y=wide[:, :H])
    assert e.value.status == mok.MOK_ERR_INVALID_ARG


@pytest.mark.parametrize("T,H,I", [(1, 4096, 1536), (40, 2048, 768), (300, 2048, 768), (4100, 520, 2056)])
def test_workspace_of_forwards_alone(T, H, I):
    """The smaller workspace gives the bits of the full one, and nothing behind it is written; with ctx too."""
    import torch
    c = {k: bf(v) for k, v in case(T, H, I, 7).items()}
    w = (c["wg"], c["wu"], c["wd"])
    full = F.get_ffn_workspace(T, H, I)
    want = F.run_ffn_forward(full, c["x"], w, residual=c["res"])
    p = F.get_ffn_workspace(T, H, I, training=False).problem
    n, nctx = mok.ffn_buffer_sizes(p)
    assert n < full.workspace.numel() and nctx == full.ctx.nbytes
    mem = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for ctx in (None, torch.zeros_like(full.ctx)):
        y = torch.empty_like(want)
        mok.ffn_forward(p, c["x"], w, y, mem[:n], residual=c["res"], ctx=ctx)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and bool((mem[n:] == 0x5A).all())
    assert torch.equal(ctx, full.ctx)
    with pytest.raises(mok.MokError) as e:
        F.run_ffn_backward(F.FfnWorkspace(p, full.workspace, full.ctx), c["x"], w, c["dy"])
    assert e.value.status == mok.MOK_ERR_INVALID_ARG
