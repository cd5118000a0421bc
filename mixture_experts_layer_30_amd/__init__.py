"""Python binding of libmok, a deterministic MoE layer for AMD MI355X (gfx950).

The binding only marshals arguments: every step of the layer runs in the HIP
kernels of libmok.so (see include/mok.h for the contract of each call). PyTorch
supplies device memory and the current stream. There is no fallback: if the
library is missing or fails to load, importing the calls raises.
"""
from __future__ import annotations

import ctypes
import os

__version__ = "0.1.0"

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmok.so")

MOK_OK = 0
MOK_ERR_INVALID_ARG = -1
MOK_ERR_UNSUPPORTED = -2
MOK_ERR_BUFFER_TOO_SMALL = -3
MOK_ERR_DEVICE = -4
MOK_BF16 = 0
MOK_MXFP8 = 1
MOK_MXFP4 = 2
ACT_SILU = 0
ACT_GELU_TANH = 1
STATUS_BAD_EXPERT_ID = 0x1
STATUS_WATCHDOG = 0x2


class MokError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Config(ctypes.Structure):
    _fields_ = [("minibatch_rows", ctypes.c_int32), ("ring_slots", ctypes.c_int32),
                ("capacity_multiplier", ctypes.c_float), ("num_cus", ctypes.c_int32),
                ("driver", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_gate", ctypes.c_void_p),
                ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("w_down_t", ctypes.c_void_p), ("w_gu_t", ctypes.c_void_p),
                ("s_down_t", ctypes.c_void_p), ("s_gu_t", ctypes.c_void_p)]


class ScheduleLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "status", "counts", "offsets", "perm", "dest", "n_fwd_tiles", "fwd_tiles",
        "mb_tile_start", "n_bwd_tiles", "bwd_tiles", "total")] + [
        (n, ctypes.c_int32) for n in (
            "minibatch_rows", "ring_slots", "n_minibatches", "max_fwd_tiles", "max_bwd_tiles",
            "fwd_tile_rows", "bwd_tile_rows")] + [("arrays", ctypes.c_size_t), ("expert_order", ctypes.c_size_t)]


class MxProblem(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("ld_d", ctypes.c_int64),
                ("a_dtype", ctypes.c_int32)]


class FfnProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64),
                ("forward_only", ctypes.c_int32)]


_lib = None

EXPORTS = ("mok_version", "mok_status_string", "mok_buffer_sizes", "mok_get_schedule_layout",
           "mok_build_schedule", "mok_forward", "mok_backward", "mok_mxfp8_quantize",
           "mok_router_forward", "mok_router_backward", "mok_trace_enable", "mok_trace_collect",
           "mok_mxfp8_quantize_transposed", "mok_probe_mfma", "mok_build_schedule_noalloc",
           "mok_forward_fused", "mok_mxfp4_quantize", "mok_mxfp4_dequantize", "mok_mx_matmul_workspace",
           "mok_mx_matmul", "mok_ffn_buffer_sizes", "mok_ffn_forward", "mok_ffn_backward")


class TraceStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_int32),
                ("total_ms", ctypes.c_double), ("max_ms", ctypes.c_double)]


def lib():
    """The loaded libmok.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libmok.so not found at {LIB_PATH}; build it with "
                              "`python -m mixture_experts_layer_30_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        L.mok_version.restype = ctypes.c_int32
        L.mok_version.argtypes = []
        L.mok_status_string.restype = ctypes.c_char_p
        L.mok_status_string.argtypes = [ctypes.c_int32]
        L.mok_buffer_sizes.restype = ctypes.c_int
        L.mok_buffer_sizes.argtypes = [P(Problem), P(Config), P(sz), P(sz), P(sz)]
        L.mok_get_schedule_layout.restype = ctypes.c_int
        L.mok_get_schedule_layout.argtypes = [P(Problem), P(Config), P(ScheduleLayout)]
        L.mok_build_schedule.restype = ctypes.c_int
        L.mok_build_schedule.argtypes = [P(Problem), P(Config), vp, vp, sz, vp]
        L.mok_build_schedule_noalloc.restype = ctypes.c_int
        L.mok_build_schedule_noalloc.argtypes = [P(Problem), P(Config), vp, vp, sz, vp]
        L.mok_forward.restype = ctypes.c_int
        L.mok_forward.argtypes = [P(Problem), P(Config), vp, vp, vp, P(Weights), vp, vp, vp, sz, vp]
        L.mok_forward_fused.restype = ctypes.c_int
        L.mok_forward_fused.argtypes = [P(Problem), P(Config), vp, vp, sz, vp, vp, P(Weights), vp, vp,
                                        vp, sz, vp]
        L.mok_backward.restype = ctypes.c_int
        L.mok_backward.argtypes = [P(Problem), P(Config), vp, vp, vp, vp, P(Weights), vp, vp,
                                   vp, vp, vp, vp, vp, sz, vp]
        L.mok_mxfp8_quantize.restype = ctypes.c_int
        L.mok_mxfp8_quantize.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, vp, vp, vp]
        L.mok_mxfp8_quantize_transposed.restype = ctypes.c_int
        L.mok_mxfp8_quantize_transposed.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, vp, vp,
                                                     ctypes.c_int64, ctypes.c_int64, vp]
        L.mok_probe_mfma.restype = ctypes.c_int
        L.mok_probe_mfma.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp]
        L.mok_router_forward.restype = ctypes.c_int
        L.mok_router_forward.argtypes = [P(Problem), vp, vp, vp, vp, vp, vp]
        L.mok_router_backward.restype = ctypes.c_int
        L.mok_router_backward.argtypes = [P(Problem), P(Config), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.mok_trace_enable.restype = ctypes.c_int
        L.mok_trace_enable.argtypes = [ctypes.c_int32]
        L.mok_trace_collect.restype = ctypes.c_int
        L.mok_trace_collect.argtypes = [P(TraceStat), ctypes.c_int32, P(ctypes.c_int32)]
        for name in ("mok_mxfp4_quantize", "mok_mxfp4_dequantize"):
            getattr(L, name).restype = ctypes.c_int
        L.mok_mxfp4_quantize.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, vp, vp, vp]
        L.mok_mxfp4_dequantize.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_int64, vp, vp]
        L.mok_mx_matmul_workspace.restype = ctypes.c_int
        L.mok_mx_matmul_workspace.argtypes = [P(MxProblem), P(sz)]
        L.mok_mx_matmul.restype = ctypes.c_int
        L.mok_mx_matmul.argtypes = [P(MxProblem), vp, vp, vp, vp, vp, vp, sz, vp]
        L.mok_ffn_buffer_sizes.restype = ctypes.c_int
        L.mok_ffn_buffer_sizes.argtypes = [P(FfnProblem), P(sz), P(sz)]
        L.mok_ffn_forward.restype = ctypes.c_int
        L.mok_ffn_forward.argtypes = [P(FfnProblem), vp, P(Weights), vp, vp, vp, vp, sz, vp]
        L.mok_ffn_backward.restype = ctypes.c_int
        L.mok_ffn_backward.argtypes = [P(FfnProblem), vp, vp, P(Weights), vp, vp, vp, vp, vp, vp, sz, vp]
        _lib = L
    return _lib


def version() -> int:
    return int(lib().mok_version())


def status_string(status: int) -> str:
    return lib().mok_status_string(int(status)).decode()


def _check(status, what):
    if status != MOK_OK:
        raise MokError(status, what)


def make_problem(T, H, I, E, topk, dtype=MOK_BF16) -> Problem:
    return Problem(int(T), int(H), int(I), int(E), int(topk), int(dtype))


def make_config(minibatch_rows=0, ring_slots=0, capacity_multiplier=0.0, num_cus=0, driver=0):
    return Config(int(minibatch_rows), int(ring_slots), float(capacity_multiplier), int(num_cus),
                  int(driver))


def _cfg(config):
    return ctypes.byref(config) if config is not None else None


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def buffer_sizes(problem, config=None):
    """(workspace_bytes, schedule_bytes, fwd_ctx_bytes); host only."""
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().mok_buffer_sizes(ctypes.byref(problem), _cfg(config), ctypes.byref(a),
                                  ctypes.byref(b), ctypes.byref(c)), "mok_buffer_sizes")
    return a.value, b.value, c.value


def schedule_layout(problem, config=None) -> ScheduleLayout:
    out = ScheduleLayout()
    _check(lib().mok_get_schedule_layout(ctypes.byref(problem), _cfg(config), ctypes.byref(out)),
           "mok_get_schedule_layout")
    return out


def build_schedule(problem, topk_ids, schedule, config=None, stream=None):
    _check(lib().mok_build_schedule(ctypes.byref(problem), _cfg(config), _ptr(topk_ids),
                                    _ptr(schedule), schedule.numel() * schedule.element_size(),
                                    _stream(stream)), "mok_build_schedule")


def build_schedule_noalloc(problem, topk_ids, schedule, config=None, stream=None):
    """mok_build_schedule with the build's scratch in the library's static
    device array (schedule needs only schedule_layout(...).arrays bytes)."""
    _check(lib().mok_build_schedule_noalloc(ctypes.byref(problem), _cfg(config), _ptr(topk_ids),
                                            _ptr(schedule), schedule.numel() * schedule.element_size(),
                                            _stream(stream)), "mok_build_schedule_noalloc")


def _weights(w_gate, w_up, w_down, s_gate=None, s_up=None, s_down=None, w_down_t=None, w_gu_t=None,
             s_down_t=None, s_gu_t=None):
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return Weights(w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), p(s_gate), p(s_up), p(s_down),
                   p(w_down_t), p(w_gu_t), p(s_down_t), p(s_gu_t))


def forward(problem, schedule, x, topk_w, weights, y, workspace, fwd_ctx=None, config=None,
            stream=None):
    """weights: (w_gate, w_up, w_down[, s_gate, s_up, s_down[, w_down_t, w_gu_t, s_down_t,
    s_gu_t]]) tensors (the last four only matter to the MXFP8 backward)."""
    w = _weights(*weights)
    _check(lib().mok_forward(ctypes.byref(problem), _cfg(config), _ptr(schedule), _ptr(x),
                             _ptr(topk_w), ctypes.byref(w), _ptr(y), _ptr(fwd_ctx),
                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(stream)), "mok_forward")


def forward_fused(problem, topk_ids, schedule, x, topk_w, weights, y, workspace, fwd_ctx=None,
                  config=None, stream=None):
    """mok_forward_fused: the schedule from topk_ids and the forward, in one
    persistent launch (weights as for forward)."""
    w = _weights(*weights)
    _check(lib().mok_forward_fused(ctypes.byref(problem), _cfg(config), _ptr(topk_ids), _ptr(schedule),
                                   schedule.numel() * schedule.element_size(), _ptr(x), _ptr(topk_w),
                                   ctypes.byref(w), _ptr(y), _ptr(fwd_ctx), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "mok_forward_fused")


def backward(problem, schedule, fwd_ctx, x, topk_w, weights, dy, dx, dw_gate, dw_up, dw_down,
             d_topk_w, workspace, config=None, stream=None):
    w = _weights(*weights)
    _check(lib().mok_backward(ctypes.byref(problem), _cfg(config), _ptr(schedule), _ptr(fwd_ctx),
                              _ptr(x), _ptr(topk_w), ctypes.byref(w), _ptr(dy), _ptr(dx),
                              _ptr(dw_gate), _ptr(dw_up), _ptr(dw_down), _ptr(d_topk_w),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream)), "mok_backward")


def mxfp8_quantize(src, q, scales, stream=None):
    """src [rows][K] bf16 -> q [rows][K] uint8 (E4M3), scales [rows][K/32] uint8 (E8M0)."""
    rows, K = src.shape[0], src.shape[-1]
    _check(lib().mok_mxfp8_quantize(_ptr(src), int(rows) if src.dim() == 2 else int(src.numel() // K),
                                    int(K), _ptr(q), _ptr(scales), _stream(stream)),
           "mok_mxfp8_quantize")


def mxfp8_quantize_transposed(src, q, scales, col0=0, stream=None):
    """src [batch][rows][cols] (or [rows][cols]) bf16 -> q[b][c][col0 + r] (E4M3) and
    scales[b][c][(col0 + r) / 32] (E8M0), blocked by 32 along the source rows; q is
    [batch][cols][ld] uint8 and scales [batch][cols][ld/32] uint8 (ld = q.shape[-1])."""
    rows, cols, ld = src.shape[-2], src.shape[-1], q.shape[-1]
    batch = int(src.numel() // (rows * cols)) if rows * cols else 0
    _check(lib().mok_mxfp8_quantize_transposed(_ptr(src), batch, int(rows), int(cols), _ptr(q), _ptr(scales),
                                               int(ld), int(col0), _stream(stream)),
           "mok_mxfp8_quantize_transposed")


def probe_mfma(kind, workgroups, iters, sink, stream=None):
    """Enqueue the matrix-core peak probe (kind 0 bf16, 1 MXFP8); sink holds
    workgroups * 256 float32. Returns the FLOPs it performs."""
    _check(lib().mok_probe_mfma(int(kind), int(workgroups), int(iters), _ptr(sink), _stream(stream)),
           "mok_probe_mfma")
    return float(workgroups) * 4 * 8 * iters * (32768 if kind == 0 else 131072)


def router_forward(problem, x, w_router, bias, topk_ids, topk_w, stream=None):
    """x [T][H] bf16, w_router [E][H] fp32, bias [E] fp32 or None -> topk_ids [T][k] int32,
    topk_w [T][k] fp32 (overwritten)."""
    _check(lib().mok_router_forward(ctypes.byref(problem), _ptr(x), _ptr(w_router), _ptr(bias),
                                    _ptr(topk_ids), _ptr(topk_w), _stream(stream)), "mok_router_forward")


def router_backward(problem, schedule, x, w_router, topk_ids, topk_w, d_topk_w, d_sel, dx, d_w_router,
                    config=None, stream=None):
    """-> d_sel [T][k] fp32, dx [T][H] bf16, d_w_router [E][H] fp32 (overwritten); schedule built
    by build_schedule for these topk_ids."""
    _check(lib().mok_router_backward(ctypes.byref(problem), _cfg(config), _ptr(schedule), _ptr(x),
                                     _ptr(w_router), _ptr(topk_ids), _ptr(topk_w), _ptr(d_topk_w),
                                     _ptr(d_sel), _ptr(dx), _ptr(d_w_router), _stream(stream)),
           "mok_router_backward")


# ---------------------------------------------------------------- MXFP4 and the dense block
# These calls check their tensors (device, type, shape, row layout) and run on
# the tensors' device: with the caller's stream, or that device's current one.

_torch = None


def _device_of(t):
    """The index of t's GPU (-1: none), at which the call's other tensors have to be."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return t.get_device()


def _want(what, t, dtype, shape, index, rows=False):
    """t is a tensor of GPU `index` of this type and shape, contiguous (rows=True: with
    contiguous elements within a row, rows at any pitch)."""
    dtype = _torch.bfloat16 if dtype == "bf16" else _torch.uint8
    if t.dtype is dtype and t.shape == shape and t.get_device() == index != -1 and t.is_contiguous():
        return
    if not t.is_cuda or t.get_device() != index:
        raise MokError(MOK_ERR_INVALID_ARG, f"{what}: not on the call's GPU ({t.device})")
    if t.dtype is not dtype or t.shape != shape:
        raise MokError(MOK_ERR_INVALID_ARG, f"{what}: {t.dtype} {tuple(t.shape)}, wanted {dtype} {tuple(shape)}")
    if not (rows and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        raise MokError(MOK_ERR_INVALID_ARG, f"{what}: strides {t.stride()}")


def _pitch(t):
    """Row pitch of a [rows][cols] tensor in elements (0: contiguous)."""
    return 0 if t.is_contiguous() else t.stride(0)


def _scratch(workspace, index):
    """(pointer, bytes) of a workspace tensor or None."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise MokError(MOK_ERR_INVALID_ARG, f"workspace: not contiguous memory of GPU {index}")
    return workspace.data_ptr(), workspace.nbytes


def _run(what, index, stream, fn, *args):
    """fn(*args, stream) on GPU `index`: the caller's stream, or that device's current one."""
    # (the raw handles: torch.cuda.current_stream builds a Stream object, 3 us a call)
    st = _torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if index == _torch._C._cuda_getDevice():
        status = fn(*args, st)
    else:
        with _torch.cuda.device(index):
            status = fn(*args, st)
    if status != MOK_OK:
        raise MokError(status, what)


def _rows_K(src):
    K = src.shape[-1]
    return (src.numel() // K if K else 0), K


def mxfp4_quantize(src, q, scales, stream=None):
    """src [..., K] bf16 -> q [..., K/2] uint8 (two E2M1 codes a byte), scales [..., K/32] uint8 (E8M0)."""
    rows, K = _rows_K(src)
    dev = _device_of(src)
    _want("src", src, "bf16", src.shape, dev)
    _want("q", q, "u8", (*src.shape[:-1], K // 2), dev)
    _want("scales", scales, "u8", (*src.shape[:-1], K // 32), dev)
    _run("mok_mxfp4_quantize", dev, stream, lib().mok_mxfp4_quantize, src.data_ptr(), rows, K, q.data_ptr(),
         scales.data_ptr())


def mxfp4_dequantize(q, scales, dst, stream=None):
    """The bf16 values dst [..., K] of the codes q [..., K/2] and scales [..., K/32]."""
    rows, K = _rows_K(dst)
    dev = _device_of(dst)
    _want("dst", dst, "bf16", dst.shape, dev)
    _want("q", q, "u8", (*dst.shape[:-1], K // 2), dev)
    _want("scales", scales, "u8", (*dst.shape[:-1], K // 32), dev)
    _run("mok_mxfp4_dequantize", dev, stream, lib().mok_mxfp4_dequantize, q.data_ptr(), scales.data_ptr(), rows, K,
         dst.data_ptr())


def make_mx_problem(M, N, K, a_dtype, ld_d=0) -> MxProblem:
    return MxProblem(int(M), int(N), int(K), int(ld_d), int(a_dtype))


def mx_matmul_workspace(problem):
    """Workspace bytes of mx_matmul; host only."""
    n = ctypes.c_size_t()
    _check(lib().mok_mx_matmul_workspace(ctypes.byref(problem), ctypes.byref(n)), "mok_mx_matmul_workspace")
    return n.value


def mx_matmul(problem, a, a_scales, b, b_scales, d, workspace, stream=None):
    """d [M][N] bf16 = A . B^T: a [M][K] (MXFP8) or [M][K/2] (MXFP4) uint8, b [N][K/2] uint8, scales
    [rows][K/32] uint8. The row pitch of d is taken from the tensor (problem.ld_d is ignored)."""
    M, N, K = problem.M, problem.N, problem.K
    dev = _device_of(d)
    _want("d", d, "bf16", (M, N), dev, rows=True)
    _want("a", a, "u8", (M, K if problem.a_dtype == MOK_MXFP8 else K // 2), dev)
    _want("a_scales", a_scales, "u8", (M, K // 32), dev)
    _want("b", b, "u8", (N, K // 2), dev)
    _want("b_scales", b_scales, "u8", (N, K // 32), dev)
    p = MxProblem(M, N, K, _pitch(d), problem.a_dtype)
    _run("mok_mx_matmul", dev, stream, lib().mok_mx_matmul, ctypes.byref(p), a.data_ptr(), a_scales.data_ptr(),
         b.data_ptr(), b_scales.data_ptr(), d.data_ptr(), *_scratch(workspace, dev))


def make_ffn_problem(T, H, I, dtype=MOK_BF16, activation=ACT_SILU, ld_x=0, ld_y=0, forward_only=False) -> FfnProblem:
    """forward_only: for forwards alone, whose workspace is smaller; ffn_backward refuses such a problem."""
    return FfnProblem(int(T), int(H), int(I), int(dtype), int(activation), int(ld_x), int(ld_y), int(forward_only))


def ffn_buffer_sizes(problem):
    """(workspace_bytes, ctx_bytes); host only."""
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().mok_ffn_buffer_sizes(ctypes.byref(problem), ctypes.byref(a), ctypes.byref(b)),
           "mok_ffn_buffer_sizes")
    return a.value, b.value


def _ffn_weights(problem, weights, device):
    H, I = problem.H, problem.I
    mx = problem.dtype == MOK_MXFP4
    if len(weights) < (6 if mx else 3):
        raise MokError(MOK_ERR_INVALID_ARG, "weights: (w_gate, w_up, w_down[, s_gate, s_up, s_down])")
    t, div = ("u8", 2) if mx else ("bf16", 1)
    for n, w, shape in zip(("w_gate", "w_up", "w_down"), weights, ((I, H // div), (I, H // div), (H, I // div))):
        _want(n, w, t, shape, device)
    if mx:
        for n, w, shape in zip(("s_gate", "s_up", "s_down"), weights[3:], ((I, H // 32), (I, H // 32), (H, I // 32))):
            _want(n, w, "u8", shape, device)
    return _weights(*weights[:6 if mx else 3])


def _ffn_call(problem, ld_x, ld_y):
    return FfnProblem(problem.T, problem.H, problem.I, problem.dtype, problem.activation, ld_x, ld_y,
                      problem.forward_only)


def ffn_forward(problem, x, weights, y, workspace, residual=None, ctx=None, stream=None):
    """y [T][H] = block(x) (+ residual); ctx [T][2I] bf16 receives the pre-activations. x, and y with residual,
    may have any row pitch that is a multiple of 8 (taken from the tensors). weights: (w_gate, w_up, w_down)
    bf16, or MXFP4 codes with (s_gate, s_up, s_down)."""
    T, H = problem.T, problem.H
    dev = _device_of(x)
    _want("x", x, "bf16", (T, H), dev, rows=True)
    _want("y", y, "bf16", (T, H), dev, rows=True)
    if residual is not None:
        _want("residual", residual, "bf16", (T, H), dev, rows=True)
        if _pitch(residual) != _pitch(y):
            raise MokError(MOK_ERR_INVALID_ARG, "residual: another row pitch than y")
    if ctx is not None:
        _want("ctx", ctx, "bf16", (T, 2 * problem.I), dev)
    w = _ffn_weights(problem, weights, dev)
    p = _ffn_call(problem, _pitch(x), _pitch(y))
    _run("mok_ffn_forward", dev, stream, lib().mok_ffn_forward, ctypes.byref(p), x.data_ptr(), ctypes.byref(w),
         _ptr(residual), y.data_ptr(), _ptr(ctx), *_scratch(workspace, dev))


def ffn_backward(problem, ctx, x, weights, dy, dx, dw_gate, dw_up, dw_down, workspace, stream=None):
    """Gradients of <dy, y>; x and dx share one row pitch, dy may have another."""
    T, H, I = problem.T, problem.H, problem.I
    dev = _device_of(x)
    if ctx is None:
        raise MokError(MOK_ERR_INVALID_ARG, "ctx: no context was saved by a forward")
    _want("x", x, "bf16", (T, H), dev, rows=True)
    _want("dy", dy, "bf16", (T, H), dev, rows=True)
    _want("dx", dx, "bf16", (T, H), dev, rows=True)
    _want("ctx", ctx, "bf16", (T, 2 * I), dev)
    for n, t, shape in (("dw_gate", dw_gate, (I, H)), ("dw_up", dw_up, (I, H)), ("dw_down", dw_down, (H, I))):
        _want(n, t, "bf16", shape, dev)
    if _pitch(x) != _pitch(dx):
        raise MokError(MOK_ERR_INVALID_ARG, "dx: another row pitch than x")
    w = _ffn_weights(problem, weights, dev)
    p = _ffn_call(problem, _pitch(x), _pitch(dy))
    _run("mok_ffn_backward", dev, stream, lib().mok_ffn_backward, ctypes.byref(p), ctx.data_ptr(), x.data_ptr(),
         ctypes.byref(w), dy.data_ptr(), dx.data_ptr(), dw_gate.data_ptr(), dw_up.data_ptr(), dw_down.data_ptr(),
         *_scratch(workspace, dev))


def trace_enable(on=True):
    _check(lib().mok_trace_enable(1 if on else 0), "mok_trace_enable")


def trace_collect():
    """{kernel name: (launches, total_ms, max_ms)}; waits for the traced work."""
    n = ctypes.c_int32()
    buf = (TraceStat * 64)()
    _check(lib().mok_trace_collect(buf, 64, ctypes.byref(n)), "mok_trace_collect")
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms, buf[i].max_ms)
            for i in range(min(n.value, 64))}
