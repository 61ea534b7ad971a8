"""Binding of the training operators: products grouped by expert with both
gradients, SwiGLU with its gradient, and the AdamW step (include/moe.h).

Shapes, strides and types come from the tensors. Row-wise tensors may be
views with a row stride (columns of a wider buffer); everything else is
contiguous. A call runs on the device of its tensors and, without `stream`,
on that device's current stream; it raises ValueError for tensors it cannot
describe and MoEError for what the library refuses.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import MoEError, lib

MOE_T_BF16, MOE_T_F32 = 0, 1
MOE_STATE_F32, MOE_STATE_8BIT = 0, 1
MOE_STATE_BLOCK = 256  # elements that share a scale of an 8-bit state
CTRL_BYTES = 256       # start of a grouped-product workspace that must be zeroed once

_TYPES = {torch.bfloat16: MOE_T_BF16, torch.float32: MOE_T_F32}
_STATES = {torch.float32: MOE_STATE_F32, torch.float8_e4m3fn: MOE_STATE_8BIT}


class moe_linear_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("E", "R", "N", "K", "ld_x", "ld_y", "out_type", "accumulate")]


class moe_swiglu_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "I", "ld_g", "ld_h", "ld_dg")] + \
        [("limit", ctypes.c_float)]


class moe_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "master", "g", "m", "v", "m_scale", "v_scale")] + \
        [("n", ctypes.c_int64), ("p_type", ctypes.c_int32), ("g_type", ctypes.c_int32),
         ("state_type", ctypes.c_int32), ("wd_scale", ctypes.c_float)]


class moe_adamw_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + \
        [("step", ctypes.c_int64), ("dyn", ctypes.c_void_p)]


def declare(L) -> None:
    """Argument types of the training calls of a loaded library."""
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lp, sp = ctypes.POINTER(moe_linear_desc), ctypes.POINTER(moe_swiglu_desc)
    L.moe_linear_workspace_size.argtypes = [lp]
    L.moe_linear_workspace_size.restype = sz
    for f in ("moe_grouped_linear", "moe_grouped_linear_dgrad", "moe_grouped_linear_wgrad"):
        getattr(L, f).argtypes = [lp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_linear_read_error.argtypes = [vp, sz, vp, ctypes.POINTER(i32)]
    L.moe_swiglu.argtypes = [sp, vp, vp, vp, vp, i32, vp, vp, vp]
    L.moe_swiglu_backward.argtypes = [sp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp]
    L.moe_adamw_step.argtypes = [ctypes.POINTER(moe_adamw_cfg), ctypes.POINTER(moe_adamw_tensor), i32, vp]
    for f in ("moe_grouped_linear", "moe_grouped_linear_dgrad", "moe_grouped_linear_wgrad",
              "moe_linear_read_error", "moe_swiglu", "moe_swiglu_backward", "moe_adamw_step"):
        getattr(L, f).restype = i32


def _rows(t: torch.Tensor, name: str, dtype=torch.bfloat16):
    """(rows, width, row stride) of a row-wise tensor."""
    if t.dtype is not dtype or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-d {dtype} tensor")
    n, w = t.shape
    ld, one = t.stride()
    if n <= 1:
        ld = w  # the stride of a single row says nothing
    if one != 1 and w > 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if (n | w | ld) >> 31:  # ctypes would cut them to 32 bits without a word
        raise ValueError(f"{name}: rows, width and row stride must fit in 31 bits")
    return n, w, ld


def _flat(t: Optional[torch.Tensor], name: str, dtype, n: Optional[int] = None, at_least: bool = False):
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor")
    if n is not None and (t.numel() < n if at_least else t.numel() != n):
        raise ValueError(f"{name}: has {t.numel()} elements, {n} are wanted")
    return t.data_ptr()


def _current_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# the same handle without building a Stream object at every call, where torch has it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


# the current device's index, without torch.cuda's initialisation check (the tensors exist)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, where: str, tensors, stream, *args) -> None:
    """fn(*args, stream) on the tensors' device; None among them is skipped."""
    dev = tensors[0].get_device()
    if dev < 0:
        raise ValueError("expected a CUDA tensor")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("expected CUDA tensors of one device")
    if stream is None:
        s = _current_stream(dev)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev != _current_device():
        with torch.cuda.device(dev):
            st = fn(*args, s)
    else:
        st = fn(*args, s)
    if st != 0:
        raise MoEError(st, where)


# ------------------------------------------------------------------ grouped products
def linear_workspace_size(E: int, R: int, N: int, K: int) -> int:
    if (E | R | N | K) >> 31:  # negative ones, too
        raise MoEError(-1, "moe_linear_workspace_size")
    d = moe_linear_desc(E, R, N, K, K, N, MOE_T_BF16, 0)
    n = lib().moe_linear_workspace_size(ctypes.byref(d))
    if n == 0:
        raise MoEError(-1, "moe_linear_workspace_size")
    return int(n)


def alloc_linear_workspace(E: int, R: int, N: int, K: int, device=None) -> torch.Tensor:
    """Workspace of the three grouped products of this shape, its error word clear."""
    ws = torch.empty(linear_workspace_size(E, R, N, K), dtype=torch.uint8, device=device or "cuda")
    ws[:CTRL_BYTES].zero_()
    return ws


def _offsets(offsets: torch.Tensor) -> int:
    E = offsets.numel() - 1
    if offsets.dim() != 1 or E < 1 or E >> 31:
        raise ValueError("offsets: expected E + 1 entries")
    _flat(offsets, "offsets", torch.int32)
    return E


def _weights(W: torch.Tensor, name: str, E: int, types):
    if W.dim() != 3 or W.dtype not in types or not W.is_contiguous() or W.shape[0] != E:
        raise ValueError(f"{name}: expected a contiguous [E, N, K] tensor of {' or '.join(map(str, types))}")
    return W.shape[1], W.shape[2]


def _out_type(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _TYPES:
        raise ValueError(f"{name}: expected bfloat16 or float32")
    return _TYPES[t.dtype]


def moe_grouped_linear(x, offsets, W, y, ws, accumulate: bool = False, stream=None) -> None:
    """y[r] (+)= x[r] @ W[e].T for the rows offsets[e] <= r < offsets[e+1].
    x [R, K] and W [E, N, K] bf16, offsets [E+1] int32, y [R, N] bf16 or fp32
    (accumulate: fp32 only)."""
    E = _offsets(offsets)
    R, K, ld_x = _rows(x, "x")
    N, wk = _weights(W, "W", E, (torch.bfloat16,))
    out = _out_type(y, "y")
    yr, yn, ld_y = _rows(y, "y", y.dtype)
    if wk != K or yn != N or yr != R:
        raise ValueError(f"shapes do not fit: x {tuple(x.shape)}, W {tuple(W.shape)}, y {tuple(y.shape)}")
    d = moe_linear_desc(E, R, N, K, ld_x, ld_y, out, int(accumulate))
    _call(lib().moe_grouped_linear, "moe_grouped_linear", (x, offsets, W, y, ws), stream, ctypes.byref(d),
          x.data_ptr(), offsets.data_ptr(), W.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel())


def moe_grouped_linear_dgrad(dy, offsets, W, dx, ws, accumulate: bool = False, stream=None) -> None:
    """dx[r] (+)= dy[r] @ W[e]: the gradient of moe_grouped_linear's x.
    dy [R, N] bf16, dx [R, K] bf16 or fp32 (accumulate: fp32 only)."""
    E = _offsets(offsets)
    R, N, ld_y = _rows(dy, "dy")
    wn, K = _weights(W, "W", E, (torch.bfloat16,))
    out = _out_type(dx, "dx")
    xr, xk, ld_x = _rows(dx, "dx", dx.dtype)
    if wn != N or xk != K or xr != R:
        raise ValueError(f"shapes do not fit: dy {tuple(dy.shape)}, W {tuple(W.shape)}, dx {tuple(dx.shape)}")
    d = moe_linear_desc(E, R, N, K, ld_x, ld_y, out, int(accumulate))
    _call(lib().moe_grouped_linear_dgrad, "moe_grouped_linear_dgrad", (dy, offsets, W, dx, ws), stream,
          ctypes.byref(d), dy.data_ptr(), offsets.data_ptr(), W.data_ptr(), dx.data_ptr(), ws.data_ptr(),
          ws.numel())


def moe_grouped_linear_wgrad(dy, x, offsets, dW, ws, accumulate: bool = False, stream=None) -> None:
    """dW[e] (+)= dy[rows of e].T @ x[rows of e]: the gradient of
    moe_grouped_linear's W. dW [E, N, K] bf16 or fp32 (accumulate: fp32
    only); an expert without rows gets zeros."""
    E = _offsets(offsets)
    R, N, ld_y = _rows(dy, "dy")
    xr, K, ld_x = _rows(x, "x")
    out = _out_type(dW, "dW")
    if _weights(dW, "dW", E, (dW.dtype,)) != (N, K) or xr != R:
        raise ValueError(f"shapes do not fit: dy {tuple(dy.shape)}, x {tuple(x.shape)}, dW {tuple(dW.shape)}")
    d = moe_linear_desc(E, R, N, K, ld_x, ld_y, out, int(accumulate))
    _call(lib().moe_grouped_linear_wgrad, "moe_grouped_linear_wgrad", (dy, x, offsets, dW, ws), stream,
          ctypes.byref(d), dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), dW.data_ptr(), ws.data_ptr(),
          ws.numel())


def moe_linear_read_error(ws, stream=None) -> int:
    """Reads (synchronously) and clears the error word of a grouped-product
    workspace; see DEVERR for the codes."""
    code = ctypes.c_int32(0)
    L = lib()
    _call(lambda p, n, s: L.moe_linear_read_error(p, n, s, ctypes.byref(code)), "moe_linear_read_error",
          (ws,), stream, ws.data_ptr(), ws.numel())
    return int(code.value)


# ------------------------------------------------------------------ SwiGLU
def _like(t, name: str, shape, stride) -> int:
    """The row stride of t, which must have g's shape and type."""
    if t.dtype is torch.bfloat16 and t.shape == shape:
        if t.stride() == stride:
            return stride[0] if shape[0] > 1 else shape[1]
        return _rows(t, name)[2]
    _rows(t, name)
    raise ValueError(f"{name}: expected the shape of g, {tuple(shape)}")


def _swiglu_desc(g, u, h, limit: float, h_name: str, dg=None, du=None):
    R, I, ld_g = _rows(g, "g")
    shape, stride = g.shape, g.stride()
    if _like(u, "u", shape, stride) != ld_g:
        raise ValueError("g and u must have one row stride")
    ld_h, ld_dg = _like(h, h_name, shape, stride), ld_g
    if dg is not None:
        ld_dg = _like(dg, "dg", shape, stride)
        if _like(du, "du", shape, stride) != ld_dg:
            raise ValueError("dg and du must have one row stride")
    return moe_swiglu_desc(R, I, ld_g, ld_h, ld_dg, limit)


def _weight_args(d, w, perm, rows):
    rp = None if rows is None else _flat(rows, "rows", torch.int32, 1, True)
    if w is None:
        if perm is not None:
            raise ValueError("perm without w")
        return None, None, 0, rp
    if perm is None:
        return _flat(w, "w", torch.float32, d.R, True), None, 0, rp
    if w.numel() >> 31:
        raise ValueError("w: its size must fit in 31 bits")
    return _flat(w, "w", torch.float32), _flat(perm, "perm", torch.int32, d.R, True), w.numel(), rp


def moe_swiglu(g, u, h, limit: float = 0.0, w=None, perm=None, rows=None, stream=None) -> None:
    """h = w * silu(clamp(g)) * clamp(u), rows of bf16. The weight of row r is
    w[perm[r]] (w[r] without perm, 1 without w); rows: a device int32, the
    number of rows that count (for example offsets[E:])."""
    d = _swiglu_desc(g, u, h, limit, "h")
    wp, pp, n_w, rp = _weight_args(d, w, perm, rows)
    _call(lib().moe_swiglu, "moe_swiglu", (g, u, h, w, perm, rows), stream, ctypes.byref(d), g.data_ptr(),
          u.data_ptr(), wp, pp, n_w, rp, h.data_ptr())


def moe_swiglu_backward(dh, g, u, dg, du, limit: float = 0.0, w=None, perm=None, dw=None, rows=None,
                        stream=None) -> None:
    """Gradients of moe_swiglu: dg and du (bf16, they may be g and u) and,
    with w, dw (fp32, laid out like w; optional)."""
    d = _swiglu_desc(g, u, dh, limit, "dh", dg, du)
    wp, pp, n_w, rp = _weight_args(d, w, perm, rows)
    if dw is not None and (w is None or dw.numel() != w.numel()):
        raise ValueError("dw: needs w and its size")
    _call(lib().moe_swiglu_backward, "moe_swiglu_backward", (dh, g, u, dg, du, w, perm, rows, dw), stream,
          ctypes.byref(d), dh.data_ptr(), g.data_ptr(), u.data_ptr(), wp, pp, n_w, rp, dg.data_ptr(),
          du.data_ptr(), _flat(dw, "dw", torch.float32))


# ------------------------------------------------------------------ AdamW
class AdamWTensors:
    """The C array of a step's tensors, and the tensors themselves, kept alive."""

    def __init__(self, array, n: int, keep):
        self.array, self.n, self.keep = array, n, keep


def make_adamw_tensors(tensors: Sequence[dict]) -> AdamWTensors:
    """The tensors of moe_adamw_step, once for many steps. Each is a dict of
    p (bf16 or fp32, contiguous), g (bf16 or fp32), m and v (both fp32, or
    both float8_e4m3fn with m_scale and v_scale, one fp32 per MOE_STATE_BLOCK
    elements), optionally master (fp32, with a bf16 p) and wd_scale."""
    out, keep, dev = (moe_adamw_tensor * max(1, len(tensors)))(), [], None
    f32 = torch.float32
    for o, t in zip(out, tensors):
        p, g, m, v = t["p"], t["g"], t["m"], t["v"]
        master, ms, vs = t.get("master"), t.get("m_scale"), t.get("v_scale")
        n, state = p.numel(), m.dtype
        if state not in _STATES or v.dtype is not state:
            raise ValueError("m and v: expected both float32 or both float8_e4m3fn")
        q8 = state is not f32
        if q8 != (ms is not None) or q8 != (vs is not None):
            raise ValueError("8-bit states, and only they, have m_scale and v_scale")
        o.p, o.g = _flat(p, "p", p.dtype), _flat(g, "g", g.dtype, n)
        o.m, o.v = _flat(m, "m", state, n), _flat(v, "v", state, n)
        o.n, o.state_type, o.wd_scale = n, _STATES[state], t.get("wd_scale", 1.0)
        o.p_type, o.g_type = _out_type(p, "p"), _out_type(g, "g")
        mine = [p, g, m, v]
        if master is not None:
            o.master = _flat(master, "master", f32, n)
            mine.append(master)
        if q8:
            blocks = -(-n // MOE_STATE_BLOCK)
            o.m_scale = _flat(ms, "m_scale", f32, blocks)
            o.v_scale = _flat(vs, "v_scale", f32, blocks)
            mine += (ms, vs)
        for x in mine:
            d = x.get_device()
            if d < 0 or (dev is not None and d != dev):
                raise ValueError("expected CUDA tensors of one device")
            dev = d
        keep += mine
    return AdamWTensors(out, len(tensors), keep)


def adamw_dyn(lr: float, beta1: float, beta2: float, step: int, grad_scale: float = 1.0) -> list:
    """The four values of moe_adamw_step's `dyn` tensor for a step."""
    return [lr, 1.0 - beta1 ** step, (1.0 - beta2 ** step) ** 0.5, grad_scale]


def moe_adamw_step(tensors: AdamWTensors, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, weight_decay: float = 0.0, step: int = 1, grad_scale: float = 1.0,
                   dyn: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step over every tensor of `tensors` (make_adamw_tensors).
    dyn: a device float32 [4] (adamw_dyn) that replaces lr, step and
    grad_scale, read when the step runs: for captured graphs."""
    if tensors.n == 0:
        return
    c = moe_adamw_cfg(lr, beta1, beta2, eps, weight_decay, grad_scale, step,
                      _flat(dyn, "dyn", torch.float32, 4))
    _call(lib().moe_adamw_step, "moe_adamw_step", (tensors.keep[0], dyn), stream, ctypes.byref(c),
          tensors.array, tensors.n)
