"""Binding of the operators around the layer (include/strata_ops.h).

Tensors are checked before a call (device, type, contiguity, element count)
and a mismatch raises StrataError with STRATA_EINVAL; everything else is
checked by the library.  A call runs on the current stream of its tensors'
device unless one is given, with that device current.  Raw device addresses
(ints) are passed on unchecked.
"""
from __future__ import annotations

import ctypes
from typing import Optional

try:
    import torch
except ImportError:  # pragma: no cover -- the rest of the package imports without it
    torch = None

POST_NORM, PRE_NORM, GATE_TOKEN, GATE_CHANNEL, GATE_SIGMOID = 1, 2, 4, 8, 16

_XTYPES = {0: torch.bfloat16, 1: torch.float32} if torch else {}   # X_BF16, X_F32
_EINVAL = 1

SYMBOLS = ("strata_moe_sort_workspace_bytes", "strata_moe_sort", "strata_moe_dispatch",
           "strata_moe_dispatch_backward", "strata_moe_combine", "strata_moe_combine_backward",
           "strata_moe_grouped_workspace_bytes", "strata_moe_grouped_product", "strata_moe_grouped_dgrad",
           "strata_moe_grouped_wgrad", "strata_block_norm", "strata_block_norm_backward_workspace_bytes",
           "strata_block_norm_backward")


class BlockNormArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("u_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("resid_scale", ctypes.c_float), ("branch_scale", ctypes.c_float), ("eps", ctypes.c_float)]


def declare(lib):
    """Signatures of the functions above on a loaded library."""
    vp, i32, sz, it = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
    norm = ctypes.POINTER(BlockNormArgs)
    for name, restype, argtypes in (
            ("strata_moe_sort_workspace_bytes", sz, [i32, i32, i32]),
            ("strata_moe_sort", it, [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            ("strata_moe_dispatch", it, [vp, it, i32, i32, i32, vp, vp, i32, vp]),
            ("strata_moe_dispatch_backward", it, [vp, it, i32, vp, i32, i32, i32, vp, vp]),
            ("strata_moe_combine", it, [vp, it, i32, vp, vp, i32, i32, i32, vp, vp, it, vp]),
            ("strata_moe_combine_backward", it, [vp, it, vp, it, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp]),
            ("strata_moe_grouped_workspace_bytes", sz, [i32, i32, i32, i32]),
            ("strata_moe_grouped_product", it, [vp, vp, vp, i32, i32, i32, i32, vp, it, vp, sz, vp]),
            ("strata_moe_grouped_dgrad", it, [vp, vp, vp, i32, i32, i32, i32, vp, it, vp, sz, vp]),
            ("strata_moe_grouped_wgrad", it, [vp, vp, vp, i32, i32, i32, i32, vp, it, vp, sz, vp]),
            ("strata_block_norm", it, [norm, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            ("strata_block_norm_backward_workspace_bytes", sz, [norm]),
            ("strata_block_norm_backward", it, [norm] + [vp] * 15 + [sz, vp])):
        f = getattr(lib, name)
        f.restype = restype
        f.argtypes = argtypes


def _bad(what: str):
    from . import StrataError
    raise StrataError(_EINVAL, what)


class _Call:
    """The tensors of one call: their addresses, checked to be on one device."""
    __slots__ = ("dev",)

    def __init__(self):
        self.dev = None

    def ptr(self, t, dtype, n: int, name: str) -> Optional[int]:
        """Address of a contiguous tensor of n elements (None and ints pass)."""
        if t is None or t.__class__ is int:
            return t
        dev = t.device
        if self.dev is None:
            if dev.type != "cuda":
                _bad(f"{name} is not in device memory")
            self.dev = dev
        elif dev != self.dev:
            _bad(f"{name} is on {dev}, not on {self.dev}")
        if t.dtype != dtype:
            _bad(f"{name} is {t.dtype}, not {dtype}")
        if t.numel() != n:
            _bad(f"{name} has {t.numel()} elements, not {n}")
        if not t.is_contiguous():
            _bad(f"{name} is not contiguous")
        return t.data_ptr()

    def ws(self, t, n: int) -> Optional[int]:
        """Address of a workspace said to hold n bytes."""
        if t is None or t.__class__ is int:
            return t
        if self.dev is not None and t.device != self.dev:
            _bad(f"the workspace is on {t.device}, not on {self.dev}")
        if t.numel() * t.element_size() < n or not t.is_contiguous():
            _bad("the workspace is smaller than ws_bytes")
        return t.data_ptr()

    def run(self, fn, *args, stream=None):
        """fn(*args, stream) with the tensors' device current."""
        if stream is not None and stream.__class__ is not int:
            stream = stream.cuda_stream
        dev = self.dev
        if dev is not None and dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                s = torch.cuda.current_stream().cuda_stream if stream is None else stream
                status = fn(*args, s)
        else:
            status = fn(*args, torch.cuda.current_stream().cuda_stream if stream is None else stream)
        if status:
            from . import _check
            _check(status)


def _lib():
    from . import load_library
    return load_library()


def _xtype(code: int, name: str):
    t = _XTYPES.get(code)
    if t is None:
        _bad(f"{name} is not X_BF16 or X_F32")
    return t


def sort_workspace_bytes(T: int, k: int, n_experts: int) -> int:
    n = _lib().strata_moe_sort_workspace_bytes(T, k, n_experts)
    if n == 0:
        _bad("unsupported sort")
    return n


def sort_picks(idx, T: int, k: int, n_experts: int, counts, offsets, perm, pos, ws, ws_bytes: int, stream=None):
    """Picks sorted by expert (see strata_moe_sort); any output may be None."""
    c, i32, n = _Call(), torch.int32, T * k
    c.run(_lib().strata_moe_sort, c.ptr(idx, i32, n, "idx"), T, k, n_experts,
          c.ptr(counts, i32, n_experts, "counts"), c.ptr(offsets, i32, n_experts + 1, "offsets"),
          c.ptr(perm, i32, n, "perm"), c.ptr(pos, i32, n, "pos"), c.ws(ws, ws_bytes), ws_bytes, stream=stream)


def dispatch(x, xdtype: int, T: int, k: int, d: int, pos, xs, rows: int, stream=None):
    """xs[pos[t*k + r]] = x[t] (see strata_moe_dispatch)."""
    c, xt = _Call(), _xtype(xdtype, "xdtype")
    c.run(_lib().strata_moe_dispatch, c.ptr(x, xt, T * d, "x"), xdtype, T, k, d, c.ptr(pos, torch.int32, T * k, "pos"),
          c.ptr(xs, xt, rows * d, "xs"), rows, stream=stream)


def dispatch_backward(dxs, xdtype: int, rows: int, pos, T: int, k: int, d: int, dx, stream=None):
    """dx[t] = sum over r of dxs[pos[t*k + r]] (see strata_moe_dispatch_backward)."""
    c, xt = _Call(), _xtype(xdtype, "xdtype")
    c.run(_lib().strata_moe_dispatch_backward, c.ptr(dxs, xt, rows * d, "dxs"), xdtype, rows,
          c.ptr(pos, torch.int32, T * k, "pos"), T, k, d, c.ptr(dx, xt, T * d, "dx"), stream=stream)


def combine(ys, ydtype: int, rows: int, pos, w, T: int, k: int, d: int, out, odtype: int, base=None, stream=None):
    """out[t] = base[t] + sum over r of w[t][r] * ys[pos[t*k + r]] (see strata_moe_combine)."""
    c, ot = _Call(), _xtype(odtype, "odtype")
    c.run(_lib().strata_moe_combine, c.ptr(ys, _xtype(ydtype, "ydtype"), rows * d, "ys"), ydtype, rows,
          c.ptr(pos, torch.int32, T * k, "pos"), c.ptr(w, torch.float32, T * k, "w"), T, k, d,
          c.ptr(base, ot, T * d, "base"), c.ptr(out, ot, T * d, "out"), odtype, stream=stream)


def combine_backward(dout, odtype: int, ys, ydtype: int, rows: int, pos, w, T: int, k: int, d: int, dys=None, dw=None,
                     dz=None, stream=None):
    """Gradients of the combine's rows, weights and picked logits (see strata_moe_combine_backward)."""
    c, yt, f32 = _Call(), _xtype(ydtype, "ydtype"), torch.float32
    c.run(_lib().strata_moe_combine_backward, c.ptr(dout, _xtype(odtype, "odtype"), T * d, "dout"), odtype,
          c.ptr(ys, yt, rows * d, "ys"), ydtype, rows, c.ptr(pos, torch.int32, T * k, "pos"),
          c.ptr(w, f32, T * k, "w"), T, k, d, c.ptr(dys, yt, rows * d, "dys"), c.ptr(dw, f32, T * k, "dw"),
          c.ptr(dz, f32, T * k, "dz"), stream=stream)


def grouped_workspace_bytes(rows: int, n_experts: int, N: int, K: int) -> int:
    n = _lib().strata_moe_grouped_workspace_bytes(rows, n_experts, N, K)
    if n == 0:
        _bad("unsupported product")
    return n


def grouped_product(x, W, offsets, rows: int, n_experts: int, N: int, K: int, y, ydtype: int, ws, ws_bytes: int,
                    stream=None):
    """y[s] = W_e x[s] over rows sorted by expert (see strata_moe_grouped_product)."""
    c, bf = _Call(), torch.bfloat16
    c.run(_lib().strata_moe_grouped_product, c.ptr(x, bf, rows * K, "x"), c.ptr(W, bf, n_experts * N * K, "W"),
          c.ptr(offsets, torch.int32, n_experts + 1, "offsets"), rows, n_experts, N, K,
          c.ptr(y, _xtype(ydtype, "ydtype"), rows * N, "y"), ydtype, c.ws(ws, ws_bytes), ws_bytes, stream=stream)


def grouped_dgrad(dy, W, offsets, rows: int, n_experts: int, N: int, K: int, dx, xdtype: int, ws, ws_bytes: int,
                  stream=None):
    """dx[s] = W_e^T dy[s] (see strata_moe_grouped_dgrad)."""
    c, bf = _Call(), torch.bfloat16
    c.run(_lib().strata_moe_grouped_dgrad, c.ptr(dy, bf, rows * N, "dy"), c.ptr(W, bf, n_experts * N * K, "W"),
          c.ptr(offsets, torch.int32, n_experts + 1, "offsets"), rows, n_experts, N, K,
          c.ptr(dx, _xtype(xdtype, "xdtype"), rows * K, "dx"), xdtype, c.ws(ws, ws_bytes), ws_bytes, stream=stream)


def grouped_wgrad(dy, x, offsets, rows: int, n_experts: int, N: int, K: int, dW, wdtype: int, ws, ws_bytes: int,
                  stream=None):
    """dW_e = sum over e's rows of dy[s] x[s]^T (see strata_moe_grouped_wgrad)."""
    c, bf = _Call(), torch.bfloat16
    c.run(_lib().strata_moe_grouped_wgrad, c.ptr(dy, bf, rows * N, "dy"), c.ptr(x, bf, rows * K, "x"),
          c.ptr(offsets, torch.int32, n_experts + 1, "offsets"), rows, n_experts, N, K,
          c.ptr(dW, _xtype(wdtype, "wdtype"), n_experts * N * K, "dW"), wdtype, c.ws(ws, ws_bytes), ws_bytes,
          stream=stream)


def block_norm_args(T: int, d: int, x_dtype: int, y_dtype: int, u_dtype: int, flags: int, resid_scale: float = 1.0,
                    branch_scale: float = 1.0, eps: float = 1e-6) -> BlockNormArgs:
    return BlockNormArgs(T, d, x_dtype, y_dtype, u_dtype, flags, resid_scale, branch_scale, eps)


def _gate(c: _Call, a: BlockNormArgs, gate, yt, name: str):
    if a.flags & GATE_TOKEN:
        return c.ptr(gate, torch.float32, a.T, name)
    return c.ptr(gate, yt, a.T * a.d, name)


def block_norm(args: BlockNormArgs, x, y, gate=None, g_post=None, g_pre=None, r=None, u=None, rstd_y=None,
               rstd_r=None, stream=None):
    """r = resid_scale x + branch_scale G norm(y), u = norm(r) (see strata_block_norm)."""
    c, a, f32 = _Call(), args, torch.float32
    T, d = a.T, a.d
    n, xt, yt = T * d, _xtype(a.x_dtype, "x_dtype"), _xtype(a.y_dtype, "y_dtype")
    c.run(_lib().strata_block_norm, ctypes.byref(a), c.ptr(x, xt, n, "x"), c.ptr(y, yt, n, "y"),
          _gate(c, a, gate, yt, "gate"), c.ptr(g_post, f32, d, "g_post"), c.ptr(g_pre, f32, d, "g_pre"),
          c.ptr(r, xt, n, "r"), c.ptr(u, _xtype(a.u_dtype, "u_dtype"), n, "u"), c.ptr(rstd_y, f32, T, "rstd_y"),
          c.ptr(rstd_r, f32, T, "rstd_r"), stream=stream)


def block_norm_backward_workspace_bytes(args: BlockNormArgs) -> int:
    n = _lib().strata_block_norm_backward_workspace_bytes(ctypes.byref(args))
    if n == 0:
        _bad("unsupported block norm")
    return n


def block_norm_backward(args: BlockNormArgs, dr, du, r, y, gate=None, g_post=None, g_pre=None, rstd_y=None,
                        rstd_r=None, dx=None, dy=None, dgate=None, dg_post=None, dg_pre=None, ws=None,
                        ws_bytes: int = 0, stream=None):
    """Gradients of block_norm's rows, gate and gains (see strata_block_norm_backward)."""
    c, a, f32 = _Call(), args, torch.float32
    T, d = a.T, a.d
    n, xt, yt, ut = T * d, _xtype(a.x_dtype, "x_dtype"), _xtype(a.y_dtype, "y_dtype"), _xtype(a.u_dtype, "u_dtype")
    c.run(_lib().strata_block_norm_backward, ctypes.byref(a), c.ptr(dr, xt, n, "dr"), c.ptr(du, ut, n, "du"),
          c.ptr(r, xt, n, "r"), c.ptr(y, yt, n, "y"), _gate(c, a, gate, yt, "gate"), c.ptr(g_post, f32, d, "g_post"),
          c.ptr(g_pre, f32, d, "g_pre"), c.ptr(rstd_y, f32, T, "rstd_y"), c.ptr(rstd_r, f32, T, "rstd_r"),
          c.ptr(dx, xt, n, "dx"), c.ptr(dy, yt, n, "dy"), _gate(c, a, dgate, yt, "dgate"),
          c.ptr(dg_post, f32, d, "dg_post"), c.ptr(dg_pre, f32, d, "dg_pre"), c.ws(ws, ws_bytes), ws_bytes,
          stream=stream)
