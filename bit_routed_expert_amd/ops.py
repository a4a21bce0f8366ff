"""Binding of the operators around the layer (include/strata_ops.h).

Tensors are checked before a call (device, type, contiguity, element count)
and a mismatch raises StrataError with STRATA_EINVAL; everything else is
checked by the library.  A call runs on the current stream of its tensors'
device unless one is given, with that device current.  Raw device addresses
(ints) are passed on unchecked, beside tensors or alone (then on the current
device).
"""
from __future__ import annotations

import ctypes
from typing import Optional

try:
    import torch
except ImportError:  # pragma: no cover -- the rest of the package imports without it
    torch = None

# The current stream's handle of a device: torch's direct accessor where it has one (a Stream object costs
# as much host time as the whole launch).
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)

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


def _wrong(t, dtype, n: int, dev: int, name: str):
    """Why _ptr refused a tensor."""
    if t.get_device() != dev:
        _bad(f"{name} is on {t.device}, not on cuda:{dev}" if dev >= 0 else f"{name} is not in device memory")
    if t.dtype is not dtype:
        _bad(f"{name} is {t.dtype}, not {dtype}")
    if t.numel() != n:
        _bad(f"{name} has {t.numel()} elements, not {n}")
    _bad(f"{name} is not contiguous")


def _device(*tensors) -> int:
    """Index of the first tensor's device; -2 when all are addresses or None."""
    for t in tensors:
        if t is not None and t.__class__ is not int:
            dev = t.get_device()
            if dev < 0:
                _bad("a tensor is not in device memory")
            return dev
    return -2


def _int32(bits: int):
    """Refuses sizes that a C int32 would cut; bits: the sizes or-ed together (a negative one shows too)."""
    if bits >> 31:
        _bad("a size is negative or does not fit 32 bits")


def _ptr(t, dtype, n: int, dev: int, name: str) -> Optional[int]:
    """Address of a contiguous tensor of n elements on the call's device (None and addresses pass)."""
    if t is None or t.__class__ is int:
        return t
    if t.get_device() != dev or t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        _wrong(t, dtype, n, dev, name)
    return t.data_ptr()


def _ws(t, n: int, dev: int) -> Optional[int]:
    """Address of a workspace said to hold n bytes."""
    if n < 0:
        _bad("ws_bytes is negative")
    if t is None or t.__class__ is int:
        return t
    if t.get_device() != dev:
        _bad(f"the workspace is on {t.device}, not on cuda:{dev}")
    if t.numel() * t.element_size() < n or not t.is_contiguous():
        _bad("the workspace is smaller than ws_bytes")
    return t.data_ptr()


def _call(fn, dev: int, stream, *args):
    """fn(*args, stream) with the tensors' device current, on its current stream unless one is given."""
    if dev >= 0 and dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = fn(*args, _stream(dev, stream))
    else:
        status = fn(*args, _stream(dev, stream))
    if status:
        from . import _check
        _check(status)


def _stream(dev: int, stream) -> int:
    if stream is not None:
        return stream if stream.__class__ is int else stream.cuda_stream
    return _raw_stream(dev if dev >= 0 else torch.cuda.current_device())


_library = None


def _lib():
    global _library
    if _library is None:
        from . import load_library
        _library = load_library()
    return _library


def _xtype(code: int, name: str):
    t = _XTYPES.get(code)
    if t is None:
        _bad(f"{name} is not X_BF16 or X_F32")
    return t


def sort_workspace_bytes(T: int, k: int, n_experts: int) -> int:
    _int32(T | k | n_experts)
    n = _lib().strata_moe_sort_workspace_bytes(T, k, n_experts)
    if n == 0:
        _bad("unsupported sort")
    return n


def sort_picks(idx, T: int, k: int, n_experts: int, counts, offsets, perm, pos, ws, ws_bytes: int, stream=None):
    """Picks sorted by expert (see strata_moe_sort); any output may be None."""
    v, i32, n = _device(idx, counts, offsets, perm, pos, ws), torch.int32, T * k
    _int32(T | k | n_experts)
    _call(_lib().strata_moe_sort, v, stream, _ptr(idx, i32, n, v, "idx"), T, k, n_experts,
          _ptr(counts, i32, n_experts, v, "counts"), _ptr(offsets, i32, n_experts + 1, v, "offsets"),
          _ptr(perm, i32, n, v, "perm"), _ptr(pos, i32, n, v, "pos"), _ws(ws, ws_bytes, v), ws_bytes)


def dispatch(x, xdtype: int, T: int, k: int, d: int, pos, xs, rows: int, stream=None):
    """xs[pos[t*k + r]] = x[t] (see strata_moe_dispatch)."""
    v, xt = _device(x, xs, pos), _xtype(xdtype, "xdtype")
    _int32(T | k | d | rows)
    _call(_lib().strata_moe_dispatch, v, stream, _ptr(x, xt, T * d, v, "x"), xdtype, T, k, d,
          _ptr(pos, torch.int32, T * k, v, "pos"), _ptr(xs, xt, rows * d, v, "xs"), rows)


def dispatch_backward(dxs, xdtype: int, rows: int, pos, T: int, k: int, d: int, dx, stream=None):
    """dx[t] = sum over r of dxs[pos[t*k + r]] (see strata_moe_dispatch_backward)."""
    v, xt = _device(dx, dxs, pos), _xtype(xdtype, "xdtype")
    _int32(T | k | d | rows)
    _call(_lib().strata_moe_dispatch_backward, v, stream, _ptr(dxs, xt, rows * d, v, "dxs"), xdtype, rows,
          _ptr(pos, torch.int32, T * k, v, "pos"), T, k, d, _ptr(dx, xt, T * d, v, "dx"))


def combine(ys, ydtype: int, rows: int, pos, w, T: int, k: int, d: int, out, odtype: int, base=None, stream=None):
    """out[t] = base[t] + sum over r of w[t][r] * ys[pos[t*k + r]] (see strata_moe_combine)."""
    v, ot = _device(out, ys, pos, w, base), _xtype(odtype, "odtype")
    _int32(T | k | d | rows)
    _call(_lib().strata_moe_combine, v, stream, _ptr(ys, _xtype(ydtype, "ydtype"), rows * d, v, "ys"), ydtype, rows,
          _ptr(pos, torch.int32, T * k, v, "pos"), _ptr(w, torch.float32, T * k, v, "w"), T, k, d,
          _ptr(base, ot, T * d, v, "base"), _ptr(out, ot, T * d, v, "out"), odtype)


def combine_backward(dout, odtype: int, ys, ydtype: int, rows: int, pos, w, T: int, k: int, d: int, dys=None, dw=None,
                     dz=None, stream=None):
    """Gradients of the combine's rows, weights and picked logits (see strata_moe_combine_backward)."""
    v, yt, f32 = _device(dout, ys, pos, w, dys, dw, dz), _xtype(ydtype, "ydtype"), torch.float32
    _int32(T | k | d | rows)
    _call(_lib().strata_moe_combine_backward, v, stream, _ptr(dout, _xtype(odtype, "odtype"), T * d, v, "dout"),
          odtype, _ptr(ys, yt, rows * d, v, "ys"), ydtype, rows, _ptr(pos, torch.int32, T * k, v, "pos"),
          _ptr(w, f32, T * k, v, "w"), T, k, d, _ptr(dys, yt, rows * d, v, "dys"), _ptr(dw, f32, T * k, v, "dw"),
          _ptr(dz, f32, T * k, v, "dz"))


def grouped_workspace_bytes(rows: int, n_experts: int, N: int, K: int) -> int:
    _int32(rows | n_experts | N | K)
    n = _lib().strata_moe_grouped_workspace_bytes(rows, n_experts, N, K)
    if n == 0:
        _bad("unsupported product")
    return n


def grouped_product(x, W, offsets, rows: int, n_experts: int, N: int, K: int, y, ydtype: int, ws, ws_bytes: int,
                    stream=None):
    """y[s] = W_e x[s] over rows sorted by expert (see strata_moe_grouped_product)."""
    v, bf = _device(W, x, y, offsets, ws), torch.bfloat16
    _int32(rows | n_experts | N | K)
    _call(_lib().strata_moe_grouped_product, v, stream, _ptr(x, bf, rows * K, v, "x"),
          _ptr(W, bf, n_experts * N * K, v, "W"), _ptr(offsets, torch.int32, n_experts + 1, v, "offsets"), rows,
          n_experts, N, K, _ptr(y, _xtype(ydtype, "ydtype"), rows * N, v, "y"), ydtype, _ws(ws, ws_bytes, v), ws_bytes)


def grouped_dgrad(dy, W, offsets, rows: int, n_experts: int, N: int, K: int, dx, xdtype: int, ws, ws_bytes: int,
                  stream=None):
    """dx[s] = W_e^T dy[s] (see strata_moe_grouped_dgrad)."""
    v, bf = _device(W, dy, dx, offsets, ws), torch.bfloat16
    _int32(rows | n_experts | N | K)
    _call(_lib().strata_moe_grouped_dgrad, v, stream, _ptr(dy, bf, rows * N, v, "dy"),
          _ptr(W, bf, n_experts * N * K, v, "W"), _ptr(offsets, torch.int32, n_experts + 1, v, "offsets"), rows,
          n_experts, N, K, _ptr(dx, _xtype(xdtype, "xdtype"), rows * K, v, "dx"), xdtype, _ws(ws, ws_bytes, v),
          ws_bytes)


def grouped_wgrad(dy, x, offsets, rows: int, n_experts: int, N: int, K: int, dW, wdtype: int, ws, ws_bytes: int,
                  stream=None):
    """dW_e = sum over e's rows of dy[s] x[s]^T (see strata_moe_grouped_wgrad)."""
    v, bf = _device(dW, dy, x, offsets, ws), torch.bfloat16
    _int32(rows | n_experts | N | K)
    _call(_lib().strata_moe_grouped_wgrad, v, stream, _ptr(dy, bf, rows * N, v, "dy"), _ptr(x, bf, rows * K, v, "x"),
          _ptr(offsets, torch.int32, n_experts + 1, v, "offsets"), rows, n_experts, N, K,
          _ptr(dW, _xtype(wdtype, "wdtype"), n_experts * N * K, v, "dW"), wdtype, _ws(ws, ws_bytes, v), ws_bytes)


def block_norm_args(T: int, d: int, x_dtype: int, y_dtype: int, u_dtype: int, flags: int, resid_scale: float = 1.0,
                    branch_scale: float = 1.0, eps: float = 1e-6) -> BlockNormArgs:
    if not (-1 << 31 <= T < 1 << 31 and -1 << 31 <= d < 1 << 31):   # the library refuses the other bad ones
        _bad("a size does not fit 32 bits")
    return BlockNormArgs(T, d, x_dtype, y_dtype, u_dtype, flags, resid_scale, branch_scale, eps)


def _gate(a: BlockNormArgs, gate, yt, dev: int, name: str):
    if gate is None:
        return None
    if a.flags & GATE_TOKEN:
        return _ptr(gate, torch.float32, a.T, dev, name)
    return _ptr(gate, yt, a.T * a.d, dev, name)


def block_norm(args: BlockNormArgs, x, y, gate=None, g_post=None, g_pre=None, r=None, u=None, rstd_y=None,
               rstd_r=None, stream=None):
    """r = resid_scale x + branch_scale G norm(y), u = norm(r) (see strata_block_norm)."""
    v, f32, T, d = _device(x, y, r, u, gate, g_post, g_pre, rstd_y, rstd_r), torch.float32, args.T, args.d
    n, xt, yt = T * d, _xtype(args.x_dtype, "x_dtype"), _xtype(args.y_dtype, "y_dtype")
    _call(_lib().strata_block_norm, v, stream, ctypes.byref(args), _ptr(x, xt, n, v, "x"), _ptr(y, yt, n, v, "y"),
          _gate(args, gate, yt, v, "gate"), _ptr(g_post, f32, d, v, "g_post"), _ptr(g_pre, f32, d, v, "g_pre"),
          _ptr(r, xt, n, v, "r"), _ptr(u, _xtype(args.u_dtype, "u_dtype"), n, v, "u"),
          _ptr(rstd_y, f32, T, v, "rstd_y"), _ptr(rstd_r, f32, T, v, "rstd_r"))


def block_norm_backward_workspace_bytes(args: BlockNormArgs) -> int:
    n = _lib().strata_block_norm_backward_workspace_bytes(ctypes.byref(args))
    if n == 0:
        _bad("unsupported block norm")
    return n


def block_norm_backward(args: BlockNormArgs, dr, du, r, y, gate=None, g_post=None, g_pre=None, rstd_y=None,
                        rstd_r=None, dx=None, dy=None, dgate=None, dg_post=None, dg_pre=None, ws=None,
                        ws_bytes: int = 0, stream=None):
    """Gradients of block_norm's rows, gate and gains (see strata_block_norm_backward)."""
    v = _device(dr, du, r, y, dx, dy, dg_post, dg_pre, gate, g_post, g_pre, rstd_y, rstd_r, dgate, ws)
    f32, T, d = torch.float32, args.T, args.d
    n, xt, yt = T * d, _xtype(args.x_dtype, "x_dtype"), _xtype(args.y_dtype, "y_dtype")
    _call(_lib().strata_block_norm_backward, v, stream, ctypes.byref(args), _ptr(dr, xt, n, v, "dr"),
          _ptr(du, _xtype(args.u_dtype, "u_dtype"), n, v, "du"), _ptr(r, xt, n, v, "r"), _ptr(y, yt, n, v, "y"),
          _gate(args, gate, yt, v, "gate"), _ptr(g_post, f32, d, v, "g_post"), _ptr(g_pre, f32, d, v, "g_pre"),
          _ptr(rstd_y, f32, T, v, "rstd_y"), _ptr(rstd_r, f32, T, v, "rstd_r"), _ptr(dx, xt, n, v, "dx"),
          _ptr(dy, yt, n, v, "dy"), _gate(args, dgate, yt, v, "dgate"), _ptr(dg_post, f32, d, v, "dg_post"),
          _ptr(dg_pre, f32, d, v, "dg_pre"), _ws(ws, ws_bytes, v), ws_bytes)
