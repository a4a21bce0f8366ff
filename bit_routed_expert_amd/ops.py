"""Binding of the operators around the layer (include/strata_ops.h) and of the
ends of a training step (include/strata_train.h).

Tensors are checked before a call (device, type, contiguity, element count)
and a mismatch raises StrataError with STRATA_EINVAL; everything else is
checked by the library.  A call runs on the current stream of its tensors'
device unless one is given, with that device current; a stream of another
device is refused.  Raw device addresses (ints) are passed on unchecked, beside
tensors or alone (then on the current device), and so is a raw stream.  The checks are compiled (csrc/binding.cpp, the module _binding): a
small call's time is the host's.
"""
from __future__ import annotations

import ctypes

POST_NORM, PRE_NORM, GATE_TOKEN, GATE_CHANNEL, GATE_SIGMOID = 1, 2, 4, 8, 16
ACCUMULATE = 1   # STRATA_ACCUMULATE

_EINVAL = 1

SYMBOLS = ("strata_moe_sort_workspace_bytes", "strata_moe_sort", "strata_moe_dispatch",
           "strata_moe_dispatch_backward", "strata_moe_combine", "strata_moe_combine_backward",
           "strata_moe_grouped_workspace_bytes", "strata_moe_grouped_product", "strata_moe_grouped_dgrad",
           "strata_moe_grouped_wgrad", "strata_block_norm", "strata_block_norm_backward_workspace_bytes",
           "strata_block_norm_backward", "strata_moe_balance_workspace_bytes", "strata_moe_balance",
           "strata_moe_balance_backward", "strata_embed", "strata_embed_backward_workspace_bytes", "strata_embed_backward",
           "strata_vocab_loss_workspace_bytes", "strata_vocab_loss_backward_workspace_bytes", "strata_vocab_loss",
           "strata_vocab_loss_backward", "strata_orthogonalise_workspace_bytes", "strata_orthogonalise")


class BlockNormArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("u_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("resid_scale", ctypes.c_float), ("branch_scale", ctypes.c_float), ("eps", ctypes.c_float)]


def declare(lib):
    """Signatures of the functions above on a loaded library."""
    vp, i32, sz, it = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
    u32, fl = ctypes.c_uint32, ctypes.c_float
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
            ("strata_block_norm_backward", it, [norm] + [vp] * 15 + [sz, vp]),
            ("strata_moe_balance_workspace_bytes", sz, [i32, i32, i32]),
            ("strata_moe_balance", it, [vp, it, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
            ("strata_moe_balance_backward", it, [vp, it, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]),
            ("strata_embed", it, [vp, it, i32, i32, vp, i32, fl, vp, it, vp]),
            ("strata_embed_backward_workspace_bytes", sz, [i32, i32, i32]),
            ("strata_embed_backward", it, [vp, it, vp, i32, i32, i32, fl, vp, it, u32, vp, sz, vp]),
            ("strata_vocab_loss_workspace_bytes", sz, [i32, i32, i32]),
            ("strata_vocab_loss_backward_workspace_bytes", sz, [i32, i32, i32]),
            ("strata_vocab_loss", it, [vp, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]),
            ("strata_vocab_loss_backward", it,
             [vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, it, vp, it, u32, vp, sz, vp]),
            ("strata_orthogonalise_workspace_bytes", sz, [i32, i32, i32]),
            ("strata_orthogonalise", it, [vp, it, i32, i32, i32, i32, ctypes.POINTER(fl), fl, fl, vp, vp, sz, vp])):
        f = getattr(lib, name)
        f.restype = restype
        f.argtypes = argtypes


def _raise(what):
    """Raises for a status of the library, or for what a check found."""
    from . import StrataError, _check
    if what.__class__ is str:
        raise StrataError(_EINVAL, what)
    _check(what)


def _elsewhere(dev: int, fn, *args):
    """fn(*args) with device dev current."""
    import torch
    with torch.cuda.device(dev):
        fn(*args)


_library = None


def _lib():
    global _library
    if _library is None:
        from . import load_library
        _library = load_library()
    return _library


class _Unloaded:
    """Stands for _binding until the first call, which loads it and gives it the library's functions."""

    def __getattr__(self, name):
        global _native
        lib = _lib()
        try:
            import torch   # here and not above: the package is imported without it, and sooner
            from . import _binding
        except ImportError as e:
            raise RuntimeError("the operators need torch and a _binding.so built against it: build it with "
                               "`python -m bit_routed_expert_amd.build`") from e
        fns = tuple(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in _BOUND)
        # torch's direct accessors where it has them: a Stream object costs as much host time as the launch
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _binding.bind(fns, _raise, _elsewhere, device, torch.cuda.current_device, stream)
        _native = _binding
        return getattr(_binding, name)


_native = _Unloaded()
_BOUND = ("strata_moe_sort", "strata_moe_dispatch", "strata_moe_dispatch_backward", "strata_moe_combine",
          "strata_moe_combine_backward", "strata_moe_grouped_product", "strata_moe_grouped_dgrad",
          "strata_moe_grouped_wgrad", "strata_block_norm", "strata_block_norm_backward", "strata_moe_balance",
          "strata_moe_balance_backward", "strata_embed", "strata_embed_backward", "strata_vocab_loss",
          "strata_vocab_loss_backward", "strata_orthogonalise")   # in _binding's order


def _int32(bits: int):
    """Refuses sizes that a C int32 would cut; bits: the sizes or-ed together (a negative one shows too)."""
    if bits >> 31:
        _raise("a size is negative or does not fit 32 bits")


def sort_workspace_bytes(T: int, k: int, n_experts: int) -> int:
    _int32(T | k | n_experts)
    n = _lib().strata_moe_sort_workspace_bytes(T, k, n_experts)
    if n == 0:
        _raise("unsupported sort")
    return n


def sort_picks(idx, T: int, k: int, n_experts: int, counts, offsets, perm, pos, ws, ws_bytes: int, stream=None):
    """Picks sorted by expert (see strata_moe_sort); any output may be None."""
    _native.sort_picks(idx, T, k, n_experts, counts, offsets, perm, pos, ws, ws_bytes, stream)


def dispatch(x, xdtype: int, T: int, k: int, d: int, pos, xs, rows: int, stream=None):
    """xs[pos[t*k + r]] = x[t] (see strata_moe_dispatch)."""
    _native.dispatch(x, xdtype, T, k, d, pos, xs, rows, stream)


def dispatch_backward(dxs, xdtype: int, rows: int, pos, T: int, k: int, d: int, dx, stream=None):
    """dx[t] = sum over r of dxs[pos[t*k + r]] (see strata_moe_dispatch_backward)."""
    _native.dispatch_backward(dxs, xdtype, rows, pos, T, k, d, dx, stream)


def combine(ys, ydtype: int, rows: int, pos, w, T: int, k: int, d: int, out, odtype: int, base=None, stream=None):
    """out[t] = base[t] + sum over r of w[t][r] * ys[pos[t*k + r]] (see strata_moe_combine)."""
    _native.combine(ys, ydtype, rows, pos, w, T, k, d, out, odtype, base, stream)


def combine_backward(dout, odtype: int, ys, ydtype: int, rows: int, pos, w, T: int, k: int, d: int, dys=None, dw=None,
                     dz=None, stream=None):
    """Gradients of the combine's rows, weights and picked logits (see strata_moe_combine_backward)."""
    _native.combine_backward(dout, odtype, ys, ydtype, rows, pos, w, T, k, d, dys, dw, dz, stream)


def grouped_workspace_bytes(rows: int, n_experts: int, N: int, K: int) -> int:
    _int32(rows | n_experts | N | K)
    n = _lib().strata_moe_grouped_workspace_bytes(rows, n_experts, N, K)
    if n == 0:
        _raise("unsupported product")
    return n


def grouped_product(x, W, offsets, rows: int, n_experts: int, N: int, K: int, y, ydtype: int, ws, ws_bytes: int,
                    stream=None):
    """y[s] = W_e x[s] over rows sorted by expert (see strata_moe_grouped_product)."""
    _native.grouped_product(x, W, offsets, rows, n_experts, N, K, y, ydtype, ws, ws_bytes, stream)


def grouped_dgrad(dy, W, offsets, rows: int, n_experts: int, N: int, K: int, dx, xdtype: int, ws, ws_bytes: int,
                  stream=None):
    """dx[s] = W_e^T dy[s] (see strata_moe_grouped_dgrad)."""
    _native.grouped_dgrad(dy, W, offsets, rows, n_experts, N, K, dx, xdtype, ws, ws_bytes, stream)


def grouped_wgrad(dy, x, offsets, rows: int, n_experts: int, N: int, K: int, dW, wdtype: int, ws, ws_bytes: int,
                  stream=None):
    """dW_e = sum over e's rows of dy[s] x[s]^T (see strata_moe_grouped_wgrad)."""
    _native.grouped_wgrad(dy, x, offsets, rows, n_experts, N, K, dW, wdtype, ws, ws_bytes, stream)


def block_norm_args(T: int, d: int, x_dtype: int, y_dtype: int, u_dtype: int, flags: int, resid_scale: float = 1.0,
                    branch_scale: float = 1.0, eps: float = 1e-6) -> BlockNormArgs:
    if not (-1 << 31 <= T < 1 << 31 and -1 << 31 <= d < 1 << 31):   # the library refuses the other bad ones
        _raise("a size does not fit 32 bits")
    return BlockNormArgs(T, d, x_dtype, y_dtype, u_dtype, flags, resid_scale, branch_scale, eps)


def block_norm(args: BlockNormArgs, x, y, gate=None, g_post=None, g_pre=None, r=None, u=None, rstd_y=None,
               rstd_r=None, stream=None):
    """r = resid_scale x + branch_scale G norm(y), u = norm(r) (see strata_block_norm)."""
    _native.block_norm(args, x, y, gate, g_post, g_pre, r, u, rstd_y, rstd_r, stream)


def block_norm_backward_workspace_bytes(args: BlockNormArgs) -> int:
    n = _lib().strata_block_norm_backward_workspace_bytes(ctypes.byref(args))
    if n == 0:
        _raise("unsupported block norm")
    return n


def block_norm_backward(args: BlockNormArgs, dr, du, r, y, gate=None, g_post=None, g_pre=None, rstd_y=None,
                        rstd_r=None, dx=None, dy=None, dgate=None, dg_post=None, dg_pre=None, ws=None,
                        ws_bytes: int = 0, stream=None):
    """Gradients of block_norm's rows, gate and gains (see strata_block_norm_backward)."""
    _native.block_norm_backward(args, dr, du, r, y, gate, g_post, g_pre, rstd_y, rstd_r, dx, dy, dgate, dg_post, dg_pre,
                                ws, ws_bytes, stream)


# ------------------------------------------------ the ends of a training step

def _workspace(name: str, what: str, a: int, b: int, c: int) -> int:
    _int32(a | b | c)
    n = getattr(_lib(), name)(a, b, c)
    if n == 0:
        _raise(f"unsupported {what}")
    return n


def balance_loss_workspace_bytes(T: int, k: int, n_experts: int) -> int:
    return _workspace("strata_moe_balance_workspace_bytes", "balance loss", T, k, n_experts)


def balance_loss(z, zdtype: int, idx, T: int, k: int, n_experts: int, losses, counts, lse, tokens, ws, ws_bytes: int,
                 prob=None, keep=None, stream=None):
    """Balance and z loss of a router's logits, its picks counted per expert (see strata_moe_balance)."""
    _native.balance_loss(z, zdtype, idx, T, k, n_experts, losses, counts, lse, tokens, ws, ws_bytes, prob, keep, stream)


def balance_loss_backward(z, zdtype: int, idx, T: int, k: int, n_experts: int, lse, counts, tokens, dlosses, dz, keep=None,
                          dpicks=None, stream=None):
    """The logits' gradient, that of the picked logits added (see strata_moe_balance_backward)."""
    _native.balance_loss_backward(z, zdtype, idx, T, k, n_experts, lse, counts, tokens, dlosses, dz, keep, dpicks, stream)


def embed(W, wdtype: int, V: int, d: int, ids, T: int, scale: float, out, odtype: int, stream=None):
    """out[t] = scale * W[ids[t]] (see strata_embed)."""
    _native.embed(W, wdtype, V, d, ids, T, scale, out, odtype, stream)


def embed_backward_workspace_bytes(T: int, V: int, d: int) -> int:
    return _workspace("strata_embed_backward_workspace_bytes", "embedding", T, V, d)


def embed_backward(dout, odtype: int, ids, T: int, V: int, d: int, scale: float, dW, wdtype: int, ws, ws_bytes: int,
                   flags: int = 0, stream=None):
    """dW[v] = scale * sum of dout[t] over the tokens of id v (see strata_embed_backward)."""
    _native.embed_backward(dout, odtype, ids, T, V, d, scale, dW, wdtype, ws, ws_bytes, flags, stream)


def vocab_loss_workspace_bytes(T: int, V: int, d: int) -> int:
    return _workspace("strata_vocab_loss_workspace_bytes", "vocabulary loss", T, V, d)


def vocab_loss(h, W, targets, T: int, V: int, d: int, loss, lse, ws, ws_bytes: int, stream=None):
    """Softmax cross entropy of W h[t] at targets[t] (see strata_vocab_loss)."""
    _native.vocab_loss(h, W, targets, T, V, d, loss, lse, ws, ws_bytes, stream)


def vocab_loss_backward_workspace_bytes(T: int, V: int, d: int) -> int:
    return _workspace("strata_vocab_loss_backward_workspace_bytes", "vocabulary loss", T, V, d)


def vocab_loss_backward(h, W, targets, T: int, V: int, d: int, lse, dloss, ws, ws_bytes: int, dlse=None, dh=None,
                        dhdtype: int = 0, dW=None, dwdtype: int = 0, flags: int = 0, stream=None):
    """Gradients of the hidden rows and of the output matrix (see strata_vocab_loss_backward)."""
    _native.vocab_loss_backward(h, W, targets, T, V, d, lse, dloss, ws, ws_bytes, dlse, dh, dhdtype, dW, dwdtype, flags,
                                stream)


def orthogonalise_workspace_bytes(n: int, N: int, K: int) -> int:
    return _workspace("strata_orthogonalise_workspace_bytes", "matrices", n, N, K)


def orthogonalise(G, gdtype: int, n: int, N: int, K: int, out, ws, ws_bytes: int, steps: int = 5,
                  coefficients=(3.4445, -4.7750, 2.0315), scale: float = 1.0, eps: float = 1e-7, stream=None):
    """out = scale * the matrices of G orthogonalised by Newton-Schulz products (see strata_orthogonalise)."""
    a, b, c = coefficients
    _native.orthogonalise(G, gdtype, n, N, K, out, ws, ws_bytes, steps, a, b, c, scale, eps, stream)
