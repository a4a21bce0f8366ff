"""Operators around the layer, without a GPU: the refusals of every entry
point (nothing is launched when validation fails), workspace sizes, and the
reference's gradients against differences."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import bit_routed_expert_amd as brx
from tests import ops_ref as R

EINVAL, EUNSUP, EWS, OK = brx.STRATA_EINVAL, brx.STRATA_EUNSUPPORTED, brx.STRATA_EWORKSPACE, brx.STRATA_OK
P = 0x10000   # placeholders: validation fails before anything touches them


def lib():
    return brx.load_library()


def test_sort_refusals():
    f, ws = lib().strata_moe_sort, lib().strata_moe_sort_workspace_bytes
    need = ws(50000, 10, 512)
    assert need >= 4 * 512 * 200 and ws(5, 10, 512) > 0 and ws(0, 1, 1) > 0

    def call(idx=P, T=50000, k=10, E=512, w=P, wb=need):
        return f(idx, T, k, E, P, P, P, P, w, wb, None)
    assert call(idx=None) == EINVAL and call(w=None) == EINVAL and call(w=P + 8) == EINVAL
    for bad in (dict(T=-1), dict(k=0), dict(k=33), dict(E=0), dict(E=1025)):
        assert call(**bad) == EINVAL
        a = dict(T=5000, k=10, E=512, **{}) | bad
        assert ws(a["T"], a["k"], a["E"]) == 0
    assert call(wb=need - 1) == EWS
    assert call(T=2**31 - 1, k=2, wb=1 << 40) == EUNSUP and ws(2**31 - 1, 2, 512) == 0


def test_sort_refuses_outputs_over_its_inputs():
    """Blocks read all the picks while others already write, so no output may
    lie over idx; nor over the workspace where it carries counts between launches."""
    f, wsb = lib().strata_moe_sort, lib().strata_moe_sort_workspace_bytes
    G = 1 << 30   # apart

    def call(T, k=10, E=512, idx=G, counts=2 * G, offsets=3 * G, perm=4 * G, pos=5 * G, w=6 * G):
        return f(idx, T, k, E, counts, offsets, perm, pos, w, wsb(T, k, E), None)
    for T in (5, 400, 50000):
        n, need = T * 10 * 4, wsb(T, 10, 512)
        for name, size in (("counts", 512 * 4), ("offsets", 513 * 4), ("perm", n), ("pos", n)):
            for at in (G, G + n - 4, G - size + 4):
                assert call(T, **{name: at}) == EINVAL, (T, name, at - G)
            if n > 65535 * 4:
                for at in (6 * G, 6 * G + need - 4, 6 * G - size + 4):
                    assert call(T, **{name: at}) == EINVAL, (T, name, at - 6 * G)
        if n > 65535 * 4:
            assert call(T, w=G) == EINVAL and call(T, w=G + n - 16) == EINVAL and call(T, idx=6 * G + need - 4) == EINVAL


def test_dispatch_and_combine_refusals():
    d, db, c, cb = (lib().strata_moe_dispatch, lib().strata_moe_dispatch_backward, lib().strata_moe_combine,
                    lib().strata_moe_combine_backward)

    def calls(a=P, b=P, pos=P, rows=20, T=5, k=4, dd=64, xt=0, w=P):
        """a: the slot rows, b: the token rows."""
        return [d(b, xt, T, k, dd, pos, a, rows, None), db(a, xt, rows, pos, T, k, dd, b, None),
                c(a, xt, rows, pos, w, T, k, dd, None, b, xt, None),
                cb(b, xt, a, xt, rows, pos, w, T, k, dd, P, P, P, None)]
    for bad in (dict(a=None), dict(b=None), dict(pos=None), dict(a=P + 2), dict(b=P + 4), dict(rows=-1), dict(T=-1),
                dict(k=0), dict(k=33), dict(dd=0), dict(xt=2)):
        assert calls(**bad) == [EINVAL] * 4, bad
    assert calls(T=2**23 + 1) == [EUNSUP] * 4 and calls(dd=2**24 + 1) == [EUNSUP] * 4
    assert calls(T=0, a=None, b=None, pos=None) == [OK] * 4
    assert cb(P, 0, P, 0, 20, P, None, 5, 4, 64, P, P, P, None) == EINVAL          # no weights
    assert cb(P, 0, P, 0, 20, P, P, 5, 4, 64, P + 8, P, P, None) == EINVAL
    assert cb(P, 0, P, 0, 20, P, P, 5, 4, 64, None, None, None, None) == OK        # nothing asked for
    assert c(P, 0, 20, P, P, 5, 4, 64, P + 8, P, 0, None) == EINVAL                # base


@pytest.mark.parametrize("name", ["product", "dgrad", "wgrad"])
def test_grouped_refusals(name):
    f, ws = getattr(lib(), f"strata_moe_grouped_{name}"), lib().strata_moe_grouped_workspace_bytes
    need = ws(100, 8, 64, 128)
    assert need > 0

    def call(a=P, b=P, off=P, rows=100, E=8, N=64, K=128, c=P, t=0, w=P, wb=need):
        return f(a, b, off, rows, E, N, K, c, t, w, wb, None)
    for bad in (dict(a=None), dict(b=None), dict(off=None), dict(c=None), dict(w=None), dict(a=P + 8),
                dict(b=P + 2), dict(c=P + 4), dict(w=P + 8), dict(t=3), dict(rows=-1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(E=0), dict(E=1025), dict(N=60), dict(K=4), dict(N=0), dict(K=65544), dict(N=65536, K=16384),
                dict(E=1024, N=32768, K=8192), dict(rows=2**22 + 1)):
        assert call(**bad, wb=1 << 40) == EUNSUP, bad
        a = dict(rows=100, E=8, N=64, K=128) | bad
        assert ws(a["rows"], a["E"], a["N"], a["K"]) == 0
    assert call(wb=need - 1) == EWS
    if name != "wgrad":
        assert call(rows=0, a=None, b=None, off=None, c=None, w=None) == OK


@pytest.mark.parametrize("name", ["product", "dgrad", "wgrad"])
def test_grouped_refuses_an_output_over_its_workspace(name):
    """Blocks take their rows from a list in the workspace while others already store."""
    f, G, rows, E, N, K = getattr(lib(), f"strata_moe_grouped_{name}"), 1 << 30, 1683, 40, 1288, 264
    need = lib().strata_moe_grouped_workspace_bytes(rows, E, N, K)
    for t, step in ((0, 2), (1, 4)):
        size = step * {"product": rows * N, "dgrad": rows * K, "wgrad": E * N * K}[name]
        for c in (5 * G, 5 * G + need // 16 * 16, 5 * G - size // 16 * 16 + 16):
            if not 5 * G - size < c < 5 * G + need:
                continue
            assert f(G, 2 * G, 3 * G, rows, E, N, K, c, t, 5 * G, need, None) == EINVAL, (t, c - 5 * G)


@pytest.mark.parametrize("name", ["product", "dgrad"])
def test_grouped_without_rows_checks_the_rest(name):
    """A call without rows does nothing whatever its pointers are, but a bad dtype or shape stays an error."""
    f = getattr(lib(), f"strata_moe_grouped_{name}")
    for t, E, N, want in ((0, 8, 64, OK), (1, 8, 64, OK), (2, 8, 64, EINVAL), (-1, 8, 64, EINVAL), (0, 0, 64, EUNSUP),
                          (1, 8, 60, EUNSUP)):
        assert f(None, None, None, 0, E, N, 128, None, t, None, 0, None) == want, (t, E, N)


def _args(**kw):
    a = dict(T=5, d=64, x_dtype=1, y_dtype=0, u_dtype=0, flags=brx.POST_NORM | brx.PRE_NORM)
    a.update(kw)
    return brx.block_norm_args(**a)


BAD_ARGS = [dict(T=-1), dict(d=0), dict(x_dtype=2), dict(y_dtype=-1), dict(u_dtype=7), dict(flags=64),
            dict(flags=brx.GATE_TOKEN | brx.GATE_CHANNEL), dict(flags=brx.GATE_SIGMOID), dict(eps=0.0),
            dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(resid_scale=float("nan")),
            dict(branch_scale=float("inf"))]


def test_block_norm_refusals():
    f = lib().strata_block_norm

    def call(a=None, x=P, y=P, gate=None, gp=P, gq=P, r=P, u=P, sy=P, sr=P, **kw):
        return f(ctypes.byref(a or _args(**kw)), x, y, gate, gp, gq, r, u, sy, sr, None)
    assert f(None, P, P, None, P, P, P, P, P, P, None) == EINVAL
    for bad in BAD_ARGS:
        assert call(**bad) == EINVAL, bad
    assert call(d=8193) == EUNSUP and call(T=2**23 + 1) == EUNSUP
    assert call(T=0, x=None, y=None, gp=None, gq=None, r=None, u=None, sy=None, sr=None) == OK
    for bad in (dict(x=None), dict(y=None), dict(u=None), dict(gate=P), dict(x=P + 4), dict(y=P + 2), dict(r=P + 8),
                dict(u=P + 8), dict(gp=P + 4), dict(gq=P + 4)):
        assert call(**bad) == EINVAL, bad
    post, pre = brx.POST_NORM, brx.PRE_NORM
    assert call(flags=post) == EINVAL                              # u and g_pre without the pre norm
    assert call(flags=post, u=None, gq=None) == EINVAL             # rstd_r
    assert call(flags=pre) == EINVAL                               # g_post without the post norm
    assert call(flags=pre, gp=None) == EINVAL                      # rstd_y
    assert call(flags=post, u=None, gq=None, sr=None, r=None) == EINVAL   # no output
    assert call(flags=post | pre | brx.GATE_TOKEN) == EINVAL       # no gate
    assert call(flags=pre | brx.GATE_CHANNEL, y=None, gate=P, gp=None, sy=None) == EINVAL   # a gate without a branch


def test_block_norm_backward_refusals():
    f, ws = lib().strata_block_norm_backward, lib().strata_block_norm_backward_workspace_bytes
    need = ws(ctypes.byref(_args()))
    assert need >= 2 * 64 * 4
    for bad in BAD_ARGS:
        assert ws(ctypes.byref(_args(**bad))) == 0

    def call(a=None, dr=P, du=P, r=P, y=P, gate=None, gp=P, gq=P, sy=P, sr=P, dx=P, dy=P, dg=None, dgp=P, dgq=P, w=P,
             wb=need, **kw):
        return f(ctypes.byref(a or _args(**kw)), dr, du, r, y, gate, gp, gq, sy, sr, dx, dy, dg, dgp, dgq, w, wb, None)
    for bad in BAD_ARGS:
        assert call(**bad) == EINVAL, bad
    assert call(d=8193) == EUNSUP
    for bad in (dict(du=None), dict(r=None), dict(sr=None), dict(sy=None), dict(y=None), dict(gate=P), dict(dg=P),
                dict(w=None), dict(w=P + 8), dict(dr=P + 4), dict(dx=P + 4), dict(dgp=P + 4), dict(dy=P + 8)):
        assert call(**bad) == EINVAL, bad
    assert call(wb=need - 1) == EWS
    post, pre = brx.POST_NORM, brx.PRE_NORM
    assert call(flags=pre, gp=None) == EINVAL                      # dg_post without the post norm
    assert call(flags=post, gq=None, du=None) == EINVAL            # dg_pre without the pre norm
    assert call(flags=post, gq=None, dgq=None) == EINVAL           # du without it
    assert call(flags=post, gq=None, dgq=None, du=None, dr=None) == EINVAL   # no gradient comes in
    assert call(flags=pre, gp=None, dgp=None, y=None, sy=None) == EINVAL     # dy without y


def test_binding_checks_tensors():
    """Tensors of the wrong type, size, layout or device are refused before the library is called."""
    i = torch.zeros(20, dtype=torch.int32)
    with pytest.raises(brx.StrataError) as e:
        brx.sort_picks(i, 5, 4, 8, None, None, None, None, None, 0)
    assert e.value.status == EINVAL and "device memory" in str(e.value)
    with pytest.raises(brx.StrataError):
        brx.dispatch(torch.zeros(5, 64), 2, 5, 4, 64, i, torch.zeros(20, 64), 20)
    with pytest.raises(brx.StrataError):
        brx.block_norm(_args(x_dtype=5), None, None)
    with pytest.raises(brx.StrataError):
        brx.grouped_workspace_bytes(10, 4, 12, 64)
    with pytest.raises(brx.StrataError):
        brx.sort_workspace_bytes(10, 4, 0)
    with pytest.raises(brx.StrataError):
        brx.block_norm_backward_workspace_bytes(_args(eps=0.0))


SIZES = {   # every entry point's sizes, and the positions of its tensors
    "sort_picks": (lambda T, *t: brx.sort_picks(t[0], T, 4, 8, *t[1:6], 256), 6),
    "dispatch": (lambda T, *t: brx.dispatch(t[0], 1, T, 4, 64, t[1], t[2], 20), 3),
    "dispatch_backward": (lambda T, *t: brx.dispatch_backward(t[0], 1, T, t[1], 5, 4, 64, t[2]), 3),
    "combine": (lambda T, *t: brx.combine(t[0], 1, T, t[1], t[2], 5, 4, 64, t[3], 1, base=t[4]), 5),
    "combine_backward": (lambda T, *t: brx.combine_backward(t[0], 1, t[1], 1, T, t[2], t[3], 5, 4, 64, *t[4:7]), 7),
    "grouped_product": (lambda T, *t: brx.grouped_product(t[0], t[1], t[2], T, 8, 64, 64, t[3], 1, t[4], 1 << 20), 5),
    "grouped_dgrad": (lambda T, *t: brx.grouped_dgrad(t[0], t[1], t[2], T, 8, 64, 64, t[3], 1, t[4], 1 << 20), 5),
    "grouped_wgrad": (lambda T, *t: brx.grouped_wgrad(t[0], t[1], t[2], T, 8, 64, 64, t[3], 1, t[4], 1 << 20), 5),
    "block_norm": (lambda T, *t: brx.block_norm(_args(T=T, flags=31 - brx.GATE_TOKEN), *t[:9]), 9),
    "block_norm_backward": (lambda T, *t: brx.block_norm_backward(_args(T=T, flags=31 - brx.GATE_TOKEN), *t[:15], 1 << 20),
                            15),
}


@pytest.mark.parametrize("name", sorted(SIZES))
def test_binding_takes_no_host_tensor_among_addresses(name):
    """One tensor in host memory among raw addresses: refused by the binding wherever it stands, the workspace too."""
    call, n = SIZES[name]
    for i in range(n):
        t = [P] * n
        t[i] = torch.zeros(1 << 20, dtype=torch.uint8)
        with pytest.raises(brx.StrataError) as e:
            call(5, *t)
        assert e.value.status == EINVAL and "device memory" in str(e.value), (i, str(e.value))


@pytest.mark.parametrize("name", sorted(SIZES))
def test_binding_takes_no_size_past_32_bits(name):
    """A size that a C int32 would cut to a smaller, valid one."""
    call, n = SIZES[name]
    for T in (2**32, 2**32 + 5, 2**31):
        with pytest.raises(brx.StrataError) as e:
            call(T, *[P + 8] * n)      # misaligned addresses: nothing is launched either way
        assert e.value.status == EINVAL and "32 bits" in str(e.value)
    with pytest.raises(brx.StrataError):
        brx.sort_workspace_bytes(2**32 + 5, 4, 8)
    with pytest.raises(brx.StrataError):
        brx.grouped_workspace_bytes(2**32 + 5, 8, 64, 64)
    with pytest.raises(brx.StrataError):
        brx.grouped_product(P, P, P, 5, 8, 64, 64, P, 1, P, -1)


def test_binding_keeps_no_references():
    """A refused call, however far it got, leaves its arguments' reference counts as they were."""
    t, args = torch.zeros(20, dtype=torch.int32), _args(T=5, flags=31 - brx.GATE_TOKEN)
    count = sys.getrefcount(t), sys.getrefcount(args)
    for _ in range(50):
        for call in (lambda: brx.sort_picks(t, 5, 4, 8, None, None, None, None, None, 0),
                     lambda: brx.dispatch(P, 1, 5, 4, 64, "pos", P, 20),
                     lambda: brx.block_norm(args, P, P, t),
                     lambda: brx.block_norm(args, P, object()),
                     lambda: brx.block_norm_backward(args, P, P, P, P, ws_bytes=-1)):
            with pytest.raises(brx.StrataError):
                call()
    with pytest.raises(TypeError):
        brx.dispatch(P, 1, "T", 4, 64, P, P, 20)
    with pytest.raises(TypeError):
        brx.block_norm(object(), P, P)
    with pytest.raises(brx.StrataError):
        brx.block_norm(bytearray(8), P, P)
    assert (sys.getrefcount(t), sys.getrefcount(args)) == count


def test_binding_takes_no_stream_of_another_device():
    """Kernels would run on the stream's device, on memory of the tensors'.  The addresses are misaligned, so that
    the library refuses what the binding lets pass."""
    class Stream:
        def __init__(self, device_index, cuda_stream=0):
            self.device_index, self.cuda_stream = device_index, cuda_stream

    class Plain:
        cuda_stream = 0
    native, library = brx.ops._native, lib()
    if isinstance(native, brx.ops._Unloaded):
        native.bind   # loads the module
        native = brx.ops._native
    try:
        native.bind(tuple(ctypes.cast(getattr(library, f), ctypes.c_void_p).value for f in brx.ops._BOUND), brx.ops._raise,
                    brx.ops._elsewhere, lambda: 2, lambda: 2, lambda dev: 0)
        for stream, refused in ((Stream(1), True), (Stream(2), False), (Plain(), False), (0, False), (None, False)):
            with pytest.raises(brx.StrataError) as e:
                brx.dispatch(P + 8, 1, 5, 4, 64, P + 8, P + 8, 20, stream=stream)
            assert e.value.status == EINVAL and ("stream is on device 1, not 2" in str(e.value)) == refused, stream
        with pytest.raises(AttributeError):
            brx.dispatch(P + 8, 1, 5, 4, 64, P + 8, P + 8, 20, stream=object())
        with pytest.raises(TypeError):
            brx.dispatch(P + 8, 1, 5, 4, 64, P + 8, P + 8, 20, stream=Stream("one"))
    finally:
        brx.ops._native = brx.ops._Unloaded()   # bound anew at the next call


def test_the_package_imports_without_torch():
    """Shapes, the build and the host's entry points need no torch: the import neither loads it nor fails with it."""
    code = ("import sys, importlib.abc\n"
            "class No(importlib.abc.MetaPathFinder):\n"
            "    def find_spec(self, name, path=None, target=None):\n"
            "        if name.split('.')[0] == 'torch':\n"
            "            raise OSError('a torch whose libraries do not load')\n"
            "sys.meta_path.insert(0, No())\n"
            "import bit_routed_expert_amd as brx, bit_routed_expert_amd.build\n"
            "assert 'torch' not in sys.modules and brx.shape(8, 2, 64, 64, 3).n_experts == 8\n"
            "assert brx.block_norm_args(1, 8, 0, 0, 0, 0).d == 8\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr


def _leaf(*shape, seed):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed)).requires_grad_(True)


def test_reference_gradients_against_differences():
    """The 64-bit forms the kernels' gradients are held to are right: automatic
    differentiation against central differences, and the closed forms of the
    combine's gradients against both."""
    T, k, d, rows = 3, 4, 5, 11
    idx = torch.tensor([[0, 2, 2, -1], [-1, -1, -1, -1], [1, 0, 2, 9]])
    _, _, _, pos = R.sort(idx, 3)
    pos = torch.tensor(pos)
    ys, w, base = _leaf(rows, d, seed=1), _leaf(T, k, seed=2), _leaf(T, d, seed=3)
    f = lambda ys, w, base: R.combine(ys, pos, w, base, T, k)  # noqa: E731
    assert torch.autograd.gradcheck(f, (ys, w, base))
    dout = torch.randn(T, d, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    z = _leaf(T, k, seed=5)
    dw_, = torch.autograd.grad(f(ys, w, base), [w], dout)
    v, _ = R.picked(ys, pos, T, k)
    assert torch.allclose(dw_, (v * dout[:, None]).sum(2), atol=1e-12)
    g = torch.softmax(z, 1)
    dz_, = torch.autograd.grad(f(ys, g, base), [z], dout)
    dw = (v * dout[:, None]).sum(2)
    assert torch.allclose(dz_, g * (dw - (g * dw).sum(1, keepdim=True)), atol=1e-12)
    off = torch.tensor([0, 2, 2, 5])
    x, W = _leaf(6, 4, seed=6), _leaf(3, 5, 4, seed=7)
    assert torch.autograd.gradcheck(lambda x, W: R.grouped_product(x, W, off), (x, W))
    for gate in (None, _leaf(T, seed=8), _leaf(T, d, seed=9)):
        for sig in (False, True):
            x, y, gp, gq = _leaf(T, d, seed=10), _leaf(T, d, seed=11), _leaf(d, seed=12), _leaf(d, seed=13)

            def nf(x, y, gp, gq, *rest):
                r, u, _, _ = R.block_norm(x, y, rest[0] if rest else None, gp, gq, post=True, pre=True, sigmoid=sig,
                                          a=0.7, b=1.3, eps=1e-3)
                return r, u
            assert torch.autograd.gradcheck(nf, (x, y, gp, gq) + (() if gate is None else (gate,)))
