"""The ends of a training step without a GPU: refusals of every entry point,
workspace sizes, the binding's checks, and the reference gradients against
differences."""
from __future__ import annotations

import ctypes

import pytest
import torch

import bit_routed_expert_amd as brx
from tests import train_ref as R

EINVAL, EUNSUP, EWS, OK = brx.STRATA_EINVAL, brx.STRATA_EUNSUPPORTED, brx.STRATA_EWORKSPACE, brx.STRATA_OK
G = 1 << 36   # placeholders, far apart: validation fails before anything touches them


def lib():
    return brx.load_library()


def test_balance_refusals():
    f, ws = lib().strata_moe_balance, lib().strata_moe_balance_workspace_bytes
    need = ws(500, 4, 64)
    assert need > 0 and ws(5, 4, 64) > 0 and ws(0, 1, 1) > 0 and ws(1 << 23, 32, 1024) > 0

    def call(z=G, t=1, idx=2 * G, keep=None, T=500, k=4, E=64, losses=3 * G, counts=4 * G, prob=5 * G, lse=6 * G,
             tokens=7 * G, w=8 * G, wb=need):
        return f(z, t, idx, keep, T, k, E, losses, counts, prob, lse, tokens, w, wb, None)
    for bad in (dict(z=None), dict(z=G + 8), dict(t=2), dict(idx=None), dict(idx=G + 2), dict(T=-1), dict(k=0), dict(k=33),
                dict(E=0), dict(E=1025), dict(losses=None), dict(losses=G + 1), dict(counts=None), dict(counts=G + 2),
                dict(prob=G + 2), dict(lse=None), dict(lse=G + 2), dict(tokens=None), dict(tokens=G + 3), dict(w=None),
                dict(w=G + 4)):
        assert call(**bad) == EINVAL, bad
    assert call(wb=need - 1) == EWS and call(T=(1 << 23) + 1, wb=1 << 40) == EUNSUP
    for bad in ((-1, 4, 64), (5, 0, 64), (5, 33, 64), (5, 4, 0), (5, 4, 1025), ((1 << 23) + 1, 4, 64)):
        assert ws(*bad) == 0


def test_balance_backward_refusals():
    f = lib().strata_moe_balance_backward

    def call(z=G, t=1, idx=2 * G, keep=None, T=500, k=4, E=64, lse=3 * G, counts=4 * G, tokens=5 * G, dl=6 * G, dp=7 * G,
             dz=8 * G):
        return f(z, t, idx, keep, T, k, E, lse, counts, tokens, dl, dp, dz, None)
    for bad in (dict(z=None), dict(z=G + 4), dict(t=-1), dict(idx=None), dict(idx=G + 1), dict(T=-1), dict(k=0), dict(k=33),
                dict(E=0), dict(E=1025), dict(lse=None), dict(lse=G + 2), dict(counts=None), dict(tokens=None), dict(dl=None),
                dict(dl=G + 2), dict(dp=G + 2), dict(dz=None), dict(dz=G + 8)):
        assert call(**bad) == EINVAL, bad
    assert call(T=(1 << 23) + 1) == EUNSUP
    assert call(T=0, z=None, idx=None, lse=None, counts=None, tokens=None, dl=None, dp=None, dz=None) == OK


def test_embed_refusals():
    f, b, ws = lib().strata_embed, lib().strata_embed_backward, lib().strata_embed_backward_workspace_bytes

    def call(W=G, t=0, V=100, d=64, ids=2 * G, T=9, scale=1.0, out=3 * G, o=1):
        return f(W, t, V, d, ids, T, scale, out, o, None)
    for bad in (dict(W=None), dict(W=G + 2), dict(t=2), dict(o=3), dict(V=0), dict(d=0), dict(ids=None), dict(ids=G + 2),
                dict(T=-1), dict(out=None), dict(out=G + 8), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == EINVAL, bad
    assert call(T=(1 << 23) + 1) == EUNSUP and call(d=(1 << 24) + 1) == EUNSUP and call(V=(1 << 24) + 1) == EUNSUP
    assert call(T=0, W=None, ids=None, out=None) == OK
    need = ws(9, 100, 64)
    assert need > 0 and ws(0, 1, 1) > 0 and ws(1 << 22, (1 << 20) - 1, 2048) > 0
    for bad in ((-1, 100, 64), (9, 0, 64), (9, 100, 0), (9, 1 << 20, 64), ((1 << 22) + 1, 100, 64)):
        assert ws(*bad) == 0

    def back(dout=G, o=1, ids=2 * G, T=9, V=100, d=64, scale=1.0, dW=3 * G, t=0, flags=0, w=4 * G, wb=need):
        return b(dout, o, ids, T, V, d, scale, dW, t, flags, w, wb, None)
    for bad in (dict(dout=None), dict(dout=G + 4), dict(o=2), dict(t=-1), dict(ids=None), dict(ids=G + 2), dict(T=-1),
                dict(V=0), dict(d=0), dict(dW=None), dict(dW=G + 8), dict(flags=2), dict(w=None), dict(w=G + 8),
                dict(scale=float("inf"))):
        assert back(**bad) == EINVAL, bad
    assert back(wb=need - 1) == EWS and back(V=1 << 20, wb=1 << 40) == EUNSUP and back(T=(1 << 22) + 1, wb=1 << 40) == EUNSUP
    # the gradient, the ids and the workspace apart: slots and runs come from the latter two
    for bad in (dict(dW=4 * G), dict(dW=4 * G + need // 16 * 16 - 16), dict(ids=4 * G + 64), dict(dW=2 * G),
                dict(dW=2 * G - 100 * 64 * 2 + 16), dict(ids=3 * G + 4)):
        assert back(**bad) == EINVAL, bad


def test_vocab_loss_refusals():
    f, b = lib().strata_vocab_loss, lib().strata_vocab_loss_backward
    fw, bw = lib().strata_vocab_loss_workspace_bytes, lib().strata_vocab_loss_backward_workspace_bytes
    nf, nb = fw(50, 1000, 64), bw(50, 1000, 64)
    assert nf > 50 * 64 * 2 and nb > 50 * 64 * 2

    def call(h=G, W=2 * G, t=3 * G, T=50, V=1000, d=64, loss=4 * G, lse=5 * G, w=6 * G, wb=nf):
        return f(h, W, t, T, V, d, loss, lse, w, wb, None)
    for bad in (dict(h=None), dict(h=G + 8), dict(W=None), dict(W=G + 2), dict(t=None), dict(t=G + 2), dict(T=-1),
                dict(loss=None), dict(loss=G + 2), dict(lse=None), dict(lse=G + 1), dict(w=None), dict(w=G + 8),
                dict(w=3 * G), dict(w=4 * G), dict(lse=6 * G + 128), dict(loss=3 * G + 4), dict(lse=3 * G - 4)):
        assert call(**bad) == EINVAL, bad
    shapes = (dict(V=0), dict(V=(1 << 20) + 1), dict(d=0), dict(d=12), dict(d=16392), dict(T=(1 << 20) + 1),
              dict(T=1 << 20, d=16384), dict(T=1 << 19, V=(1 << 19) + 1))
    for bad in shapes:
        a = dict(T=50, V=1000, d=64) | bad
        assert call(**bad, wb=1 << 50) == EUNSUP and fw(a["T"], a["V"], a["d"]) == bw(a["T"], a["V"], a["d"]) == 0, bad
    assert call(wb=nf - 1) == EWS and call(T=0, h=None, W=None, t=None, loss=None, lse=None, w=None) == OK

    def back(h=G, W=2 * G, t=3 * G, T=50, V=1000, d=64, lse=4 * G, dl=5 * G, ds=6 * G, dh=7 * G, ht=0, dW=8 * G, wt=1, fl=0,
             w=9 * G, wb=nb):
        return b(h, W, t, T, V, d, lse, dl, ds, dh, ht, dW, wt, fl, w, wb, None)
    for bad in (dict(h=None), dict(h=G + 2), dict(W=None), dict(t=None), dict(t=G + 1), dict(T=-1), dict(lse=None),
                dict(lse=G + 2), dict(dl=None), dict(dl=G + 2), dict(ds=G + 2), dict(dh=G + 4), dict(ht=2), dict(dW=G + 2),
                dict(wt=5), dict(fl=2), dict(w=None), dict(w=G + 8), dict(w=3 * G), dict(dh=9 * G), dict(dW=9 * G + 256),
                dict(dW=3 * G), dict(t=7 * G + 4)):
        assert back(**bad) == EINVAL, bad
    for bad in shapes:
        assert back(**bad, wb=1 << 50) == EUNSUP, bad
    assert back(wb=nb - 1) == EWS
    assert back(dh=None, dW=None, ht=9, wt=9) == OK                       # nothing asked for
    assert back(T=0, h=None, W=None, t=None, lse=None, dl=None, ds=None, dh=None, dW=None, w=None) == OK
    assert back(T=0, fl=1) == OK                                          # adds nothing


def test_orthogonalise_refusals():
    f, ws = lib().strata_orthogonalise, lib().strata_orthogonalise_workspace_bytes
    need = ws(3, 40, 72)
    assert need > 3 * 40 * 72 * 6 and ws(0, 8, 8) > 0
    good = (3.4445, -4.775, 2.0315)

    def call(g=G, t=1, n=3, N=40, K=72, steps=5, c=good, scale=1.0, eps=1e-7, out=2 * G, w=3 * G, wb=need):
        return f(g, t, n, N, K, steps, None if c is None else (ctypes.c_float * 3)(*c), scale, eps, out, w, wb, None)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(g=None), dict(g=G + 8), dict(t=2), dict(n=-1), dict(N=0), dict(K=0), dict(steps=-1), dict(steps=33),
                dict(c=None), dict(c=(nan, 1, 1)), dict(c=(1, inf, 1)), dict(c=(1, 1, -inf)), dict(scale=nan), dict(scale=inf),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(out=None), dict(out=G + 2), dict(w=None),
                dict(w=G + 8), dict(out=G), dict(out=G + 16), dict(t=0, out=G + 16), dict(t=0, out=G - 16), dict(steps=0, out=G)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(N=16385), dict(K=16385), dict(n=1025), dict(n=1024, N=16384, K=16384)):
        a = dict(n=3, N=40, K=72) | bad
        assert call(**bad, wb=1 << 50) == EUNSUP and ws(a["n"], a["N"], a["K"]) == 0, bad
    assert call(wb=need - 1) == EWS and call(n=0, g=None, out=None, w=None) == OK


CALLS = {   # every entry point with T tokens (or matrices), and how many tensors it takes
    "balance_loss": (lambda T, *t: brx.balance_loss(t[0], 1, t[1], T, 4, 8, *t[2:7], 256, prob=t[7], keep=t[8]), 9),
    "balance_loss_backward": (lambda T, *t: brx.balance_loss_backward(t[0], 1, t[1], T, 4, 8, *t[2:7], keep=t[7],
                                                                      dpicks=t[8]), 9),
    "embed": (lambda T, *t: brx.embed(t[0], 1, 100, 64, t[1], T, 1.0, t[2], 1), 3),
    "embed_backward": (lambda T, *t: brx.embed_backward(t[0], 1, t[1], T, 100, 64, 1.0, t[2], 1, t[3], 1 << 20), 4),
    "vocab_loss": (lambda T, *t: brx.vocab_loss(t[0], t[1], t[2], T, 100, 64, t[3], t[4], t[5], 1 << 20), 6),
    "vocab_loss_backward": (lambda T, *t: brx.vocab_loss_backward(t[0], t[1], t[2], T, 100, 64, t[3], t[4], t[5], 1 << 20,
                                                                  dlse=t[6], dh=t[7], dhdtype=1, dW=t[8], dwdtype=1), 9),
    "orthogonalise": (lambda T, *t: brx.orthogonalise(t[0], 1, T, 8, 64, t[1], t[2], 1 << 20), 3),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_binding_takes_no_host_tensor_and_no_size_past_32_bits(name):
    call, n = CALLS[name]
    for i in range(n):
        t = [0x10000] * n
        t[i] = torch.zeros(1 << 20, dtype=torch.uint8)
        with pytest.raises(brx.StrataError) as e:
            call(5, *t)
        assert e.value.status == EINVAL and "device memory" in str(e.value), (i, str(e.value))
    for T in (2**31, 2**32 + 5, -1):
        with pytest.raises(brx.StrataError) as e:
            call(T, *[0x10008] * n)
        assert e.value.status == EINVAL and "32 bits" in str(e.value)


def test_binding_numbers_and_workspace_sizes():
    for f, bad in ((brx.balance_loss_workspace_bytes, (5, 4, 0)), (brx.embed_backward_workspace_bytes, (5, 1 << 20, 64)),
                   (brx.vocab_loss_workspace_bytes, (5, 100, 12)), (brx.vocab_loss_backward_workspace_bytes, (5, 0, 64)),
                   (brx.orthogonalise_workspace_bytes, (5, 0, 64)), (brx.vocab_loss_workspace_bytes, (2**32 + 5, 100, 64))):
        with pytest.raises(brx.StrataError):
            f(*bad)
    P = 0x10008
    with pytest.raises(TypeError):
        brx.embed(P, 1, 100, 64, P, 5, "one", P, 1)
    with pytest.raises(TypeError):
        brx.orthogonalise(P, 1, 5, 8, 64, P, P, 1 << 20, coefficients=(1.0, None, 2.0))
    with pytest.raises(ValueError):
        brx.orthogonalise(P, 1, 5, 8, 64, P, P, 1 << 20, coefficients=(1.0, 2.0))
    with pytest.raises(brx.StrataError) as e:
        brx.orthogonalise(P, 1, 5, 8, 64, P, P, -1)
    assert e.value.status == EINVAL


def _leaf(*shape, seed):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed)).requires_grad_(True)


def test_reference_gradients_against_differences():
    """Automatic differentiation of the 64-bit forms against differences, and the closed forms of the header against it."""
    T, k, E = 6, 3, 5
    idx = torch.tensor([[0, 2, 2], [1, -1, 4], [3, 3, 3], [0, 1, 9], [4, 2, 0], [1, 1, 2]])
    keep = torch.tensor([1, 1, 0, 1, 1, 1])
    z = _leaf(T, E, seed=1)
    assert torch.autograd.gradcheck(lambda z: R.balance(z, idx, keep, E)[0], (z,))
    losses, counts, prob, lse, n = R.balance(z, idx, keep, E)
    dl = torch.tensor([0.7, 0.3], dtype=torch.float64)
    want, = torch.autograd.grad((losses * dl).sum(), z)
    p = torch.softmax(z, 1).detach()
    g = dl[0] * E * counts / (n * n * k)
    dz = p * (g - (p * g).sum(1, keepdim=True) + (2 * dl[1] * lse.detach() / n)[:, None]) * keep[:, None]
    assert torch.allclose(dz, want, atol=1e-12) and n == 5 and abs(float(losses[0].detach()) - E * float((counts * prob.detach()).sum()) / 15) < 1e-12
    W, h = _leaf(7, 4, seed=2), _leaf(5, 4, seed=3)
    t = torch.tensor([0, 6, -1, 3, 7])
    assert torch.autograd.gradcheck(lambda h, W: R.vocab(h, W, t)[:2], (h, W))
    loss, lse, ok = R.vocab(h, W, t)
    up, un = torch.randn(5, dtype=torch.float64), torch.randn(5, dtype=torch.float64)
    gh, gW = torch.autograd.grad((loss * up + lse * un).sum(), (h, W))
    dh, _, dW, _ = R.vocab_grads(h.detach(), W.detach(), t, lse.detach(), up, un, (0.0, 0.0))
    assert ok.tolist() == [True, True, False, True, False]
    assert torch.allclose(dh, gh, atol=1e-12) and torch.allclose(dW, gW, atol=1e-12)
    ids = torch.tensor([1, 6, 1, -1, 7, 0])
    assert torch.autograd.gradcheck(lambda W: R.embed(W, ids, 1.5), (W,))
    out = torch.randn(6, 4, dtype=torch.float64)
    ge, = torch.autograd.grad((R.embed(W, ids, 1.5) * out).sum(), W)
    assert torch.allclose(R.embed_backward(out, ids, 7, 1.5)[0], ge, atol=1e-12)


def test_reference_orthogonalisation():
    """The polynomial acts on the singular values; from either side alike."""
    G = torch.randn(2, 5, 9, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    c = (3.4445, -4.775, 2.0315)
    u, s, v = torch.linalg.svd(G, full_matrices=False)
    s = s / s.norm(dim=1, keepdim=True)
    for _ in range(5):
        s = c[0] * s + c[1] * s ** 3 + c[2] * s ** 5
    got = R.orthogonalise(G, 5, c, 2.0, 1e-12)
    assert torch.allclose(got, 2.0 * (u * s[:, None]) @ v, atol=1e-9)
    assert torch.allclose(R.orthogonalise(G.transpose(1, 2), 5, c, 2.0, 1e-12), got.transpose(1, 2), atol=1e-9)
