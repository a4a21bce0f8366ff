"""Plain 64-bit forms of the ends of a training step, with error bounds for
the kernels' arithmetic (see ops_ref for the bounds of fp32 sums).

exp and log of fp32 values are taken to be off by 4 U of the result (the
hardware's 1 ulp, the argument's scaling and the correction around it), and an
exponential additionally by 2 U |argument| (two roundings of the argument)."""
from __future__ import annotations

import torch

from tests.ops_ref import U

HALF = 2.0 ** -11   # half a step of fp16, relative
HALF_LEAST = 2.0 ** -25   # half the smallest step of fp16


# ---------------------------------------------------------------- balance

def counted(z, keep):
    """Tokens that count: kept ones with a logit that is not -inf."""
    on = torch.ones(z.shape[0], dtype=torch.bool) if keep is None else keep.bool()
    return on & ~(z == float("-inf")).all(1)


def balance(z, idx, keep, E):
    """losses, counts, prob, lse, n; z may require a gradient."""
    T, k = idx.shape
    on = counted(z.detach(), keep)
    n = int(on.sum())
    counts = torch.zeros(E, dtype=torch.int64)
    for e in idx[on].reshape(-1).tolist():
        if 0 <= e < E:
            counts[e] += 1
    lse = torch.zeros(T, dtype=torch.float64)
    if n == 0:
        return torch.zeros(2, dtype=torch.float64), counts, torch.zeros(E, dtype=torch.float64), lse, 0
    zo = z[on]
    l = torch.logsumexp(zo, 1)
    p = torch.softmax(zo, 1)
    lse = lse.index_put((on.nonzero().flatten(),), l)
    prob = p.mean(0)
    return torch.stack([E * (counts.double() / (n * k) * prob).sum(), l.square().mean()]), counts, prob, lse, n


# ------------------------------------------------------------- embedding

def embed(W, ids, scale):
    V = W.shape[0]
    ok = (ids >= 0) & (ids < V)
    v = W[torch.where(ok, ids, torch.zeros_like(ids)).long()] * scale
    return torch.where(ok[:, None], v, torch.zeros_like(v))


def embed_backward(dout, ids, V, scale):
    """The gradient, the sums of magnitudes, and how many tokens each row has."""
    ok = ((ids >= 0) & (ids < V)).nonzero().flatten()
    at = ids[ok].long()
    dW, mag = torch.zeros(V, dout.shape[1], dtype=torch.float64, device=dout.device), \
        torch.zeros(V, dout.shape[1], dtype=torch.float64, device=dout.device)
    dW.index_add_(0, at, dout[ok])
    mag.index_add_(0, at, dout[ok].abs())
    n = torch.zeros(V, dtype=torch.float64, device=dout.device).index_add_(0, at, torch.ones(len(ok), dtype=torch.float64,
                                                                                             device=dout.device))
    return dW * scale, mag * abs(scale), n


# ------------------------------------------------------- vocabulary loss

def vocab(h, W, targets):
    """loss and lse (zeros without a target) and which tokens have one; h and W may require gradients."""
    V = W.shape[0]
    ok = (targets >= 0) & (targets < V)
    at = ok.nonzero().flatten()
    z = h[at] @ W.t()
    l = torch.logsumexp(z, 1)
    T = h.shape[0]
    zero = torch.zeros(T, dtype=h.dtype, device=h.device)
    lse = zero.index_put((at,), l)
    loss = zero.index_put((at,), l - z.gather(1, targets[at].long()[:, None])[:, 0])
    return loss, lse, ok


def vocab_bounds(h, W, targets):
    """Bounds of loss and lse: logits are fp32 sums of d exact products (2 d U of
    their magnitudes), V exponentials added."""
    V, d = W.shape
    z, m = h @ W.t(), h.abs() @ W.t().abs()
    dz = 2 * d * U * m
    p = torch.softmax(z, 1)
    x = (z - z.max(1, keepdim=True).values).abs()
    l = torch.logsumexp(z, 1)
    # a sum over tiles takes each term through up to three rescalings by exponentials
    b = (p * (dz + (8 * x + 16) * U)).sum(1) + (V + 8) * U + 4 * U * l.abs()
    t = targets.clamp(0, V - 1).long()[:, None]
    return b + dz.gather(1, t)[:, 0] + 2 * U * (l.abs() + z.gather(1, t)[:, 0].abs()), b


def vocab_grads(h, W, targets, lse, dloss, dlse, piece):
    """dh and dW from the stored lse, with bounds; piece: relative rounding of dz
    as it enters the products (2^-8 in one bf16 piece, 2^-16 in two), a pair for
    (dh, dW)."""
    V, d = W.shape
    T = h.shape[0]
    ok = ((targets >= 0) & (targets < V)).nonzero().flatten()
    hs, t = h[ok], targets[ok].long()
    z = hs @ W.t()
    dzz = 2 * d * U * (hs.abs() @ W.t().abs())
    up = dloss[ok] + (0 if dlse is None else dlse[ok])
    q = torch.exp(z - lse[ok][:, None]) * up[:, None]
    e = q.abs() * (dzz + (2 * (z - lse[ok][:, None]).abs() + 8) * U)
    at = torch.arange(len(ok), device=h.device)
    g = q.clone()
    g[at, t] -= dloss[ok]
    e[at, t] += U * (q[at, t].abs() + dloss[ok].abs())
    out = []
    for p, A, B, n in ((piece[0], g, W, V), (piece[1], g.t(), hs, len(ok))):
        E = e if A is g else e.t()
        ref = A @ B
        bound = (E + p * (A.abs() + E) + 1e-38) @ B.abs() + 4 * n * U * (A.abs() @ B.abs())
        out += [ref, bound]
    dh = torch.zeros(T, d, dtype=torch.float64, device=h.device)
    bh = torch.zeros_like(dh)
    dh[ok], bh[ok] = out[0], out[1]
    return dh, bh, out[2], out[3]


# ------------------------------------------------------ orthogonalisation

def orth_step(X, a, b, c):
    A = X @ X.transpose(-1, -2)
    return a * X + (b * A + c * A @ A) @ X


def orthogonalise(G, steps, coefficients, scale, eps):
    X = G / (G.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    X = X.transpose(-1, -2) if G.shape[-2] > G.shape[-1] else X
    for _ in range(steps):
        X = orth_step(X, *coefficients)
    return scale * (X.transpose(-1, -2) if G.shape[-2] > G.shape[-1] else X)


def orth_one_step_bound(G, coefficients, scale, eps, size):
    """Elementwise bound of one step from the magnitudes: operands rounded to
    fp16 once (A from rounded X), sums of n terms in fp32, X in 22 bits."""
    a, b, c = (abs(v) for v in coefficients)
    X = (G / (G.square().sum((-2, -1), keepdim=True).sqrt() + eps)).abs()
    tall = G.shape[-2] > G.shape[-1]
    X = X.transpose(-1, -2) if tall else X
    n, K = X.shape[-2:]
    xh = HALF * X + HALF_LEAST / size                      # X against its first piece
    xx = 2.0 ** -21 * X + 2 * HALF_LEAST / size * HALF     # X against both
    T = lambda M: M.transpose(-1, -2)  # noqa: E731
    A = (X + xh) @ T(X + xh)
    dA = X @ T(xh) + xh @ T(X) + xh @ T(xh)
    dA = dA + (2 * K + 4) * U * A + HALF * A + HALF_LEAST
    A2 = A @ A
    dB = b * dA + c * (A @ dA + dA @ A + dA @ dA) + (2 * n + 8) * U * (b * A + c * A2)
    B = b * A + c * A2
    dB = dB + HALF * (B + dB) + HALF_LEAST
    dX = dB @ (X + xh) + B @ xh + (2 * n + 8) * U * ((B + dB) @ (X + xh) + a * X) + a * xx
    return abs(scale) * (T(dX) if tall else dX)


def orth_norm_bound(G, steps, coefficients, eps, size):
    """Bound of the result's error in Frobenius norm (scale 1), per matrix: each
    step's own error from the norms, taken to the end by the largest divided
    difference of the remaining polynomial over the matrix's singular values
    (first order; the second is the square of what comes out)."""
    a, b, c = coefficients
    out = []
    for g in G:
        X = g / (g.norm() + eps)
        n, K = min(X.shape), max(X.shape)
        s = torch.linalg.svdvals(X)
        f = lambda v: a * v + b * v ** 3 + c * v ** 5  # noqa: E731
        total = 0.0
        for i in range(steps):
            F, S = float(s.norm()), float(s.max())
            # a rounding's matrix is at most HALF of the rounded one in Frobenius norm
            xh = HALF * F + HALF_LEAST / size * (n * K) ** 0.5
            A = F * S
            dA = 2 * S * xh + HALF * A + HALF_LEAST * n + 2 * K * U * F * F
            spec = float((b * s ** 2 + c * s ** 4).abs().max())
            dB = (abs(b) + 2 * abs(c) * S * S) * dA + HALF * (abs(b) + abs(c) * S * S) * A + HALF_LEAST * n + 2 * n * U * A * A
            # X has 22 bits but ahead of the last of several steps, which takes its first piece
            kept = xh if steps > 1 and i == steps - 1 else 2.0 ** -21 * F
            own = dB * S + spec * xh + abs(a) * kept + 2 * n * U * F * (abs(b) + abs(c) * S * S) * S
            s1 = f(s)
            v, w = torch.cat([s1, torch.zeros(1, dtype=s.dtype)]), torch.cat([s1, torch.zeros(1, dtype=s.dtype)])
            d = torch.ones_like(v)
            for _ in range(i + 1, steps):
                d = d * (a + 3 * b * w ** 2 + 5 * c * w ** 4)
                w = f(w)
            dif, sm = v[:, None] - v[None], v[:, None] + v[None]
            near = dif.abs() < 1e-6
            minus = torch.where(near, d[:, None].expand_as(dif).abs(), ((w[:, None] - w[None]) / torch.where(near, torch.ones_like(dif), dif)).abs())
            small = sm.abs() < 1e-6
            plus = torch.where(small, d[:, None].expand_as(sm).abs(), ((w[:, None] + w[None]) / torch.where(small, torch.ones_like(sm), sm)).abs())
            total += own * float(torch.maximum(minus, plus).max())
            s = s1
        out.append(total)
    return torch.tensor(out, dtype=torch.float64)
