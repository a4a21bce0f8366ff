"""Inputs and limits of the orthogonalised updates of several steps, and
models of the two forms' arithmetic in which mistakes can be planted."""
from __future__ import annotations

import math

import torch

from tests import train_ref as R

COEF = tuple(float(torch.tensor(v)) for v in (3.4445, -4.7750, 2.0315))
EPS = float(torch.tensor(1e-7))

# How far five steps may be off in 2-norm, relative to the result.  The output's rounding to bf16 is at most 2^-8 of each
# value, over many values 2^-8 / sqrt(3) (evenly spread within half a step) = 2.3e-3.  A step's operands A, B and X are off
# by 2^-11 / sqrt(3) each, times |b| s^2 + |c| s^4 = 6.8 at most (singular values s up to about 1) and independent of each
# other: 2^-11 * 6.8 = 3.3e-3 if all of it met off the diagonals, which are known in fp32.  Both in squares are 4.0e-3, and
# 2^-8 = 3.9e-3; what an earlier step left is taken on by a slope of about 1.  Matrices of fewer than 500 values, whose
# roundings need not average, are left out.
LIMIT = 2.0 ** -8

# Polynomials of the same kind, b and c no larger; three steps.
POLYNOMIALS = [tuple(float(torch.tensor(v)) for v in c) for c in ((1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (2.0, -1.2, 0.2), (1.875, -1.25, 0.375))]

KINDS = ("full", "low", "bad")


def update_case(n, N, K, kind, seed=1):
    """fp32 matrices: a few strong directions in a full-rank rest; a quarter of the directions and no others;
    singular values spread evenly over 13 powers of two."""
    g = torch.Generator().manual_seed(seed)
    side = min(N, K)
    if kind == "bad":
        q = [torch.linalg.qr(torch.randn(n, m, side, generator=g, dtype=torch.float64)).Q for m in (N, K)]
        s = 2.0 ** -torch.linspace(0, 12, side, dtype=torch.float64)
        return (torch.bmm(q[0] * s, q[1].transpose(1, 2).contiguous())).float()
    r = max(1, side // (4 if kind == "low" else 8))
    low = torch.bmm(torch.randn(n, N, r, generator=g), torch.randn(n, r, K, generator=g))
    return low if kind == "low" else torch.randn(n, N, K, generator=g) + low


def off_by(got, G, steps=5, coefficients=COEF):
    """Each matrix's error in 2-norm over its result's."""
    ref = R.orthogonalise(G.double(), steps, coefficients, 1.0, EPS)
    return (got.double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)


def missing(got, rank):
    """The largest singular value behind `rank` of a result that has no more, over what the rounding of its values to
    bf16 makes of it: a matrix of independent values of 2^-8 / sqrt(3) times theirs has singular values up to
    sqrt(N) + sqrt(K) times that; without the sqrt(3) there is room for the last step's X in one piece, 3.4 * 2^-11."""
    N, K = got.shape[-2:]
    s = torch.linalg.svdvals(got.double())
    return s[:, rank] / (2.0 ** -8 * (N ** 0.5 + K ** 0.5) * got.double().square().mean((1, 2)).sqrt())


def size_of(N, K):
    return 2.0 ** round(0.5 * math.log2(max(N, K)))


MISTAKES = ("no low piece", "low piece of the start alone", "low piece beside its place", "bf16 operands", "a step less", "zeros")


def tiled(G, steps=5, mistake=None, coefficients=COEF):
    """The tiled form: fp16 operands, X = hi + lo, diagonals in fp32; sums in 64 bits."""
    half = lambda v: v.to(torch.bfloat16 if mistake == "bf16 operands" else torch.float16).double()  # noqa: E731
    T = lambda v: v.transpose(-1, -2)  # noqa: E731
    a, b, c = coefficients
    n, N, K = G.shape
    s = size_of(N, K)
    x = G.double() / (G.double().flatten(1).norm(dim=1)[:, None, None] + EPS) * s
    x = T(x) if N > K else x
    eye = torch.eye(x.shape[1], dtype=torch.float64)
    if mistake == "a step less":
        steps -= 1
    for i in range(steps):
        hi = half(x)
        lo = half((x - hi) * 2.0 ** 11) * 2.0 ** -11
        if mistake == "no low piece" or (mistake == "low piece of the start alone" and i):
            lo = torch.zeros_like(lo)
        if mistake == "low piece beside its place":
            lo = lo.roll(4, -1)
        A = torch.bmm(hi, T(hi)) / s ** 2
        Ah = half(A)
        dA = (A - Ah) * eye
        B = b * Ah + c * torch.bmm(Ah, Ah)
        Bh = half(B)
        dB = (b + 2 * c * Ah) * dA + (B - Bh) * eye
        x = a * hi + torch.bmm(Bh + dB, hi)
        if i + 1 < steps or steps == 1:
            x = x + a * lo
    x = torch.zeros_like(x) if mistake == "zeros" else x / s
    return (T(x) if N > K else x).float().to(torch.bfloat16)


def one_block(G, steps=5, diagonal_apart=False):
    """The one-block form: X in fp32, its fp16 copy the operand, diagonals in fp32; B's diagonal goes with the copy but
    for the last two steps (diagonal_apart: never, the mistake)."""
    half = lambda v: v.to(torch.float16).double()  # noqa: E731
    T = lambda v: v.transpose(-1, -2)  # noqa: E731
    a, b, c = COEF
    n, N, K = G.shape
    s = size_of(N, K)
    x = (G.double() / (G.double().flatten(1).norm(dim=1)[:, None, None] + EPS) * s).float().double()
    x = T(x) if N > K else x
    off = 1 - torch.eye(x.shape[1], dtype=torch.float64)
    for i in range(steps):
        hi = half(x)
        A = torch.bmm(hi, T(hi)) / s ** 2
        d = A.diagonal(dim1=-2, dim2=-1)
        Ah = half(A * off)
        S = torch.bmm(Ah, Ah)
        dB = b * d + c * (d * d + S.diagonal(dim1=-2, dim2=-1))
        Bh = half((b * A + c * (S + (d[:, :, None] + d[:, None]) * A)) * off)
        own = x if diagonal_apart or i + 2 >= steps else hi
        x = (a * x + dB[:, :, None] * own + torch.bmm(Bh, hi)).float().double()
    x = x / s
    return (T(x) if N > K else x).float().to(torch.bfloat16)
