"""Plain 64-bit forms of the operators around the layer, on the CPU, with
error bounds for the kernels' 32-bit sums.

Bounds.  A sum of n terms in fp32 is off by at most (n - 1) 2^-24 of the sum
of the terms' magnitudes, whatever the order; a product or fma adds 2^-24 of
its magnitude.  A stored value is off by half a step of its type: 2^-8
(bf16) or 2^-24 (fp32) of its magnitude.
"""
from __future__ import annotations

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def check(got, ref, bound, what):
    """|got - ref| <= half a step of the stored value + the bound of its computation."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)}, not {tuple(ref.shape)}"
    assert bool(torch.isfinite(g).all()), f"{what}: not finite"
    h = HALF_STEP[got.dtype]
    tol = h * (ref.abs() + bound) + bound + 1e-37
    off = (g - ref).abs() - tol
    assert bool((off <= 0).all()), f"{what}: {int((off > 0).sum())} of {off.numel()} outside, worst by {float(off.max()):.3e}"


def sort(idx, E):
    """counts, offsets, perm, pos of the picks [T][k] (lists of ints)."""
    flat = idx.reshape(-1).tolist()
    kept = sorted((e, f) for f, e in enumerate(flat) if 0 <= e < E)
    counts, perm, pos = [0] * E, [-1] * len(flat), [-1] * len(flat)
    for s, (e, f) in enumerate(kept):
        counts[e] += 1
        perm[s] = f
        pos[f] = s
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    return counts, offsets, perm, pos


def picked(rows, pos, T, k):
    """rows[pos] as [T][k][d], zeros for skipped picks, and which picks are kept."""
    p = pos.view(T, k).long()
    has = (p >= 0) & (p < rows.shape[0])
    if rows.shape[0] == 0:
        return torch.zeros(T, k, rows.shape[1], dtype=rows.dtype), has
    v = rows[torch.where(has, p, torch.zeros_like(p))]
    return torch.where(has[..., None], v, torch.zeros_like(v)), has


def combine(ys, pos, w, base, T, k):
    v, has = picked(ys, pos, T, k)
    if w is not None:
        v = v * torch.where(has, w.view(T, k), torch.zeros_like(w.view(T, k)))[..., None]
    out = v.sum(1)
    return out if base is None else out + base


def segments(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def grouped_product(x, W, offsets):
    y = torch.zeros(x.shape[0], W.shape[1], dtype=x.dtype)
    for e, a, b in segments(offsets):
        y[a:b] = x[a:b] @ W[e].t()
    return y


def gate_factor(gate, sigmoid):
    if gate is None:
        return 1.0
    g = torch.sigmoid(gate) if sigmoid else gate
    return g[:, None] if g.dim() == 1 else g


def block_norm(x, y, gate, g_post, g_pre, *, post, pre, sigmoid, a, b, eps):
    """r, u, rstd_y, rstd_r (None where there is none)."""
    r, ry, u, rr = a * x, None, None, None
    if y is not None:
        n = y
        if post:
            ry = 1.0 / torch.sqrt((y * y).mean(1) + eps)
            n = n * ry[:, None] * (1.0 if g_post is None else g_post)
        r = r + b * gate_factor(gate, sigmoid) * n
    if pre:
        rr = 1.0 / torch.sqrt((r * r).mean(1) + eps)
        u = r * rr[:, None] * (1.0 if g_pre is None else g_pre)
    return r, u, ry, rr


def norm_rows(r, g, eps):
    return r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * (1.0 if g is None else g)
