"""A router's gradient from all that it learns from, in 64 bits: token rows ->
norm -> router -> picks' weights of fixed rows, their product with fixed
gradients, and the router's balance and z losses."""
from __future__ import annotations

import torch

from tests import ops_ref as O
from tests import train_ref as R

T, V, D, E, K, PAD = 150, 300, 256, 32, 4, 25   # the last PAD tokens are padding
SCALE = 3.0

# Between the operators u and du are bf16.  u enters the logits, the picks' weights and the router's gradient, du its
# rows': four roundings on a path, each at most 2^-8 of its value.
LIMIT = 4 * 2.0 ** -8

# What the loss is made of: the rows' weights, the balance loss, the z loss; factors that make their gradients alike in size.
TERMS = {"picks": (1.0, 0.0, 0.0), "balance": (0.0, 40.0, 0.0), "z": (0.0, 0.0, 1.5), "all": (1.0, 40.0, 1.5)}


def inputs():
    g = torch.Generator().manual_seed(7)
    r = lambda *s, by=1.0: torch.randn(*s, generator=g) * by  # noqa: E731
    table = r(V, D, by=0.3).to(torch.bfloat16)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    ids[T - PAD:] = -1
    # unlike experts, so that the balance loss has a slope
    Wr = r(E, D, by=D ** -0.5) + r(1, D, by=D ** -0.5) * torch.linspace(-1, 1, E)[:, None]
    ys = r(T * K, D).to(torch.bfloat16)
    dy = r(T, D, by=1.0 / T)
    gain = 1 + 0.1 * r(D)
    return table, ids, Wr, gain, ys, dy


def gradients(table, ids, Wr, gain, ys, dy, idx, pos, term):
    """Of the table, the router and the gain; idx and pos [T][K], -1: dropped."""
    w = TERMS[term]
    L = [v.double().clone().requires_grad_(True) for v in (table, Wr, gain)]
    on = ids >= 0
    x = L[0][ids[on].long()] * SCALE
    z = O.norm_rows(x, L[2], float(torch.tensor(1e-6))) @ L[1].t()
    i = idx[on].long()
    p = torch.softmax(z.gather(1, i), 1)
    y = (p[:, :, None] * ys.double()[pos[on].long()]).sum(1)
    losses = R.balance(z, i, None, E)[0]
    total = w[0] * (y * dy[on].double()).sum() + w[1] * losses[0] + w[2] * losses[1]
    return torch.autograd.grad(total, L)


def picks(table, ids, Wr, gain):
    """The router's picks in 64 bits, and their slots sorted by expert."""
    x = table.double()[ids.clamp_min(0).long()] * SCALE
    idx = torch.topk(O.norm_rows(x, gain.double(), 1e-6) @ Wr.double().t(), K, 1).indices
    idx[ids < 0] = -1
    return idx, torch.tensor(O.sort(idx, E)[3]).view(T, K)
