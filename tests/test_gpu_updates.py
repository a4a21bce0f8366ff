"""Orthogonalised updates on the GPU, further: the ends of the types' ranges
and of X's two pieces, in each of the forms that a size selects."""
from __future__ import annotations

import pytest
import torch

from tests import train_ref as R
from tests.test_gpu_ops import BF, F32, gen
from tests.test_gpu_train import COEF, check, f32, run_orth, size_of

pytestmark = pytest.mark.gpu

# One matrix to a block; tiles of a step of 64 x 128, 128 square with four and with two buffers, 256 square; both ways.
FORMS = [(3, 72, 136), (3, 136, 72), (3, 200, 300), (3, 300, 200), (24, 250, 260), (24, 260, 250), (70, 200, 264), (70, 264, 200),
         (20, 1000, 1010), (20, 1010, 1000)]


@pytest.mark.parametrize("steps", [0, 1, 5])
@pytest.mark.parametrize("n,N,K", FORMS)
def test_orthogonalise_zeros_with_the_least_eps(n, N, K, steps):
    """size / (|G| + eps) is past fp32 for zeros and an eps below size / 3.4e38; the result is zeros all the same."""
    print(f"case orth zeros n={n} N={N} K={K} steps={steps}", flush=True)
    G = torch.randn(n, N, K, generator=gen(1))
    G[1] = 0
    G = G.cuda()
    want = run_orth(G, steps, COEF, 1.0, 1e-30)   # beside a norm of 100 or more no eps here shows
    assert bool(want.isfinite().all()) and not want[1].any() and bool(want[0].any())
    for eps in (torch.finfo(F32).tiny, 2.0 ** -149):
        assert torch.equal(run_orth(G, steps, COEF, 1.0, eps), want)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,N,K", FORMS)
def test_orthogonalise_at_the_ends_of_the_range(n, N, K, dt):
    """G and eps times a power of two is the same quotient, also where it takes the values to the type's smallest
    subnormal ones (exact: they are whole multiples of the least) or its largest, and 1 / (|G| + eps) out of fp32."""
    print(f"case orth range n={n} N={N} K={K} {dt}", flush=True)
    whole = 100 if dt is F32 else 1   # of bf16, whose least value is 2^-133, only such a small norm's inverse is past fp32
    G = torch.randint(-whole, whole + 1, (n, N, K), generator=gen(2)).float()
    want = run_orth(G.to(dt).cuda(), 5, COEF, 1.0, 1.0)
    assert bool(want.isfinite().all()) and bool(want.flatten(1).any(1).all())
    for s in (2.0 ** (-149 if dt is F32 else -133), 2.0 ** 121):
        g = (G.double() * s).to(dt)
        assert torch.equal(g.double(), G.double() * s)
        assert torch.equal(run_orth(g.cuda(), 5, COEF, 1.0, s), want), s


@pytest.mark.parametrize("n,N,K", FORMS)
def test_orthogonalise_keeps_values_far_below_the_largest(n, N, K):
    """One value of a matrix holds its norm, the others lie 2^-18 to 2^-27 below: fp16 keeps a few bits of them, and
    both pieces together the 22 that the bound of one step counts (X' = X here, so nothing else enters)."""
    print(f"case orth far values n={n} N={N} K={K}", flush=True)
    g = gen(3)
    G = torch.randn(n, N, K, generator=g) * 2.0 ** torch.randint(-27, -17, (n, N, K), generator=g)
    for e, at in enumerate(torch.randint(0, N * K, (n,), generator=g).tolist()):
        G[e].view(-1)[at] = -3.0 if e % 2 else 3.0
    c, eps = (1.0, 0.0, 0.0), f32(1e-7)
    got = run_orth(G.cuda(), 1, c, 1.0, 1e-7)
    for e in {0, n // 2, n - 1}:
        m = G[e:e + 1].cuda().double()
        check(got[e:e + 1], R.orthogonalise(m, 1, c, 1.0, eps), R.orth_one_step_bound(m, c, 1.0, eps, size_of(N, K)), f"matrix {e}")
