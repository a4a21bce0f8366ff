"""Orthogonalised updates on the GPU, further: the ends of the types' ranges
and of X's two pieces, several steps against 64 bits within limits that the
mistakes planted in update_forms' model fail, infinities and NaN, in each of
the forms that a size selects."""
from __future__ import annotations

import pytest
import torch

from tests import train_ref as R
from tests import update_forms as F
from tests.test_gpu_ops import BF, F32, gen, rand
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


# The one-block form's other shapes, and sizes that leave parts of tiles, waves and 16-byte pieces.
MORE = [(2, 31, 257), (2, 257, 31), (2, 64, 500), (2, 61, 1000), (2, 128, 256), (2, 97, 383), (2, 383, 97), (2, 129, 127), (2, 130, 61),
        (1, 257, 513), (40, 520, 264), (2, 136, 1000), (1, 1000, 1000), (1, 65, 1030)]


def few_of(n, N, K, kind, dt):
    """n matrices, three of them different ones."""
    G = F.update_case(min(n, 3), N, K, kind).to(dt)
    return G.cuda()[torch.arange(n) % len(G)].contiguous()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kind", F.KINDS)
@pytest.mark.parametrize("n,N,K", FORMS + MORE)
def test_orthogonalise_five_steps(n, N, K, kind, dt):
    print(f"case orth five steps n={n} N={N} K={K} {kind} {dt}", flush=True)
    G = few_of(n, N, K, kind, dt)
    got = run_orth(G, 5, F.COEF, 1.0, F.EPS)
    off = F.off_by(got[:3], G[:3])
    print(f"  off {float(off.max()):.2e}", flush=True)
    assert bool((off <= F.LIMIT).all())
    assert torch.equal(got, got[torch.arange(n) % min(n, 3)])


@pytest.mark.parametrize("n,N,K", FORMS + MORE)
def test_orthogonalise_makes_no_directions(n, N, K):
    """What a gradient of few directions lacks stays missing but for the rounding of the result."""
    G = few_of(n, N, K, "low", F32)
    got = run_orth(G, 5, F.COEF, 1.0, F.EPS)
    made = F.missing(got[:3].cpu(), min(N, K) // 4)
    assert bool((made <= 1.0).all()), made


@pytest.mark.parametrize("c", F.POLYNOMIALS)
@pytest.mark.parametrize("n,N,K", FORMS)
def test_orthogonalise_three_steps_of_other_polynomials(n, N, K, c):
    for kind in ("low", "bad"):
        G = few_of(n, N, K, kind, F32)
        off = F.off_by(run_orth(G, 3, c, 1.0, F.EPS)[:3], G[:3], 3, c)
        assert bool((off <= F.LIMIT).all()), (kind, off)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("n,N,K", [(6, *f[1:]) if f[0] < 6 else f for f in FORMS])
def test_orthogonalise_infinities_stay_in_their_matrix(n, N, K, value):
    """Operands of a tile go on into the row behind, and a matrix' last row into nothing: none reaches a neighbour."""
    print(f"case orth {value} n={n} N={N} K={K}", flush=True)
    G = rand(n, N, K, seed=3).cuda()
    places = {1: (0, 0), 3: (N - 1, K - 1), n - 1: (N // 2, K - 1)}
    for e in places:
        G[e] = 0
    want = run_orth(G, 5, F.COEF, 1.0, F.EPS).clone()
    for e, (i, j) in places.items():
        G[e] = rand(N, K, seed=4).cuda()
        G[e, i, j] = value
    got = run_orth(G, 5, F.COEF, 1.0, F.EPS)
    for e in range(n):
        if e in places:
            assert not bool(got[e].isfinite().all()) and not want[e].any()
        else:
            assert torch.equal(got[e], want[e]) and bool(want[e].isfinite().all())
