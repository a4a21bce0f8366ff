"""The limits of the orthogonalised updates' tests, on the CPU: the arithmetic
of either form stays within them, and each of the mistakes that could be
made in it, planted in its model, does not."""
from __future__ import annotations

import pytest

from tests import update_forms as F

SHAPES = [(2, 200, 300), (2, 300, 200), (2, 250, 260), (2, 60, 30), (1, 500, 520)]


@pytest.mark.parametrize("n,N,K", SHAPES)
def test_five_steps_are_within_the_limit(n, N, K):
    for kind in F.KINDS:
        G = F.update_case(n, N, K, kind)
        assert float(F.off_by(F.tiled(G), G).max()) <= F.LIMIT, kind


@pytest.mark.parametrize("mistake", F.MISTAKES)
@pytest.mark.parametrize("n,N,K", SHAPES)
def test_a_mistake_is_not(n, N, K, mistake):
    for kind in ("low", "bad"):
        G = F.update_case(n, N, K, kind)
        assert float(F.off_by(F.tiled(G, mistake=mistake), G).min()) > F.LIMIT, kind


@pytest.mark.parametrize("n,N,K", [(2, 31, 257), (2, 60, 30), (2, 61, 1000), (2, 16, 500)])
def test_one_block(n, N, K):
    for kind in F.KINDS:
        G = F.update_case(n, N, K, kind)
        assert float(F.off_by(F.one_block(G), G).max()) <= F.LIMIT, kind
    G, rank = F.update_case(n, N, K, "low"), min(N, K) // 4
    assert float(F.missing(F.one_block(G), rank).max()) <= 1.0
    apart = F.one_block(G, diagonal_apart=True)
    assert float(F.off_by(apart, G).min()) > F.LIMIT and float(F.missing(apart, rank).min()) > 1.0


@pytest.mark.parametrize("n,N,K", SHAPES)
def test_missing_directions_are_the_roundings_of_the_result(n, N, K):
    G, rank = F.update_case(n, N, K, "low"), min(N, K) // 4
    assert float(F.missing(F.tiled(G), rank).max()) <= 1.0
    for mistake in F.MISTAKES[:3]:
        assert float(F.missing(F.tiled(G, mistake=mistake), rank).min()) > 1.0, mistake


@pytest.mark.parametrize("c", F.POLYNOMIALS)
def test_three_steps_of_other_polynomials(c):
    for n, N, K in SHAPES:
        for kind in ("low", "bad"):
            G = F.update_case(n, N, K, kind)
            assert float(F.off_by(F.tiled(G, 3, None, c), G, 3, c).max()) <= F.LIMIT, (kind, N, K)
            for mistake in ("a step less", "zeros"):
                assert float(F.off_by(F.tiled(G, 3, mistake, c), G, 3, c).min()) > F.LIMIT, (kind, N, K, mistake)
