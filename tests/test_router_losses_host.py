"""That the inputs of the router's gradient test show each of its terms."""
from __future__ import annotations

from tests import router_ref as Q


def test_every_term_shows_in_every_gradient():
    """A term that is missing moves each gradient by several times what roundings may."""
    case = Q.inputs()
    idx, pos = Q.picks(*case[:4])
    part = {t: Q.gradients(*case, idx, pos, t) for t in Q.TERMS}
    for term in ("picks", "balance", "z"):
        for name, one, whole in zip(("table", "Wr", "gain"), part[term], part["all"]):
            share = float(one.norm() / whole.norm())
            assert share >= 10 * Q.LIMIT, f"{term} is {share:.3f} of the gradient of {name}"
