"""The router's gradient from all that it learns from, through the library:
rows -> norm -> route -> sort -> combine, the balance losses, and back to the
router, the norm's gain and the table; each loss alone and all joined."""
from __future__ import annotations

import pytest
import torch

import bit_routed_expert_amd as brx
from tests import router_ref as Q
from tests.test_gpu_ops import BF, F32, ws_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("term", Q.TERMS)
def test_router_gradient_of_each_loss(term):
    T, V, d, E, k, n = Q.T, Q.V, Q.D, Q.E, Q.K, Q.T * Q.K
    host = Q.inputs()
    table, ids, Wr, gain, ys, dy = (v.cuda() for v in host)
    w = Q.TERMS[term]
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    keep = ids >= 0
    x, u, rstd = e(T, d), e(T, d, dt=BF), e(T)
    brx.embed(table, 0, V, d, ids, T, Q.SCALE, x, 1)
    args = brx.block_norm_args(T, d, 1, 0, 0, brx.PRE_NORM)
    brx.block_norm(args, x, None, g_pre=gain, u=u, rstd_r=rstd)
    sh = brx.shape(E, k, d, 128, 3)
    nb = brx.workspace_bytes(sh, T)
    ro = dict(topk_idx=e(T, k, dt=i32), topk_w=e(T, k))
    brx.route(sh, brx.LayerData(router_w=Wr, codes=None, scales=None), u, brx.X_BF16, T, ro, ws_of(nb), nb)
    idx = torch.where(keep[:, None], ro["topk_idx"], -1).to(i32).contiguous()   # padding picks nothing
    z = u.float() @ Wr.t()
    losses, counts, lse, tokens = e(2), e(E, dt=i32), e(T), e(1, dt=i32)
    bb = brx.balance_loss_workspace_bytes(T, k, E)
    brx.balance_loss(z, 1, idx, T, k, E, losses, counts, lse, tokens, ws_of(bb), bb, keep=keep)
    pos = e(n, dt=i32)
    sb = brx.sort_workspace_bytes(T, k, E)
    brx.sort_picks(idx, T, k, E, None, None, None, pos, ws_of(sb), sb)
    dpicks = e(T, k)
    brx.combine_backward(dy * w[0], 1, ys, 0, n, pos, ro["topk_w"], T, k, d, dz=dpicks)
    dz = e(T, E)
    brx.balance_loss_backward(z, 1, idx, T, k, E, lse, counts, tokens, torch.tensor(w[1:], device="cuda"), dz, keep=keep,
                              dpicks=dpicks)
    dWr, du = dz.t().contiguous() @ u.float(), (dz @ Wr).to(BF)
    dx, dgain, dT = e(T, d), e(d), e(V, d)
    wb = brx.block_norm_backward_workspace_bytes(args)
    brx.block_norm_backward(args, None, du, x, None, g_pre=gain, rstd_r=rstd, dx=dx, dg_pre=dgain, ws=ws_of(wb), ws_bytes=wb)
    eb = brx.embed_backward_workspace_bytes(T, V, d)
    brx.embed_backward(dx, 1, ids, T, V, d, Q.SCALE, dT, 1, ws_of(eb), eb)
    want = Q.gradients(*host, idx.cpu(), pos.view(T, k).cpu(), term)
    assert int(tokens) == T - Q.PAD
    for name, got, ref in zip(("table", "Wr", "gain"), (dT, dWr, dgain), want):
        off = float((got.cpu().double() - ref).norm() / ref.norm())
        print(f"  {term} {name}: {off:.2e}", flush=True)
        assert off <= Q.LIMIT, f"{name}: off by {off:.3e}"
