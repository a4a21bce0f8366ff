"""The vocabulary loss's fp32 gradients hold fp32's bits: rows and matrices of
ones and zeros make every output a single value of dz."""
from __future__ import annotations

import pytest
import torch

import bit_routed_expert_amd as brx
from tests.test_gpu_ops import BF, CODE, F32, Out, U, gen, rand, ws_of
from tests.test_gpu_train import run_vocab

pytestmark = pytest.mark.gpu


def single_values(T, V, seed=1):
    """h[t] = e_t and W[v] = (a row of logits, e_v): z[t][v] = W[v][t], dh[t][T + v] = dz[t][v] and dW[v][t] = dz[t][v]."""
    p = (T + 7) // 8 * 8
    d = p + (V + 7) // 8 * 8
    h, W = torch.zeros(T, d, dtype=BF), torch.zeros(V, d, dtype=BF)
    h[torch.arange(T), torch.arange(T)] = 1
    W[:, :T] = rand(V, T, seed=seed, dtype=BF, scale=1.5)
    W[torch.arange(V), p + torch.arange(V)] = 1
    t = torch.randint(0, V, (T,), generator=gen(seed + 1), dtype=torch.int32)
    t[torch.rand(T, generator=gen(seed + 2)) < 0.2] = -1
    t[0] = V - 1
    up, un = rand(T, seed=seed + 3), 0.1 * rand(T, seed=seed + 4)   # weights unlike each other
    return [v.cuda() for v in (h, W, t, up, un)], p, d


@pytest.mark.parametrize("dh_type,dw_type", [(F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("T,V", [(1, 50), (3, 700), (31, 300), (33, 200), (100, 1000), (300, 260), (700, 1500), (9000, 520)])
def test_fp32_gradients_of_single_values(T, V, dh_type, dw_type):
    print(f"case vocab bits T={T} V={V} {dh_type} {dw_type}", flush=True)
    (h, W, t, up, un), p, d = single_values(T, V)
    _, lse = run_vocab(h, W, t, T, V, d)
    dh, dW = Out(T, d, dtype=dh_type), Out(V, d, dtype=dw_type)
    nb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
    brx.vocab_loss_backward(h, W, t, T, V, d, lse, up, ws_of(nb), nb, dlse=un, dh=dh.t, dhdtype=CODE[dh_type], dW=dW.t,
                            dwdtype=CODE[dw_type])
    on = t >= 0
    x = W[:, :T].double().t() - lse.double()[:, None]
    q = torch.exp(x) * (up.double() + un.double())[:, None]
    # exp: 4 U and 2 U of its argument, the argument's subtraction U of it; dloss + dlse, the unit's two products, the
    # exponential's and the target's: 6 U; the store U.  Nothing is left of dz out of its pieces.
    bound = q.abs() * (3 * x.abs() + 11) * U + 1e-37
    dz = q.clone()
    at = torch.arange(T, device="cuda")
    y = t.clamp_min(0).long()
    dz[at, y] -= up.double()
    bound[at, y] += 4 * U * up.double().abs()
    bound = bound + 2 * U * dz.abs()
    dz[~on], bound[~on] = 0, 0
    for got, kind in ((dh.guarded()[:, p:p + V], dh_type), (dW.guarded()[:, :T].t(), dw_type)):
        if kind is F32:
            off = (got.double() - dz).abs() - bound
            assert bool((off <= 0).all()), f"{int((off > 0).sum())} of {off.numel()}, worst {float(off.max()):.2e}"
