"""Operators around the layer on the GPU: sort, dispatch, combine, the
experts' products and the block norms, each with its gradient, against the
64-bit forms of ops_ref at the sizes and masks where they can go wrong, with
guard bands behind every output; captured and replayed in graphs, on other
streams, twice with the same bits, and together as one trainable block."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import bit_routed_expert_amd as brx
from tests import ops_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CODE = {BF: brx.X_BF16, F32: brx.X_F32}
U = R.U
GUARD = 64


class Out:
    """An output tensor filled with a pattern, with guard elements behind it."""

    def __init__(self, *shape, dtype, fill=7.0):
        n = int(np.prod(shape))
        self.fill = fill
        self.all = torch.full((n + GUARD,), fill, dtype=dtype, device="cuda")
        self.t = self.all[:n].view(*shape)

    def guarded(self):
        torch.cuda.synchronize()
        assert bool((self.all[self.t.numel():] == self.fill).all()), "guard elements were written"
        return self.t


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(*shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed)) * scale).to(dtype)


def ws_of(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")


def draw_idx(T, k, E, drop, seed):
    """Ids with repeats inside a token, some dropped as -1, E, or far outside."""
    g = gen(seed)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    out = torch.rand(T, k, generator=g) < drop
    bad = torch.tensor([-1, E, -2**31, 2**31 - 1], dtype=torch.int32)[torch.randint(0, 4, (T, k), generator=g)]
    return torch.where(out, bad, idx)


def run_sort(idx, T, k, E):
    n = T * k
    counts, offsets = Out(E, dtype=torch.int32, fill=-9), Out(E + 1, dtype=torch.int32, fill=-9)
    perm, pos = Out(n, dtype=torch.int32, fill=-9), Out(n, dtype=torch.int32, fill=-9)
    nb = brx.sort_workspace_bytes(T, k, E)
    brx.sort_picks(idx.cuda(), T, k, E, counts.t, offsets.t, perm.t, pos.t, ws_of(nb), nb)
    return [o.guarded().cpu().tolist() for o in (counts, offsets, perm, pos)]


# ------------------------------------------------------------------- sort

@pytest.mark.parametrize("T,k,E,drop", [
    (0, 4, 8, 0.0), (1, 1, 1, 0.0), (1, 1, 1, 1.0), (5, 10, 512, 0.0), (7, 3, 5, 0.4), (64, 1, 1024, 0.0),
    (100, 32, 3, 0.2), (128, 32, 1024, 0.1), (4095, 1, 63, 0.1), (1025, 4, 64, 0.0), (1366, 3, 1, 0.5),
    (4096, 10, 512, 0.0), (3001, 7, 1024, 0.9), (21845, 3, 512, 0.0), (16384, 4, 1024, 0.1), (13107, 5, 2, 0.0),
    (65535, 1, 1, 0.0), (40000, 7, 33, 0.1), (2000, 3, 17, 1.0)])
def test_sort(T, k, E, drop):
    print(f"case sort T={T} k={k} E={E} drop={drop}", flush=True)
    idx = draw_idx(T, k, E, drop, seed=T + k + E)
    got, want = run_sort(idx, T, k, E), R.sort(idx, E)
    for g, w, name in zip(got, want, ("counts", "offsets", "perm", "pos")):
        assert g == w, name


def test_sort_equals_the_route_outputs():
    """Without drops, the permutation strata_moe_route gives for its own picks."""
    T, E, k, d = 77, 64, 6, 256
    sh = brx.shape(E, k, d, 128, 3)
    x = rand(T, d, seed=1, dtype=BF).cuda()
    layer = brx.LayerData(router_w=rand(E, d, seed=2).cuda(), codes=None, scales=None)
    out = {n: torch.empty(s, dtype=torch.int32, device="cuda") for n, s in
           (("topk_idx", (T, k)), ("counts", E), ("offsets", E + 1), ("perm", T * k), ("pos", T * k))}
    nb = brx.workspace_bytes(sh, T)
    brx.route(sh, layer, x, brx.X_BF16, T, out, ws_of(nb), nb)
    got = run_sort(out["topk_idx"].cpu(), T, k, E)
    for g, name in zip(got, ("counts", "offsets", "perm", "pos")):
        assert g == out[name].cpu().tolist(), name


def test_sort_outputs_may_be_left_out():
    idx = draw_idx(900, 6, 40, 0.2, seed=3)
    want = R.sort(idx, 40)
    nb = brx.sort_workspace_bytes(900, 6, 40)
    for only in range(4):
        outs = [None] * 4
        outs[only] = torch.full(((40, 41, 5400, 5400)[only],), -9, dtype=torch.int32, device="cuda")
        brx.sort_picks(idx.cuda(), 900, 6, 40, *outs, ws_of(nb), nb)
        assert outs[only].cpu().tolist() == want[only]


# ---------------------------------------------------- dispatch and combine

ROWS = [(1, 1, 1, 1, 0.0), (3, 2, 2, 3, 0.5), (5, 10, 512, 2048, 0.0), (37, 4, 8, 130, 0.3), (19, 32, 40, 264, 0.1),
        (50, 3, 6, 1000, 0.2), (9, 17, 20, 2052, 0.2), (21, 5, 4, 5001, 0.1), (6, 3, 4, 64, 1.0), (300, 8, 16, 24, 0.1),
        (7, 32, 9, 2056, 0.1), (5, 20, 40, 1028, 0.0)]


def positions(T, k, E, drop, seed):
    idx = draw_idx(T, k, E, drop, seed)
    return torch.tensor(R.sort(idx, E)[3], dtype=torch.int32)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,k,E,d,drop", ROWS)
def test_dispatch(T, k, E, d, drop, dt):
    print(f"case dispatch T={T} k={k} d={d} {dt}", flush=True)
    pos, rows = positions(T, k, E, drop, d + T), T * k
    x = rand(T, d, seed=d, dtype=dt)
    xs = Out(rows, d, dtype=dt)
    brx.dispatch(x.cuda(), CODE[dt], T, k, d, pos.cuda(), xs.t, rows)
    want = torch.full((rows, d), 7.0, dtype=dt)   # rows without a pick stay as they were
    for f, p in enumerate(pos.tolist()):
        if p >= 0:
            want[p] = x[f // k]
    assert torch.equal(xs.guarded().cpu(), want)
    dxs = rand(rows, d, seed=d + 1, dtype=dt)
    dx = Out(T, d, dtype=dt)
    brx.dispatch_backward(dxs.cuda(), CODE[dt], rows, pos.cuda(), T, k, d, dx.t)
    ref = R.combine(dxs.double(), pos, None, None, T, k)
    mag = R.combine(dxs.double().abs(), pos, None, None, T, k)
    R.check(dx.guarded(), ref, k * U * mag, "dx")


@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("T,k,E,d,drop", ROWS)
def test_combine(T, k, E, d, drop, yt, ot):
    """Forward and gradient; rows and weights of dropped picks hold NaN and are not used."""
    print(f"case combine T={T} k={k} d={d} {yt} {ot}", flush=True)
    pos, rows = positions(T, k, E, drop, d + T + 1), T * k
    ys, w = rand(rows, d, seed=1, dtype=yt), rand(T * k, seed=2)
    kept = int((pos >= 0).sum())
    ys[kept:] = float("nan")
    w_bad = torch.where(pos >= 0, w, torch.full_like(w, float("nan")))
    yd = torch.nan_to_num(ys.double())
    for base, weights in ((None, w_bad), (rand(T, d, seed=3, dtype=ot), w_bad), (rand(T, d, seed=4, dtype=ot), None)):
        out = Out(T, d, dtype=ot)
        bd = None if base is None else base.double()
        if base is not None:
            out.t.copy_(base)   # in place: the output is the base
        brx.combine(ys.cuda(), CODE[yt], rows, pos.cuda(), None if weights is None else weights.cuda(), T, k, d, out.t,
                    CODE[ot], base=None if base is None else out.t)
        wd = None if weights is None else w.double()
        ref = R.combine(yd, pos, wd, bd, T, k)
        mag = R.combine(yd.abs(), pos, None if wd is None else wd.abs(), None if bd is None else bd.abs(), T, k)
        R.check(out.guarded(), ref, (k + 1) * U * mag, "out")
    # gradient, the gates a softmax over the picks
    gates = torch.softmax(rand(T, k, seed=5), 1)
    dout = rand(T, d, seed=6, dtype=ot)
    dys, dw, dz = Out(rows, d, dtype=yt), Out(T, k, dtype=F32), Out(T, k, dtype=F32)
    brx.combine_backward(dout.cuda(), CODE[ot], ys.cuda(), CODE[yt], rows, pos.cuda(), gates.cuda(), T, k, d,
                         dys=dys.t, dw=dw.t, dz=dz.t)
    v, has = R.picked(yd, pos, T, k)
    g, o = gates.double(), dout.double()
    rdw = (v * o[:, None]).sum(2)
    bdw = d * U * (v.abs() * o.abs()[:, None]).sum(2)
    R.check(dw.guarded(), rdw, bdw, "dw")
    rdz = g * (rdw - (g * rdw).sum(1, keepdim=True))
    bdz = g * (bdw + (g * bdw).sum(1, keepdim=True)) + (k + 4) * U * g * (rdw.abs() + (g * rdw.abs()).sum(1, keepdim=True))
    R.check(dz.guarded(), rdz, bdz, "dz")
    got = dys.guarded().cpu()
    p, f = pos[pos >= 0].long(), (pos >= 0).nonzero().flatten()
    if kept:
        want = g.reshape(-1)[f][:, None] * o[f // k]
        R.check(got[p], want, U * want.abs(), "dys")
    assert bool((got[kept:] == 7.0).all()), "rows without a pick were written"


def test_combine_backward_outputs_apart_and_in_place():
    T, k, d, E = 30, 4, 200, 6
    pos, rows = positions(T, k, E, 0.2, 9).cuda(), T * k
    ys, dout = rand(rows, d, seed=1).cuda(), rand(T, d, seed=2).cuda()
    w = torch.softmax(rand(T, k, seed=3), 1).cuda()
    full = [torch.zeros(rows, d, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, k, device="cuda")]
    brx.combine_backward(dout, 1, ys, 1, rows, pos, w, T, k, d, *full)
    for i in range(3):
        outs = [None] * 3
        outs[i] = torch.zeros_like(full[i])
        brx.combine_backward(dout, 1, ys, 1, rows, pos, w, T, k, d, *outs)
        assert torch.equal(outs[i], full[i])
    same, dw = ys.clone(), torch.empty(T, k, device="cuda")
    brx.combine_backward(dout, 1, same, 1, rows, pos, w, T, k, d, dys=same, dw=dw)   # dys over ys
    kept = int((pos >= 0).sum())
    assert torch.equal(same[:kept], full[0][:kept]) and torch.equal(same[kept:], ys[kept:])
    assert torch.equal(dw, full[1])


def test_positions_outside_the_rows_copy_nothing():
    T, k, d, rows = 4, 2, 64, 5
    pos = torch.tensor([0, 5, -1, 4, 2**31 - 1, 2, -2**31, 6], dtype=torch.int32).cuda()
    x, xs = rand(T, d, seed=1).cuda(), Out(rows, d, dtype=F32)
    brx.dispatch(x, 1, T, k, d, pos, xs.t, rows)
    got = xs.guarded()
    assert torch.equal(got[0], x[0]) and torch.equal(got[4], x[1]) and torch.equal(got[2], x[2])
    assert bool((got[[1, 3]] == 7.0).all())
    out = Out(T, d, dtype=F32)
    brx.combine(x[:1].repeat(rows, 1), 1, rows, pos, None, T, k, d, out.t, 1)
    assert torch.equal(out.guarded(), torch.stack([x[0], x[0], x[0], torch.zeros_like(x[0])]))
    none = Out(T, d, dtype=F32)   # no rows at all
    brx.combine(None, 1, 0, pos, None, T, k, d, none.t, 1)
    assert bool((none.guarded() == 0).all())


# --------------------------------------------------------- experts' products

GROUPS = [  # rows per expert, N, K, rows behind the last
    ([1], 8, 8, 0), ([0, 3, 0], 64, 128, 5), ([1, 0, 2, 1, 0, 1], 1536, 2048, 0), ([5, 64, 65, 0, 1], 72, 104, 3),
    ([130, 0, 257], 264, 520, 1), ([0, 0], 64, 64, 4), ([33] * 40, 128, 256, 0), ([300], 256, 1024, 0),
    ([16, 17, 31, 32, 48], 2048, 768, 0), ([700, 3], 200, 24, 0), ([90, 70, 0, 110], 512, 1032, 2),
    # few rows against the experts: one to nine rows of the experts that have any
    ([0, 1, 2, 0, 3, 4, 5] + [0] * 62 + [1], 200, 1032, 1), ([0] * 40 + [9], 72, 24, 0), ([0, 2] + [0] * 6, 1536, 2048, 0),
    ([1] + [0] * 19 + [3], 88, 8192, 1), ([1] + [0] * 3, 8, 8, 0), ([0] * 9, 16, 16, 2),
    # the largest tiles and grids whose tiles an earlier launch lists; more than 64 experts
    ([5000, 131, 7769], 1000, 904, 2), ([39000, 900], 1000, 136, 0), ([20, 0, 41, 19] * 32 + [300], 520, 1032, 1),
    ([3, 1, 5] * 67, 520, 264, 0), ([(7 * i) % 90 for i in range(40)], 1288, 1288, 3), ([0] * 30 + [700] * 2, 136, 1000, 0),
    ([40, 39, 0, 161] * 10, 520, 600, 2)]


def group_inputs(ns, N, K, tail, seed=1):
    rows = sum(ns) + tail
    off = torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32)
    x, dy = rand(rows, K, seed=seed, dtype=BF), rand(rows, N, seed=seed + 1, dtype=BF)
    W = rand(len(ns), N, K, seed=seed + 2, dtype=BF, scale=K ** -0.5)
    if tail:   # rows behind the last expert's are not read
        x[-tail:] = float("nan")
        dy[-tail:] = float("nan")
    return rows, off, x, dy, W


@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("ns,N,K,tail", GROUPS)
def test_grouped_products(ns, N, K, tail, ot):
    print(f"case grouped {ns[:6]} N={N} K={K} {ot}", flush=True)
    rows, off, x, dy, W = group_inputs(ns, N, K, tail)
    E, real = len(ns), sum(ns)
    nb = brx.grouped_workspace_bytes(rows, E, N, K)
    ws = ws_of(nb)
    xd, yd, Wd = x.double(), dy.double(), W.double()
    y, dx, dW = Out(rows, N, dtype=ot), Out(rows, K, dtype=ot), Out(E, N, K, dtype=ot)
    xc, yc, Wc, oc = x.cuda(), dy.cuda(), W.cuda(), off.cuda()
    brx.grouped_product(xc, Wc, oc, rows, E, N, K, y.t, CODE[ot], ws, nb)
    print("  product", flush=True)
    got = y.guarded()
    assert bool((got[real:] == 7.0).all()), "rows behind the last expert's were written"
    R.check(got[:real], R.grouped_product(xd[:real], Wd, off), 2 * K * U * R.grouped_product(xd[:real].abs(), Wd.abs(), off), "y")
    brx.grouped_dgrad(yc, Wc, oc, rows, E, N, K, dx.t, CODE[ot], ws, nb)
    print("  dgrad", flush=True)
    got = dx.guarded()
    assert bool((got[real:] == 7.0).all()), "rows behind the last expert's were written"
    Wt = Wd.transpose(1, 2).contiguous()
    R.check(got[:real], R.grouped_product(yd[:real], Wt, off), 2 * N * U * R.grouped_product(yd[:real].abs(), Wt.abs(), off), "dx")
    brx.grouped_wgrad(yc, xc, oc, rows, E, N, K, dW.t, CODE[ot], ws, nb)
    print("  wgrad", flush=True)
    ref, mag = torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64)
    for e, a, b in R.segments(off):
        ref[e] = yd[a:b].t() @ xd[a:b]
        mag[e] = 2 * (b - a) * U * (yd[a:b].abs().t() @ xd[a:b].abs())
    R.check(dW.guarded(), ref, mag, "dW")


LENGTHS = [   # rows per expert, N, K, what is run: contractions of 1 to 13 whole and ragged steps in every tile
    *[([7, 0, 50], 136, 64 * n + r, "product") for n in range(1, 10) for r in (0, -8)],                 # 32-row tiles
    *[([7, 0, 50], 64 * n + r, 136, "dgrad") for n in range(1, 10) for r in (0, -8)],
    *[([300, 200, 7, 0, 260], 1224, 64 * n + r, "product") for n in range(1, 10) for r in (0, -8)],     # 64-row tiles
    *[([300, 200, 7, 0, 260], 64 * n + r, 1224, "dgrad") for n in range(1, 10) for r in (0, -8)],
    *[([120] * 40, 520, 64 * n + r, "product") for n in range(1, 8) for r in (0, 8)],                   # 128-row tiles
    *[([120] * 40, 64 * n + r, 520, "dgrad") for n in range(1, 8) for r in (0, 8)],
    *[([25000, 24200], 256, 64 * n + r, "product") for n in range(1, 6) for r in (0, -56)],             # 256-row tiles
    *[([25000, 24200], 64 * n + r, 256, "dgrad") for n in range(1, 6) for r in (0, -56)],
    *[([25000, 24200, 130], 136, n, "dgrad") for n in (264, 328, 456)],                                 # waves without columns
    *[([25000, 24200, 130], n, 136, "product") for n in (264, 328, 456)],
    *[([300, 120, 7] * 14, n, 200, "product") for n in (264, 328, 392, 456)],
    ([16 * i + i % 3 for i in range(25)], 128, 128, "wgrad"),                                           # 64 square
    ([16 * i + i % 3 for i in range(25)], 512, 512, "wgrad"),                                           # 128 square
    ([16 * i + i % 3 for i in range(25)] + [31, 32, 33] * 5, 1288, 1288, "wgrad"),                      # 256 square
    ([16 * (i % 25) + i % 3 for i in range(70)], 1032, 776, "wgrad"),                                   # the same, not ranked
]


@pytest.mark.parametrize("ns,N,K,what", LENGTHS)
def test_grouped_contractions_of_every_length(ns, N, K, what):
    """The buffered contraction's start, turns and end: as test_grouped_products, fp32 outputs."""
    print(f"case length {len(ns)} N={N} K={K} {what}", flush=True)
    rows, off, x, dy, W = group_inputs(ns, N, K, 0, seed=4)
    E = len(ns)
    nb = brx.grouped_workspace_bytes(rows, E, N, K)
    ws, oc = ws_of(nb), off.cuda()
    xc, yc, Wc = x.cuda(), dy.cuda(), W.cuda()
    first = None
    for _ in range(2):
        if what == "product":
            out = Out(rows, N, dtype=F32)
            brx.grouped_product(xc, Wc, oc, rows, E, N, K, out.t, 1, ws, nb)
        elif what == "dgrad":
            out = Out(rows, K, dtype=F32)
            brx.grouped_dgrad(yc, Wc, oc, rows, E, N, K, out.t, 1, ws, nb)
        else:
            out = Out(E, N, K, dtype=F32)
            brx.grouped_wgrad(yc, xc, oc, rows, E, N, K, out.t, 1, ws, nb)
        got = out.guarded()
        first = got if first is None else first
        assert torch.equal(got, first)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if what == "wgrad":
            a, b, n, g = yc[lo:hi].double().t().contiguous(), xc[lo:hi].double(), hi - lo, got[e]
        elif what == "product":
            a, b, n, g = xc[lo:hi].double(), Wc[e].double().t().contiguous(), K, got[lo:hi]
        else:
            a, b, n, g = yc[lo:hi].double(), Wc[e].double(), N, got[lo:hi]
        R.check(g, (a @ b).cpu(), (2 * n * U * (a.abs() @ b.abs())).cpu(), f"{what} of expert {e}")


def test_grouped_without_rows():
    E, N, K = 3, 64, 72
    nb = brx.grouped_workspace_bytes(0, E, N, K)
    dW = Out(E, N, K, dtype=BF)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    brx.grouped_wgrad(None, None, off, 0, E, N, K, dW.t, brx.X_BF16, ws_of(nb), nb)
    assert bool((dW.guarded() == 0).all())


@pytest.mark.parametrize("off", [[5, 2, 9, 9], [-7, 4, 99, 3], [0, 0, 0, 0], [30, 30, 30, 30], [12, 0, 12, 0]])
@pytest.mark.parametrize("pad", [0, 100])
def test_grouped_offsets_that_do_not_ascend_stay_inside(off, pad):
    """Which rows such offsets mean is not specified; nothing outside the
    buffers is written.  With 100 experts more the product takes its path for
    few rows."""
    N, K, rows = 72, 64, 20
    _, _, x, dy, W = group_inputs([20], N, K, 0)
    off = off[:2] + [off[1]] * (pad // 2) + off[2:] + [off[3]] * (pad // 2)
    E = len(off) - 1
    W = W.repeat(E, 1, 1)
    nb = brx.grouped_workspace_bytes(rows, E, N, K)
    wsb = torch.full((nb + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    y, dx, dW = Out(rows, N, dtype=F32), Out(rows, K, dtype=F32), Out(E, N, K, dtype=F32)
    brx.grouped_product(x.cuda(), W.cuda(), o, rows, E, N, K, y.t, 1, wsb, nb)
    brx.grouped_dgrad(dy.cuda(), W.cuda(), o, rows, E, N, K, dx.t, 1, wsb, nb)
    brx.grouped_wgrad(dy.cuda(), x.cuda(), o, rows, E, N, K, dW.t, 1, wsb, nb)
    for q in (y, dx, dW):
        q.guarded()
    assert bool((wsb[nb:] == 0x5A).all())


def test_grouped_experts_do_not_touch_each_other():
    """NaN in one expert's rows or weights stays with it, in every tile size."""
    for ns in ([5, 7, 40, 9], [130, 70, 300, 90], [600, 500, 700, 800], [1, 2, 0, 1] + [0] * 30):
        N, K, E, bad = 264, 136, len(ns), 1
        rows, off, x, dy, W = group_inputs(ns, N, K, 0)
        a, b = int(off[bad]), int(off[bad + 1])
        x[a:b], dy[a:b], W[bad] = float("nan"), float("inf"), float("nan")
        nb = brx.grouped_workspace_bytes(rows, E, N, K)
        ws = ws_of(nb)
        y, dx, dW = Out(rows, N, dtype=F32), Out(rows, K, dtype=F32), Out(E, N, K, dtype=F32)
        xc, yc, Wc, oc = x.cuda(), dy.cuda(), W.cuda(), off.cuda()
        brx.grouped_product(xc, Wc, oc, rows, E, N, K, y.t, 1, ws, nb)
        brx.grouped_dgrad(yc, Wc, oc, rows, E, N, K, dx.t, 1, ws, nb)
        brx.grouped_wgrad(yc, xc, oc, rows, E, N, K, dW.t, 1, ws, nb)
        others = torch.ones(rows, dtype=torch.bool)
        others[a:b] = False
        for q in (y, dx):
            got = q.guarded().cpu()
            assert bool(torch.isfinite(got[others]).all()) and not bool(torch.isfinite(got[a:b]).any())
        got = dW.guarded().cpu()
        assert bool(torch.isfinite(got[[e for e in range(E) if e != bad]]).all())


# ------------------------------------------------------ past 32-bit offsets

def test_rows_past_32_bit_offsets():
    """Slots, experts' rows, weights and norm rows whose element offsets pass 2^31."""
    d, rows = 2048, 1_100_000
    assert rows * d > 2**31
    print("case dispatch and combine past 2^31 elements", flush=True)
    T, k = 3, 2
    pos = torch.tensor([rows - 1, 0, rows - 2, 7, 2**20 + 5, rows - 3], dtype=torch.int32, device="cuda")
    x = rand(T, d, seed=1, dtype=BF).cuda()
    xs = torch.zeros(rows, d, dtype=BF, device="cuda")
    brx.dispatch(x, 0, T, k, d, pos, xs, rows)
    assert torch.equal(xs[pos.long()], x.repeat_interleave(k, 0)) and int((xs != 0).any(1).sum()) == T * k
    out = torch.empty(T, d, dtype=F32, device="cuda")
    brx.combine(xs, 0, rows, pos, None, T, k, d, out, 1)
    assert torch.equal(out, 2 * x.float())
    print("case products past 2^31 elements", flush=True)
    N = 64
    W = rand(2, N, d, seed=2, dtype=BF, scale=d ** -0.5).cuda()
    off = torch.tensor([0, rows - 3, rows], dtype=torch.int32, device="cuda")
    xs[-3:] = rand(3, d, seed=3, dtype=BF).cuda()
    nb = brx.grouped_workspace_bytes(rows, 2, N, d)
    ws, y = ws_of(nb), torch.empty(rows, N, dtype=F32, device="cuda")
    brx.grouped_product(xs, W, off, rows, 2, N, d, y, 1, ws, nb)
    tail, Wd = xs[-3:].double().cpu(), W.double().cpu()
    R.check(y[-3:], tail @ Wd[1].t(), 2 * d * U * (tail.abs() @ Wd[1].abs().t()), "y")
    dy = torch.zeros(rows, N, dtype=BF, device="cuda")
    dy[-3:] = rand(3, N, seed=4, dtype=BF).cuda()
    dx = torch.empty(rows, d, dtype=BF, device="cuda")
    brx.grouped_dgrad(dy, W, off, rows, 2, N, d, dx, 0, ws, nb)
    gt = dy[-3:].double().cpu()
    R.check(dx[-3:], gt @ Wd[1], 2 * N * U * (gt.abs() @ Wd[1].abs()), "dx")
    dW = torch.empty(2, N, d, dtype=F32, device="cuda")
    brx.grouped_wgrad(dy, xs, off, rows, 2, N, d, dW, 1, ws, nb)
    R.check(dW[1], gt.t() @ tail, 6 * U * (gt.abs().t() @ tail.abs()), "dW")
    assert bool((dW[0] == 0).all())   # its dy are zeros
    del dx, dy, y
    print("case block norm past 2^31 elements", flush=True)
    u = torch.empty(rows, d, dtype=BF, device="cuda")
    xs[1] = 1.5
    brx.block_norm(brx.block_norm_args(rows, d, 0, 0, 0, brx.PRE_NORM), xs, None, u=u)
    want = R.norm_rows(xs[-3:].double().cpu(), None, f32(1e-6))
    R.check(u[-3:], want, (d + 8) * U * want.abs(), "u")
    del xs, u
    print("case weights past 2^31 elements", flush=True)
    E, N, K = 700, 1536, 2048
    W = torch.zeros(E, N, K, dtype=BF, device="cuda")
    W[-1] = rand(N, K, seed=5, dtype=BF, scale=K ** -0.5).cuda()
    for n in (2, 800):   # the path for few rows, and the tiles
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[-1] = n
        x = rand(n, K, seed=6, dtype=BF).cuda()
        y = torch.empty(n, N, dtype=F32, device="cuda")
        nb = brx.grouped_workspace_bytes(n, E, N, K)
        brx.grouped_product(x, W, off, n, E, N, K, y, 1, ws_of(nb), nb)
        xd, Wd = x.double().cpu(), W[-1].double().cpu()
        R.check(y, xd @ Wd.t(), 2 * K * U * (xd.abs() @ Wd.abs().t()), "y")
    dW = torch.empty(E, N, K, dtype=BF, device="cuda")
    dy = rand(n, N, seed=7, dtype=BF).cuda()
    brx.grouped_wgrad(dy, x, off, n, E, N, K, dW, 0, ws_of(nb), nb)
    gd = dy.double().cpu()
    R.check(dW[-1], gd.t() @ xd, 2 * n * U * (gd.abs().t() @ xd.abs()), "dW")
    assert not bool(dW[:-1].any())


# ------------------------------------------------------------- block norms

NORMS = [  # T, d, x, y, u types, post, pre, gate, sigmoid
    (1, 2048, F32, F32, BF, True, True, "token", True), (1, 1, F32, F32, F32, True, True, None, False),
    (5, 3, BF, BF, BF, True, True, "channel", True), (7, 510, BF, F32, F32, True, True, "channel", False),
    (9, 512, F32, BF, BF, False, True, "token", False), (6, 520, BF, BF, F32, True, False, "channel", True),
    (4, 1001, F32, BF, BF, True, True, "token", True), (3, 1024, BF, BF, BF, False, False, None, False),
    (5, 1032, F32, F32, F32, True, True, "channel", True), (33, 2048, BF, BF, BF, True, True, "channel", False),
    (3, 2050, BF, F32, BF, True, True, None, False), (3, 4096, F32, BF, F32, True, True, "token", True),
    (2, 4097, BF, BF, BF, True, True, "channel", True), (2, 8192, F32, F32, BF, True, True, "channel", True),
    (2, 8191, F32, F32, F32, True, True, "token", False), (6, 256, F32, None, BF, False, True, None, False),
    (1100, 136, BF, BF, BF, True, True, "channel", True), (4500, 64, F32, F32, F32, True, True, "token", True),
    (1500, 1160, BF, BF, F32, True, True, "token", False),
    # around the rows that one block takes alone, gains' gradients and all
    (8, 512, F32, BF, BF, True, True, "channel", False), (9, 520, BF, BF, F32, True, True, "token", True),
    (8, 1024, BF, F32, BF, True, True, None, False), (2, 2048, F32, BF, BF, True, True, "token", False),
    (1, 8192, BF, BF, BF, True, True, None, False), (3, 4096, BF, BF, BF, True, False, "channel", True)]


def norm_case(T, d, xt, yt, ut, post, pre, gate, sig, seed=1):
    flags = (brx.POST_NORM if post else 0) | (brx.PRE_NORM if pre else 0) | (brx.GATE_SIGMOID if sig else 0) | \
        {None: 0, "token": brx.GATE_TOKEN, "channel": brx.GATE_CHANNEL}[gate]
    a = brx.block_norm_args(T=T, d=d, x_dtype=CODE[xt], y_dtype=CODE[yt or F32], u_dtype=CODE[ut], flags=flags,
                            resid_scale=0.75, branch_scale=-1.25, eps=1e-5)
    t = dict(x=rand(T, d, seed=seed, dtype=xt, scale=2.0), y=None if yt is None else rand(T, d, seed=seed + 1, dtype=yt),
             g_post=1 + 0.3 * rand(d, seed=seed + 2) if post else None,
             g_pre=1 + 0.3 * rand(d, seed=seed + 3) if pre else None,
             gate={None: None, "token": rand(T, seed=seed + 4),
                   "channel": rand(T, d, seed=seed + 4, dtype=yt or F32)}[gate])
    if T > 2 and yt is not None:
        t["y"][1] = 0   # a row whose norm is eps alone
    return a, t


def f32(v):
    return float(torch.tensor(v, dtype=F32))   # the scale as the library gets it


def dbl(t):
    return {n: None if v is None else v.double() for n, v in t.items()}


def cu(v):
    return None if v is None else v.cuda()


@pytest.mark.parametrize("case", NORMS)
def test_block_norm(case):
    """Bounds: rstd's sum of d squares and four more steps halve in the root;
    the gate's exponential adds (|v| + 6) steps."""
    print(f"case block_norm {case}", flush=True)
    T, d, xt, yt, ut, post, pre, gate, sig = case
    a, t = norm_case(*case)
    D = dbl(t)
    kw = dict(post=post, pre=pre, sigmoid=sig, a=f32(0.75), b=f32(-1.25), eps=f32(1e-5))
    r, u, ry, rr = R.block_norm(D["x"], D["y"], D["gate"], D["g_post"], D["g_pre"], **kw)
    out = dict(r=Out(T, d, dtype=xt), u=Out(T, d, dtype=ut) if pre else None,
               rstd_y=Out(T, dtype=F32) if post else None, rstd_r=Out(T, dtype=F32) if pre else None)
    brx.block_norm(a, cu(t["x"]), cu(t["y"]), gate=cu(t["gate"]), g_post=cu(t["g_post"]), g_pre=cu(t["g_pre"]),
                   **{n: None if o is None else o.t for n, o in out.items()})
    e1 = (d / 2 + 4) * U
    er = 2 * U * (0.75 * D["x"]).abs()
    if t["y"] is not None:
        n = D["y"] if not post else D["y"] * ry[:, None] * D["g_post"]
        eg = 0.0 if gate is None else (D["gate"].abs().max() + 6) * U
        er = er + (1.25 * R.gate_factor(D["gate"], sig) * n).abs() * (e1 + eg + 6 * U)
    R.check(out["r"].guarded(), r, er, "r")
    if post:
        R.check(out["rstd_y"].guarded(), ry, e1 * ry, "rstd_y")
    if pre:
        err = rr * ((r.abs() * er).sum(1) * rr * rr / d + e1)
        R.check(out["rstd_r"].guarded(), rr, err, "rstd_r")
        R.check(out["u"].guarded(), u, rr[:, None] * D["g_pre"].abs() * er + u.abs() * ((err / rr)[:, None] + 3 * U), "u")


@pytest.mark.parametrize("case", NORMS)
def test_block_norm_backward(case):
    """Bounds: every value is a chain of at most 2d + T + 64 roundings on terms
    whose magnitudes the formula sums when every sign is taken positive (for a
    gate's own derivative g (1 - g), g: 1 - g is exact to a step of g)."""
    print(f"case block_norm_backward {case}", flush=True)
    T, d, xt, yt, ut, post, pre, gate, sig = case
    a, t = norm_case(*case)
    D = dbl(t)
    A, B, eps = f32(0.75), f32(-1.25), f32(1e-5)
    kw = dict(post=post, pre=pre, sigmoid=sig, a=A, b=B, eps=eps)
    r = R.block_norm(D["x"], D["y"], D["gate"], D["g_post"], D["g_pre"], **kw)[0].to(xt)   # the stored rows
    rd = r.double()
    rr = 1.0 / torch.sqrt((rd * rd).mean(1) + eps)
    ry = None if not post else 1.0 / torch.sqrt((D["y"] * D["y"]).mean(1) + eps)
    dr, du = rand(T, d, seed=21, dtype=xt), rand(T, d, seed=22, dtype=ut) if pre else None
    has_y = t["y"] is not None
    out = dict(dx=Out(T, d, dtype=xt), dy=Out(T, d, dtype=yt) if has_y else None,
               dgate={None: None, "token": Out(T, dtype=F32), "channel": Out(T, d, dtype=yt or F32)}[gate],
               dg_post=Out(d, dtype=F32) if post else None, dg_pre=Out(d, dtype=F32) if pre else None)
    nb = brx.block_norm_backward_workspace_bytes(a)
    ins = dict(gate=cu(t["gate"]), g_post=cu(t["g_post"]), g_pre=cu(t["g_pre"]), rstd_y=None if ry is None else ry.float().cuda(),
               rstd_r=rr.float().cuda() if pre else None)
    brx.block_norm_backward(a, dr.cuda(), cu(du), r.cuda(), cu(t["y"]), **ins,
                            **{n: None if o is None else o.t for n, o in out.items()}, ws=ws_of(nb), ws_bytes=nb)
    # references by automatic differentiation in 64 bits
    leaves = {n: D[n].clone().requires_grad_(True) for n in ("y", "gate", "g_post") if D[n] is not None}
    g = dr.double()
    c = (2 * d + T + 64) * U
    mD = g.abs()
    if pre:
        rl, gl = rd.clone().requires_grad_(True), D["g_pre"].clone().requires_grad_(True)
        ga, gb = torch.autograd.grad(R.norm_rows(rl, gl, eps), [rl, gl], du.double())
        rn = (rd * rr[:, None]).abs()
        q = (du.double() * D["g_pre"]).abs()
        mD = mD + rr[:, None] * (q + rn * (q * rn).mean(1, keepdim=True))
        g = g + ga
        R.check(out["dg_pre"].guarded(), gb, c * (du.double().abs() * rn).sum(0), "dg_pre")
    R.check(out["dx"].guarded(), A * g, c * abs(A) * mD, "dx")
    if not has_y:
        return
    n = leaves["y"]
    if post:
        n = R.norm_rows(n, leaves["g_post"], eps)
    branch = B * R.gate_factor(leaves.get("gate"), sig) * n
    grads = dict(zip(leaves, torch.autograd.grad(branch, list(leaves.values()), g)))
    G = R.gate_factor(D["gate"], sig)
    G = abs(G) if gate is None else G.abs()
    yn = D["y"].abs() * (ry[:, None] if post else 1.0)
    gp = D["g_post"].abs() if post else 1.0
    mt = abs(B) * G * mD
    mg = mt * gp
    my = ry[:, None] * (mg + yn * (mg * yn).mean(1, keepdim=True)) if post else mg
    R.check(out["dy"].guarded(), grads["y"], c * my, "dy")
    if post:
        R.check(out["dg_post"].guarded(), grads["g_post"], c * (mt * yn).sum(0), "dg_post")
    if gate:
        m = abs(B) * mD * yn * gp * (G if sig else 1.0)
        R.check(out["dgate"].guarded(), grads["gate"], c * (m if gate == "channel" else m.sum(1)), "dgate")


@pytest.mark.parametrize("gate,yt", [("token", F32), ("token", BF), ("channel", F32), ("channel", BF)])
@pytest.mark.parametrize("d", [65, 130, 264, 1032, 2056, 4104])
def test_block_norm_gradient_of_sigmoid_gates_far_from_zero(d, gate, yt):
    """The gate's own gradient b D n s (1 - s), s = sigmoid(v), to its own
    magnitude: 1 - s is not taken from an s that has rounded to 1.  Bounds: the
    exponential is off by 2|v| + 2 steps (its argument by two roundings of v
    log2 e, the instruction by two), so s (1 - s) by no more than 4|v| + 10; b D n
    adds 3, a token's sum d."""
    print(f"case sigmoid gates d={d} {gate} {yt}", flush=True)
    vals = torch.tensor([0.0, 1.0, 4.0, 8.0, 10.0, 12.0, 15.0, 16.5, 17.0, 17.5, 20.0, 30.0, 60.0, 80.0, 100.0, 1000.0])
    vals = torch.cat([vals, -vals])
    T = 37
    v = vals[torch.arange(T) % 32] if gate == "token" else vals[(torch.arange(T)[:, None] * 5 + torch.arange(d)) % 32].to(yt)
    y, dr = rand(T, d, seed=1, dtype=yt), rand(T, d, seed=2)
    a = brx.block_norm_args(T, d, CODE[F32], CODE[yt], CODE[F32],
                            brx.GATE_SIGMOID | (brx.GATE_TOKEN if gate == "token" else brx.GATE_CHANNEL), 1.0, -1.25)
    dg = Out(T, dtype=F32) if gate == "token" else Out(T, d, dtype=yt)
    brx.block_norm_backward(a, dr.cuda(), None, None, y.cuda(), gate=v.cuda(), dgate=dg.t)
    terms, vd = -1.25 * dr.double() * y.double(), v.double()
    mag = terms.abs()
    if gate == "token":
        terms, mag = terms.sum(1), mag.sum(1)
    der = torch.sigmoid(vd) * torch.sigmoid(-vd)
    steps = 4 * vd.abs() + 16 + (d if gate == "token" else 0)
    R.check(dg.guarded(), terms * der, steps * U * mag * der, "dgate")


@pytest.mark.parametrize("gate", ["token", "channel"])
def test_block_norm_sigmoid_gates_at_infinity(gate):
    """Gates of either infinity are 1 and 0 and have no gradient; one of NaN stays in its row."""
    T, d = 4, 264
    v = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0])
    v = v if gate == "token" else v[:, None].expand(T, d).contiguous()
    x, y, dr = rand(T, d, seed=1), rand(T, d, seed=2), rand(T, d, seed=3)
    a = brx.block_norm_args(T, d, 1, 1, 1, brx.GATE_SIGMOID | (brx.GATE_TOKEN if gate == "token" else brx.GATE_CHANNEL))
    r, dy, dg = Out(T, d, dtype=F32), Out(T, d, dtype=F32), Out(*v.shape, dtype=F32)
    brx.block_norm(a, x.cuda(), y.cuda(), gate=v.cuda(), r=r.t)
    brx.block_norm_backward(a, dr.cuda(), None, None, y.cuda(), gate=v.cuda(), dy=dy.t, dgate=dg.t)
    got = r.guarded().cpu()
    assert torch.equal(got[0], x[0] + y[0]) and torch.equal(got[1], x[1]) and bool(got[2].isnan().all())
    assert torch.equal(got[3], torch.add(x[3], y[3], alpha=0.5))
    got = dy.guarded().cpu()
    assert torch.equal(got[0], dr[0]) and bool((got[1] == 0).all()) and torch.equal(got[3], 0.5 * dr[3])
    got = dg.guarded().cpu()
    assert bool((got[:2] == 0).all()) and bool(got[2].isnan().all()) and bool(got[3].isfinite().all())


def test_block_norm_in_place_and_outputs_apart():
    T, d = 40, 768
    a, t = norm_case(T, d, F32, BF, BF, True, True, "channel", True)
    g = {n: cu(v) for n, v in t.items()}
    r, u = torch.empty(T, d, device="cuda"), torch.empty(T, d, dtype=BF, device="cuda")
    sy, sr = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ins = dict(gate=g["gate"], g_post=g["g_post"], g_pre=g["g_pre"])
    brx.block_norm(a, g["x"], g["y"], **ins, r=r, u=u, rstd_y=sy, rstd_r=sr)
    x2, u2 = g["x"].clone(), torch.empty_like(u)
    brx.block_norm(a, x2, g["y"], **ins, r=x2, u=u2)          # r over x
    assert torch.equal(x2, r) and torch.equal(u2, u)
    brx.block_norm(a, g["x"], g["y"], **ins, u=u2.zero_())    # u alone
    assert torch.equal(u2, u)
    dr, du = rand(T, d, seed=31).cuda(), rand(T, d, seed=32, dtype=BF).cuda()
    nb = brx.block_norm_backward_workspace_bytes(a)
    full = dict(dx=torch.empty(T, d, device="cuda"), dy=torch.empty(T, d, dtype=BF, device="cuda"),
                dgate=torch.empty(T, d, dtype=BF, device="cuda"), dg_post=torch.empty(d, device="cuda"),
                dg_pre=torch.empty(d, device="cuda"))
    brx.block_norm_backward(a, dr, du, r, g["y"], **ins, rstd_y=sy, rstd_r=sr, **full, ws=ws_of(nb), ws_bytes=nb)
    for n, v in full.items():
        one = torch.zeros_like(v)
        brx.block_norm_backward(a, dr, du, r, g["y"], **ins, rstd_y=sy, rstd_r=sr, **{n: one}, ws=ws_of(nb), ws_bytes=nb)
        assert torch.equal(one, v), n
    same = dr.clone()
    brx.block_norm_backward(a, same, du, r, g["y"], **ins, rstd_y=sy, rstd_r=sr, dx=same)   # dx over dr
    assert torch.equal(same, full["dx"])
    zero, none = torch.empty_like(full["dx"]), torch.empty_like(full["dx"])
    brx.block_norm_backward(a, torch.zeros_like(dr), du, r, g["y"], **ins, rstd_y=sy, rstd_r=sr, dx=zero)
    brx.block_norm_backward(a, None, du, r, g["y"], **ins, rstd_y=sy, rstd_r=sr, dx=none)   # no gradient of r itself
    assert torch.equal(zero, none)


def test_block_norm_gains_of_one():
    """A null gain is a gain of 1, forward and backward."""
    for d in (264, 2048, 3001):
        T = 9
        a, t = norm_case(T, d, F32, F32, F32, True, True, "token", False)
        g = {n: cu(v) for n, v in t.items()}
        one = torch.ones(d, device="cuda")
        outs = []
        for gp, gq in ((None, None), (one, one)):
            r, u, sy, sr = (torch.empty(T, d, device="cuda"), torch.empty(T, d, device="cuda"),
                            torch.empty(T, device="cuda"), torch.empty(T, device="cuda"))
            brx.block_norm(a, g["x"], g["y"], gate=g["gate"], g_post=gp, g_pre=gq, r=r, u=u, rstd_y=sy, rstd_r=sr)
            o = [torch.empty(T, d, device="cuda"), torch.empty(T, d, device="cuda"), torch.empty(T, device="cuda"),
                 torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
            nb = brx.block_norm_backward_workspace_bytes(a)
            brx.block_norm_backward(a, g["x"], g["y"], r, g["y"], gate=g["gate"], g_post=gp, g_pre=gq, rstd_y=sy,
                                    rstd_r=sr, dx=o[0], dy=o[1], dgate=o[2], dg_post=o[3], dg_pre=o[4], ws=ws_of(nb),
                                    ws_bytes=nb)
            outs.append([r, u, sy, sr] + o)
        assert same(*outs)


def test_block_norm_without_rows():
    a = brx.block_norm_args(T=0, d=96, x_dtype=1, y_dtype=1, u_dtype=1, flags=brx.POST_NORM | brx.PRE_NORM)
    gp, gq = Out(96, dtype=F32), Out(96, dtype=F32)
    brx.block_norm_backward(a, None, None, None, None, dg_post=gp.t, dg_pre=gq.t)
    assert bool((gp.guarded() == 0).all()) and bool((gq.guarded() == 0).all())


# --------------------------------------------- graphs, streams, repetition

def every_call(seed):
    """One call of each entry point on small inputs: (run, inputs to overwrite, outputs)."""
    T, k, E, d, N = 70, 4, 6, 264, 136
    idx = draw_idx(T, k, E, 0.1, seed)
    calls = []
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    ic, counts, offsets, perm, pos = idx.cuda(), i32(E), i32(E + 1), i32(T * k), i32(T * k)
    nb = brx.sort_workspace_bytes(T, k, E)
    wss = ws_of(nb)
    calls.append(("sort", lambda: brx.sort_picks(ic, T, k, E, counts, offsets, perm, pos, wss, nb), [ic],
                  [counts, offsets, perm, pos]))
    big = draw_idx(1500, k, E, 0.1, seed + 1).cuda()
    bpos, bnb = i32(1500 * k), brx.sort_workspace_bytes(1500, k, E)
    wsb = ws_of(bnb)
    calls.append(("sort_large", lambda: brx.sort_picks(big, 1500, k, E, None, None, None, bpos, wsb, bnb), [big], [bpos]))
    p = torch.tensor(R.sort(idx, E)[3], dtype=torch.int32).cuda()
    off = torch.tensor(R.sort(idx, E)[1], dtype=torch.int32).cuda()
    rows = T * k
    x, xs, dx = rand(T, d, seed=seed, dtype=BF).cuda(), torch.zeros(rows, d, dtype=BF, device="cuda"), \
        torch.zeros(T, d, dtype=BF, device="cuda")
    calls.append(("dispatch", lambda: brx.dispatch(x, 0, T, k, d, p, xs, rows), [x], [xs]))
    ys = rand(rows, d, seed=seed + 2, dtype=BF).cuda()
    calls.append(("dispatch_backward", lambda: brx.dispatch_backward(ys, 0, rows, p, T, k, d, dx), [ys], [dx]))
    w, out = torch.softmax(rand(T, k, seed=seed + 3), 1).cuda(), torch.zeros(T, d, device="cuda")
    calls.append(("combine", lambda: brx.combine(ys, 0, rows, p, w, T, k, d, out, 1), [ys, w], [out]))
    dout = rand(T, d, seed=seed + 4).cuda()
    dys, dw, dz = torch.zeros(rows, d, dtype=BF, device="cuda"), torch.zeros(T, k, device="cuda"), \
        torch.zeros(T, k, device="cuda")
    calls.append(("combine_backward", lambda: brx.combine_backward(dout, 1, ys, 0, rows, p, w, T, k, d, dys, dw, dz),
                  [ys, dout], [dys, dw, dz]))
    W, gy = rand(E, N, d, seed=seed + 5, dtype=BF).cuda(), rand(rows, N, seed=seed + 6, dtype=BF).cuda()
    gb = brx.grouped_workspace_bytes(rows, E, N, d)
    g1, g2, g3 = ws_of(gb), ws_of(gb), ws_of(gb)
    yo, xo = torch.zeros(rows, N, device="cuda"), torch.zeros(rows, d, device="cuda")
    Wo = torch.zeros(E, N, d, device="cuda")
    calls.append(("product", lambda: brx.grouped_product(ys, W, off, rows, E, N, d, yo, 1, g1, gb), [ys, W], [yo]))
    calls.append(("dgrad", lambda: brx.grouped_dgrad(gy, W, off, rows, E, N, d, xo, 1, g2, gb), [gy, W], [xo]))
    calls.append(("wgrad", lambda: brx.grouped_wgrad(gy, ys, off, rows, E, N, d, Wo, 1, g3, gb), [gy, ys], [Wo]))
    a, t = norm_case(T, d, F32, BF, BF, True, True, "channel", True, seed)
    t = {n: cu(v) for n, v in t.items()}
    r, u = torch.zeros(T, d, device="cuda"), torch.zeros(T, d, dtype=BF, device="cuda")
    sy, sr = torch.ones(T, device="cuda"), torch.ones(T, device="cuda")
    ins = dict(gate=t["gate"], g_post=t["g_post"], g_pre=t["g_pre"])
    calls.append(("block_norm", lambda: brx.block_norm(a, t["x"], t["y"], **ins, r=r, u=u, rstd_y=sy, rstd_r=sr),
                  [t["x"], t["y"], t["gate"]], [r, u, sy, sr]))
    xr, du = rand(T, d, seed=seed + 7).cuda(), rand(T, d, seed=seed + 8, dtype=BF).cuda()
    cy, cr = torch.full((T,), 0.9, device="cuda"), torch.full((T,), 1.1, device="cuda")
    outs = [torch.zeros(T, d, device="cuda"), torch.zeros(T, d, dtype=BF, device="cuda"),
            torch.zeros(T, d, dtype=BF, device="cuda"), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")]
    nnb = brx.block_norm_backward_workspace_bytes(a)
    nws = ws_of(nnb)
    calls.append(("block_norm_backward",
                  lambda: brx.block_norm_backward(a, dout, du, xr, t["y"], **ins, rstd_y=cy, rstd_r=cr, dx=outs[0],
                                                  dy=outs[1], dgate=outs[2], dg_post=outs[3], dg_pre=outs[4], ws=nws,
                                                  ws_bytes=nnb), [dout, du, xr, t["y"]], outs))
    return calls


def bits(outs):
    torch.cuda.synchronize()
    return [o.clone() for o in outs]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("which", range(11))
def test_graph_replays_equal_eager_calls(which):
    name, run, ins, outs = every_call(5)[which]
    other = every_call(77)[which][2]
    print(f"case graph {name}", flush=True)
    first = [i.clone() for i in ins]
    run()
    eager0 = bits(outs)
    run()
    assert same(bits(outs), eager0), "two calls differ"
    for i, o in zip(ins, other):
        i.copy_(o)
    run()
    eager1 = bits(outs)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run()
    for _ in range(2):
        for source, want in ((first, eager0), (other, eager1)):
            for i, v in zip(ins, source):
                i.copy_(v)
            for o in outs:
                o.zero_()
            if name in ("block_norm_backward",):
                pass
            g.replay()
            assert same(bits(outs), want), "a replay differs from the eager call"
            run()   # eager work between the replays
            assert same(bits(outs), want)


@pytest.mark.parametrize("which", range(11))
def test_calls_on_another_stream(which):
    name, run, ins, outs = every_call(9)[which]
    print(f"case stream {name}", flush=True)
    run()
    want = bits(outs)
    for o in outs:
        o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    assert same(bits(outs), want)


def test_addresses_beside_tensors():
    """Raw addresses may stand for any of the tensors, or for all of them."""
    T, k, E, d = 9, 4, 6, 64
    pos, rows = positions(T, k, E, 0.2, 3).cuda(), T * k
    x = rand(T, d, seed=1).cuda()
    want = torch.zeros(rows, d, device="cuda")
    brx.dispatch(x, 1, T, k, d, pos, want, rows)
    for give in range(8):
        xs = torch.zeros(rows, d, device="cuda")
        a = [t.data_ptr() if give >> i & 1 else t for i, t in enumerate((x, pos, xs))]
        brx.dispatch(a[0], 1, T, k, d, a[1], a[2], rows)
        assert torch.equal(xs, want), give


def test_a_call_whose_device_is_not_current():
    """The call is made once more with its tensors' device current, and on a
    stream that is given; what it returns and raises stays the same."""
    brx.sort_workspace_bytes(1, 1, 1)
    T, k, d, rows = 5, 4, 64, 20
    pos = torch.arange(T * k, dtype=torch.int32, device="cuda")
    x, xs = rand(T, d, seed=1).cuda(), Out(rows, d, dtype=F32)
    brx.dispatch(x, 1, T, k, d, pos, xs.t, rows)
    native = brx.ops._native
    seen = []

    def elsewhere(dev, fn, *args):
        seen.append(dev)
        bind(lambda: 0)
        brx.ops._elsewhere(dev, fn, *args)

    def bind(device):
        lib = brx.load_library()
        native.bind(tuple(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in brx.ops._BOUND), brx.ops._raise,
                    elsewhere, device, torch.cuda.current_device, torch._C._cuda_getCurrentRawStream)
    try:
        for stream in (None, torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
            bind(lambda: 1)   # as if device 1 were current
            out = Out(rows, d, dtype=F32)
            brx.dispatch(x, 1, T, k, d, pos, out.t, rows, stream=stream)
            assert torch.equal(out.guarded(), xs.guarded()) and seen.pop() == 0 and not seen
        bind(lambda: 1)
        with pytest.raises(brx.StrataError) as e:
            brx.dispatch(x, 1, T, 33, d, pos.repeat(9)[:T * 33].contiguous(), xs.t, rows)
        assert e.value.status == brx.STRATA_EINVAL
    finally:
        bind(torch._C._cuda_getDevice)
        brx.ops._native = brx.ops._Unloaded()   # bound anew at the next call
    brx.dispatch(x, 1, T, k, d, pos, xs.t, rows)
    assert brx.ops._native is native


# ------------------------------------------------------------- all together

def test_a_trainable_sparse_block():
    """norm -> route -> sort -> dispatch -> gate/up product -> SwiGLU -> down
    product -> combine -> post norm, gate and residual -> norm, forward and
    backward, against automatic differentiation in 64 bits with the same
    picks.  The rows between the operators are bf16: each of the about ten
    roundings on a path is at most 2^-8 of its value, and independent ones add
    in squares, so outputs and gradients are within 10 * 2^-8 in 2-norm."""
    T, d, E, k, f = 96, 256, 16, 4, 128
    sh = brx.shape(E, k, d, f, 3)
    x = rand(T, d, seed=1)
    Wr, g0, gp, gq = rand(E, d, seed=2, scale=d ** -0.5), 1 + 0.1 * rand(d, seed=3), 1 + 0.1 * rand(d, seed=4), \
        1 + 0.1 * rand(d, seed=5)
    W1, W2 = rand(E, 2 * f, d, seed=6, dtype=BF, scale=d ** -0.5), rand(E, d, f, seed=7, dtype=BF, scale=f ** -0.5)
    gate = rand(T, seed=8)
    cr, cuu = rand(T, d, seed=9), rand(T, d, seed=10, dtype=BF)
    X, WR, G0, GP, GQ, W1c, W2c, GT = (v.cuda() for v in (x, Wr, g0, gp, gq, W1, W2, gate))
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    n = T * k
    # forward
    a0 = brx.block_norm_args(T, d, 1, 0, 0, brx.PRE_NORM)
    u, r0 = e(T, d, dt=BF), e(T)
    brx.block_norm(a0, X, None, g_pre=G0, u=u, rstd_r=r0)
    nb = brx.workspace_bytes(sh, T)
    ro = dict(topk_idx=e(T, k, dt=torch.int32), topk_w=e(T, k))
    brx.route(sh, brx.LayerData(router_w=WR, codes=None, scales=None), u, brx.X_BF16, T, ro, ws_of(nb), nb)
    off, pos = e(E + 1, dt=torch.int32), e(n, dt=torch.int32)
    sb = brx.sort_workspace_bytes(T, k, E)
    brx.sort_picks(ro["topk_idx"], T, k, E, None, off, None, pos, ws_of(sb), sb)
    xs, gu, ys = e(n, d, dt=BF), e(n, 2 * f, dt=BF), e(n, d, dt=BF)
    brx.dispatch(u, 0, T, k, d, pos, xs, n)
    gb = max(brx.grouped_workspace_bytes(n, E, 2 * f, d), brx.grouped_workspace_bytes(n, E, d, f))
    gws = ws_of(gb)
    brx.grouped_product(xs, W1c, off, n, E, 2 * f, d, gu, 0, gws, gb)
    gl, ul = gu.float()[:, :f], gu.float()[:, f:]
    h = (gl * torch.sigmoid(gl) * ul).to(BF)
    brx.grouped_product(h, W2c, off, n, E, d, f, ys, 0, gws, gb)
    y = e(T, d, dt=BF)
    brx.combine(ys, 0, n, pos, ro["topk_w"], T, k, d, y, 0)
    a1 = brx.block_norm_args(T, d, 1, 0, 0, brx.POST_NORM | brx.PRE_NORM | brx.GATE_TOKEN | brx.GATE_SIGMOID, 0.8, 0.6)
    r, u1, sy, sr = e(T, d), e(T, d, dt=BF), e(T), e(T)
    brx.block_norm(a1, X, y, gate=GT, g_post=GP, g_pre=GQ, r=r, u=u1, rstd_y=sy, rstd_r=sr)
    # backward of <cr, r> + <cu, u1>
    dX, dy, dgt, dgp, dgq = e(T, d), e(T, d, dt=BF), e(T), e(d), e(d)
    wb = brx.block_norm_backward_workspace_bytes(a1)
    brx.block_norm_backward(a1, cr.cuda(), cuu.cuda(), r, y, gate=GT, g_post=GP, g_pre=GQ, rstd_y=sy, rstd_r=sr,
                            dx=dX, dy=dy, dgate=dgt, dg_post=dgp, dg_pre=dgq, ws=ws_of(wb), ws_bytes=wb)
    dys, dz = e(n, d, dt=BF), e(T, k)
    brx.combine_backward(dy, 0, ys, 0, n, pos, ro["topk_w"], T, k, d, dys=dys, dz=dz)
    dh, dxs = e(n, f), e(n, d, dt=BF)
    dW1, dW2 = e(E, 2 * f, d), e(E, d, f)
    brx.grouped_dgrad(dys, W2c, off, n, E, d, f, dh, 1, gws, gb)
    brx.grouped_wgrad(dys, h, off, n, E, d, f, dW2, 1, gws, gb)
    sg = torch.sigmoid(gl)
    dgu = torch.cat([dh * ul * sg * (1 + gl * (1 - sg)), dh * gl * sg], 1).to(BF)
    brx.grouped_dgrad(dgu, W1c, off, n, E, 2 * f, d, dxs, 0, gws, gb)
    brx.grouped_wgrad(dgu, xs, off, n, E, 2 * f, d, dW1, 1, gws, gb)
    du = e(T, d, dt=BF)
    brx.dispatch_backward(dxs, 0, n, pos, T, k, d, du)
    zfull = torch.zeros(T, E, device="cuda").scatter_(1, ro["topk_idx"].long(), dz)
    dWr = zfull.t().contiguous() @ u.float()
    du_all = (du.float() + zfull @ WR).to(BF)
    dXn, dg0 = e(T, d), e(d)
    wb0 = brx.block_norm_backward_workspace_bytes(a0)
    brx.block_norm_backward(a0, dX, du_all, X, None, g_pre=G0, rstd_r=r0, dx=dXn, dg_pre=dg0, ws=ws_of(wb0),
                            ws_bytes=wb0)
    torch.cuda.synchronize()
    # the same in 64 bits
    L = {m: v.double().clone().requires_grad_(True) for m, v in
         dict(x=x, Wr=Wr, g0=g0, gp=gp, gq=gq, W1=W1, W2=W2, gate=gate).items()}
    idx = ro["topk_idx"].cpu().long()
    ud = R.norm_rows(L["x"], L["g0"], f32(1e-6))
    z = ud @ L["Wr"].t()
    wd = torch.softmax(z.gather(1, idx), 1)
    yd = torch.zeros(T, d, dtype=torch.float64)
    for q in range(k):
        guv = torch.bmm(L["W1"][idx[:, q]], ud[:, :, None])[:, :, 0]
        hv = torch.nn.functional.silu(guv[:, :f]) * guv[:, f:]
        yd = yd + wd[:, q:q + 1] * torch.bmm(L["W2"][idx[:, q]], hv[:, :, None])[:, :, 0]
    rd, u1d, _, _ = R.block_norm(L["x"], yd, L["gate"], L["gp"], L["gq"], post=True, pre=True, sigmoid=True, a=f32(0.8),
                                 b=f32(0.6), eps=f32(1e-6))
    loss = (rd * cr.double()).sum() + (u1d * cuu.double()).sum()
    names = ("x", "Wr", "g0", "gp", "gq", "W1", "W2", "gate")
    grads = dict(zip(names, torch.autograd.grad(loss, [L[m] for m in names])))
    bound = 10 * 2.0 ** -8
    for m, got, ref in (("r", r, rd), ("u", u1, u1d), ("x", dXn, grads["x"]), ("Wr", dWr, grads["Wr"]),
                        ("g0", dg0, grads["g0"]), ("g_post", dgp, grads["gp"]), ("g_pre", dgq, grads["gq"]),
                        ("W1", dW1, grads["W1"]), ("W2", dW2, grads["W2"]), ("gate", dgt, grads["gate"])):
        ref = ref.detach()
        off_by = float((got.cpu().double() - ref).norm() / ref.norm())
        print(f"  {m}: {off_by:.2e}", flush=True)
        assert off_by <= bound, f"{m}: off by {off_by:.3e} in 2-norm"
