"""The operators around the layer on every kernel that the library's rules
choose between: experts that do not touch each other in any tile, calls whose
first launch hands data to the next, replayed with other picks, and norm
gradients of every width with more rows than blocks."""
from __future__ import annotations

import pytest
import torch

import bit_routed_expert_amd as brx
from tests import test_gpu_ops as T

pytestmark = pytest.mark.gpu

BF, F32 = T.BF, T.F32


# ------------------------------------- the tiles of the experts' products

def rows_tile(rows, E, Nn, K=None):
    """What runs a product (K given: the forward one) or the rows' gradient
    with Nn output columns: "few", or the tile's rows and whether a launch
    before lists the tiles.  The rule of the library's launch code, restated."""
    if K is not None and rows * 4 <= E and K <= 8192:
        return "few"
    up = lambda a, b: -(-a // b)  # noqa: E731
    tiles64 = (rows // 64 + (E + 1) // 2) * up(Nn, 128)
    if rows <= 16 * E or tiles64 < 128:
        bm, bn = 32, 128
    elif tiles64 <= 256:
        bm, bn = 64, 128
    elif rows < 384 * E or rows // 256 * up(Nn, 256) < 192:
        bm, bn = 128, 256
    else:
        bm, bn = 256, 256
    blocks = up((rows // bm + min(rows, E)) * up(Nn, bn), 8) * 8
    return bm, bm != 64 and blocks > 512


def weights_tile(rows, E, N, K):
    """The same for the weights' gradient: tile, and whether experts are taken by falling row count."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    large, small = E * up(N, 256) * up(K, 256), E * up(N, 128) * up(K, 128)
    t = 256 if large >= 1024 or (large >= 512 and rows >= 512 * E) else 128 if small >= 256 else 64
    return t, E <= 64


TILES = [  # rows per expert, N, K; what runs product, dgrad and wgrad
    ([1, 2, 0, 1] + [0] * 30, 264, 136, "few", (32, False), (64, True)),
    ([300, 200, 7, 0, 260], 1224, 136, (64, False), (32, False), (64, True)),
    ([300, 200, 7, 0, 260], 136, 1224, (32, False), (64, False), (64, True)),
    ([120, 118, 122] * 13, 520, 264, (128, False), (128, False), (128, True)),
    ([120, 118, 122] * 20, 1288, 264, (128, True), (128, False), (128, True)),
    ([120, 118, 122] * 20, 264, 1288, (128, False), (128, True), (128, True)),
    ([9000, 8000, 9003], 520, 136, (256, False), (128, False), (64, True)),
    ([9000, 8000, 9003], 1288, 520, (256, True), (256, False), (64, True)),
    ([9000, 8000, 9003], 520, 1288, (256, False), (256, True), (64, True)),
    ([3, 1, 5] * 100, 520, 264, (32, True), (32, True), (256, False)),
    ([(7 * i) % 90 + 1 for i in range(40)], 1288, 1288, (128, False), (128, False), (256, True)),
    ([16 * (i % 25) + i % 3 + 1 for i in range(70)], 264, 264, (128, False), (128, False), (128, False)),
    ([40, 1, 33, 7] * 25, 64, 64, (32, False), (32, False), (64, False)),
]


@pytest.mark.parametrize("ns,N,K,product,dgrad,wgrad", TILES)
def test_experts_do_not_touch_each_other_in_any_tile(ns, N, K, product, dgrad, wgrad):
    """NaN and infinity in one expert's rows and weights leave the bits of all
    the others' results as they were, and none of its own finite."""
    E, rows = len(ns), sum(ns)
    assert rows_tile(rows, E, N, K) == product and rows_tile(rows, E, K) == dgrad
    assert weights_tile(rows, E, N, K) == wgrad
    print(f"case apart {ns[:4]} N={N} K={K} {product} {dgrad} {wgrad}", flush=True)
    _, off, x, dy, W = T.group_inputs(ns, N, K, 0)
    nb = brx.grouped_workspace_bytes(rows, E, N, K)
    ws, oc = T.ws_of(nb), off.cuda()
    xc, yc, Wc = x.cuda(), dy.cuda(), W.cuda()
    bad = 1
    a, b = int(off[bad]), int(off[bad + 1])

    def run(ot):
        outs = T.Out(rows, N, dtype=ot), T.Out(rows, K, dtype=ot), T.Out(E, N, K, dtype=ot)
        brx.grouped_product(xc, Wc, oc, rows, E, N, K, outs[0].t, T.CODE[ot], ws, nb)
        print("  product", flush=True)
        brx.grouped_dgrad(yc, Wc, oc, rows, E, N, K, outs[1].t, T.CODE[ot], ws, nb)
        print("  dgrad", flush=True)
        brx.grouped_wgrad(yc, xc, oc, rows, E, N, K, outs[2].t, T.CODE[ot], ws, nb)
        print("  wgrad", flush=True)
        return [o.guarded() for o in outs]
    clean = {ot: run(ot) for ot in (BF, F32)}
    xc[a:b], yc[a:b], Wc[bad] = float("nan"), float("inf"), float("nan")
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[a:b] = False
    for ot in (BF, F32):
        got = run(ot)
        for g, c in zip(got[:2], clean[ot][:2]):
            assert bool(torch.isfinite(c).all())
            assert torch.equal(g[others], c[others]) and not bool(torch.isfinite(g[a:b]).any())
        keep = [e for e in range(E) if e != bad]
        assert torch.equal(got[2][keep], clean[ot][2][keep]) and not bool(torch.isfinite(got[2][bad]).any())


@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("N,K", [(1224, 200), (200, 1224)])
def test_products_in_64_row_tiles(N, K, ot):
    """Bf16 and fp32 stores of the 64-row tiles, rows of NaN behind the last expert's."""
    ns, tail = [300, 200, 7, 0, 260], 3
    Nn = max(N, K)
    assert rows_tile(sum(ns) + tail, len(ns), Nn) == (64, False)
    T.test_grouped_products(ns, N, K, tail, ot)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("E,rows,N,K", [(60, 7203, 1288, 264), (60, 7203, 264, 1288), (300, 900, 520, 264),
                                        (300, 60, 520, 264), (3, 26000, 1288, 136), (70, 900, 136, 264)])
def test_listed_tiles_of_offsets_that_do_not_ascend_stay_inside(E, rows, N, K, seed):
    """As with few experts: which rows such offsets mean is not specified, nothing outside the buffers is written."""
    print(f"case garbage offsets E={E} rows={rows} seed={seed}", flush=True)
    g = T.gen(seed)
    off = torch.randint(-rows, 2 * rows, (E + 1,), generator=g, dtype=torch.int32)
    if seed == 3:
        ends = torch.tensor([-2**31, 2**31 - 1], dtype=torch.int32)[torch.randint(0, 2, (E + 1,), generator=g)]
        off = torch.where(torch.rand(E + 1, generator=g) < 0.5, ends, off)
    _, _, x, dy, W = T.group_inputs([rows], N, K, 0)
    Wc = W.cuda().repeat(E, 1, 1)
    nb = brx.grouped_workspace_bytes(rows, E, N, K)
    wsb = torch.full((nb + T.GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    o, xc, yc = off.cuda(), x.cuda(), dy.cuda()
    outs = T.Out(rows, N, dtype=F32), T.Out(rows, K, dtype=BF), T.Out(E, N, K, dtype=BF)
    brx.grouped_product(xc, Wc, o, rows, E, N, K, outs[0].t, 1, wsb, nb)
    outs[0].guarded()
    brx.grouped_dgrad(yc, Wc, o, rows, E, N, K, outs[1].t, 0, wsb, nb)
    outs[1].guarded()
    brx.grouped_wgrad(yc, xc, o, rows, E, N, K, outs[2].t, 0, wsb, nb)
    outs[2].guarded()
    assert bool((wsb[nb:] == 0x5A).all())


# ----------------------------- graphs and streams, with other picks each time

def split(rows, E, seed):
    """Offsets that deal rows unevenly to E experts, some with none."""
    cuts = torch.randint(0, rows + 1, (E - 1,), generator=T.gen(seed), dtype=torch.int32).sort().values
    ends = torch.tensor([0]), cuts, torch.tensor([rows])
    return torch.cat([v.to(torch.int32) for v in ends]).cuda()


def i32(n):
    return torch.zeros(n, dtype=torch.int32, device="cuda")


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def sort_call(seed):
    t, k, E = 17000, 4, 6
    assert t * k > 65535
    idx = T.draw_idx(t, k, E, 0.1, seed).cuda()
    nb = brx.sort_workspace_bytes(t, k, E)
    outs, ws = [i32(E), i32(E + 1), i32(t * k), i32(t * k)], T.ws_of(nb)
    return lambda: brx.sort_picks(idx, t, k, E, *outs, ws, nb), [idx], outs


def row_call(seed, name):
    t, k, d, rows = 70, 4, 264, 280
    pos = T.positions(t, k, 6, 0.1, seed).cuda()
    x, ys = T.rand(t, d, seed=seed, dtype=BF).cuda(), T.rand(rows, d, seed=seed + 1, dtype=BF).cuda()
    w, dout = torch.softmax(T.rand(t, k, seed=seed + 2), 1).cuda(), T.rand(t, d, seed=seed + 3).cuda()
    if name == "dispatch":
        xs = zeros(rows, d, dtype=BF)
        return lambda: brx.dispatch(x, 0, t, k, d, pos, xs, rows), [x, pos], [xs]
    if name == "dispatch_backward":
        dx = zeros(t, d, dtype=BF)
        return lambda: brx.dispatch_backward(ys, 0, rows, pos, t, k, d, dx), [ys, pos], [dx]
    if name == "combine":
        out = zeros(t, d)
        return lambda: brx.combine(ys, 0, rows, pos, w, t, k, d, out, 1), [ys, pos, w], [out]
    outs = [zeros(rows, d, dtype=BF), zeros(t, k), zeros(t, k)]
    return lambda: brx.combine_backward(dout, 1, ys, 0, rows, pos, w, t, k, d, *outs), [dout, ys, pos, w], outs


SHAPES = {  # experts, rows, N, K; what runs product and dgrad
    "listed 128-row tiles": (60, 7203, 1288, 264, (128, True), (128, False)),
    "listed 128-row tiles across": (60, 7203, 264, 1288, (128, False), (128, True)),
    "listed 32-row tiles": (300, 900, 520, 264, (32, True), (32, True)),
    "few rows": (300, 60, 520, 264, "few", (32, False)),
    "tiles found by each block": (6, 280, 136, 264, (32, False), (32, False))}


def product_call(seed, name, shape):
    E, rows, N, K, forward, across = SHAPES[shape]
    assert (rows_tile(rows, E, N, K), rows_tile(rows, E, K)) == (forward, across)
    off = split(rows, E, seed + E)
    x, dy = T.rand(rows, K, seed=seed + 4, dtype=BF).cuda(), T.rand(rows, N, seed=seed + 5, dtype=BF).cuda()
    W = T.rand(E, N, K, seed=seed + 6, dtype=BF).cuda()
    nb = brx.grouped_workspace_bytes(rows, E, N, K)
    ws = T.ws_of(nb)
    if name == "product":
        y = zeros(rows, N)
        return lambda: brx.grouped_product(x, W, off, rows, E, N, K, y, 1, ws, nb), [x, W, off], [y]
    if name == "dgrad":
        dx = zeros(rows, K)
        return lambda: brx.grouped_dgrad(dy, W, off, rows, E, N, K, dx, 1, ws, nb), [dy, W, off], [dx]
    dW = zeros(E, N, K, dtype=BF)
    return lambda: brx.grouped_wgrad(dy, x, off, rows, E, N, K, dW, 0, ws, nb), [dy, x, off], [dW]


def norm_call(seed):
    t, d = 2100, 514
    a, q = T.norm_case(t, d, F32, BF, BF, True, True, "channel", True, seed)
    q = {n: T.cu(v) for n, v in q.items()}
    dr, du, r = T.rand(t, d, seed=seed + 7).cuda(), T.rand(t, d, seed=seed + 8, dtype=BF).cuda(), \
        T.rand(t, d, seed=seed + 9).cuda()
    ry, rr = T.rand(t, seed=seed + 10).cuda(), T.rand(t, seed=seed + 11).cuda()
    outs = [zeros(t, d), zeros(t, d, dtype=BF), zeros(t, d, dtype=BF), zeros(d), zeros(d)]
    nb = brx.block_norm_backward_workspace_bytes(a)
    ws = T.ws_of(nb)
    return lambda: brx.block_norm_backward(
        a, dr, du, r, q["y"], gate=q["gate"], g_post=q["g_post"], g_pre=q["g_pre"], rstd_y=ry, rstd_r=rr, dx=outs[0],
        dy=outs[1], dgate=outs[2], dg_post=outs[3], dg_pre=outs[4], ws=ws, ws_bytes=nb), \
        [dr, du, r, q["y"], q["gate"], q["g_post"], q["g_pre"], ry, rr], outs


# Calls whose work depends on picks: (run, every input that it reads, outputs) from a seed.
CALLS = {"sort of two launches": sort_call, "norm gradient of two launches": norm_call}
CALLS |= {n: (lambda s, n=n: row_call(s, n)) for n in ("dispatch", "dispatch_backward", "combine", "combine_backward")}
CALLS |= {f"{n}, {shape}": (lambda s, n=n, shape=shape: product_call(s, n, shape))
          for n in ("product", "dgrad", "wgrad") for shape in SHAPES}


def eager(run, outs):
    for o in outs:
        o.zero_()
    run()
    return T.bits(outs)


@pytest.mark.parametrize("name", CALLS)
def test_replays_follow_the_picks(name):
    """A captured call replayed with other picks, offsets and rows gives the eager call's bits for them."""
    print(f"case replay {name}", flush=True)
    run, ins, outs = CALLS[name](5)
    first, other = [i.clone() for i in ins], CALLS[name](77)[1]
    assert all(not torch.equal(p, q) for p, q in zip(first, other))
    want0 = eager(run, outs)
    for i, v in zip(ins, other):
        i.copy_(v)
    want1 = eager(run, outs)
    assert not T.same(want0, want1)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        for source, want in ((first, want0), (other, want1)):
            for i, v in zip(ins, source):
                i.copy_(v)
            for o in outs:
                o.zero_()
            g.replay()
            assert T.same(T.bits(outs), want), "a replay differs from the eager call"
            assert T.same(eager(run, outs), want)


@pytest.mark.parametrize("name", CALLS)
def test_the_same_on_another_stream(name):
    print(f"case stream {name}", flush=True)
    run, ins, outs = CALLS[name](9)
    want = eager(run, outs)
    for o in outs:
        o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    assert T.same(T.bits(outs), want)


@pytest.mark.parametrize("name", CALLS)
def test_two_at_once(name):
    """Two calls under way together on two streams, each with its own workspace and outputs."""
    print(f"case two at once {name}", flush=True)
    pair = [CALLS[name](s) for s in (5, 77)]
    want = [eager(run, outs) for run, _, outs in pair]
    for _, _, outs in pair:
        for o in outs:
            o.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for st, (run, _, _) in zip(streams, pair):
            with torch.cuda.stream(st):
                run()
    torch.cuda.synchronize()
    for (_, _, outs), w in zip(pair, want):
        assert T.same(T.bits(outs), w)


# --------------------------------- norms of every width, more rows than blocks

WIDTHS = [  # widths that 8 does not divide, and all above 4096; T above the 512 blocks' rows
    (2100, 130, F32, BF, BF, True, True, "channel", True), (2100, 515, BF, F32, F32, True, True, "token", True),
    (2100, 1002, BF, BF, F32, True, True, "channel", False), (2100, 1001, F32, F32, BF, False, True, "token", False),
    (1100, 1030, F32, BF, BF, True, True, "token", True), (1100, 2047, BF, BF, BF, True, True, "channel", True),
    (1100, 2050, BF, F32, F32, True, True, None, False), (700, 4095, F32, BF, F32, True, True, "channel", False),
    (700, 4098, F32, F32, BF, True, True, "token", True), (600, 4097, BF, BF, BF, True, True, "channel", True),
    (600, 8190, F32, BF, BF, True, True, "channel", True), (600, 8191, BF, F32, F32, True, True, "token", False),
    (600, 4104, BF, BF, BF, True, True, "channel", True), (600, 8192, F32, F32, F32, True, True, "token", True)]


@pytest.mark.parametrize("case", WIDTHS)
def test_block_norm_of_every_width(case):
    T.test_block_norm(case)


@pytest.mark.parametrize("case", WIDTHS)
def test_block_norm_backward_of_every_width(case):
    T.test_block_norm_backward(case)


@pytest.mark.parametrize("case", [c for c in WIDTHS if c[1] % 8])
def test_norm_gradients_twice_give_the_same_bits(case):
    n, d = case[:2]
    a, t = T.norm_case(*case)
    t = {m: T.cu(v) for m, v in t.items()}
    dr, du = T.rand(n, d, seed=31, dtype=case[2]).cuda(), T.rand(n, d, seed=32, dtype=case[4]).cuda()
    ry, rr = (torch.full((n,), 0.9, device="cuda") if case[5] else None), torch.full((n,), 1.1, device="cuda")
    nb = brx.block_norm_backward_workspace_bytes(a)
    runs = []
    for fill in (0x00, 0xFF):   # whatever the workspace holds
        o = [T.Out(n, d, dtype=case[2]), T.Out(n, d, dtype=case[3]), T.Out(d, dtype=F32), T.Out(d, dtype=F32)]
        ws = torch.full((nb,), fill, dtype=torch.uint8, device="cuda")
        brx.block_norm_backward(a, dr, du, t["x"], t["y"], gate=t["gate"], g_post=t["g_post"], g_pre=t["g_pre"],
                                rstd_y=ry, rstd_r=rr, dx=o[0].t, dy=o[1].t, dg_post=o[2].t if case[5] else None,
                                dg_pre=o[3].t, ws=ws, ws_bytes=nb)
        runs.append([q.guarded() for q in o])
    assert T.same(*runs)
