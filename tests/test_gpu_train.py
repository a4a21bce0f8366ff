"""The ends of a training step on the GPU: balance losses, embedding,
vocabulary loss and orthogonalised updates, each with its gradient, against
the 64-bit forms of train_ref at the sizes and masks where they can go wrong,
with guard bands behind every output; captured and replayed in graphs, on
other streams, twice with the same bits, and together with the sparse block as
one training step."""
from __future__ import annotations

import pytest
import torch

import bit_routed_expert_amd as brx
from tests import ops_ref as O
from tests import train_ref as R
from tests.test_gpu_ops import BF, CODE, F32, Out, bits, draw_idx, gen, rand, same, ws_of

pytestmark = pytest.mark.gpu

U = O.U
INF, NAN = float("inf"), float("nan")
f32 = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731


def check(got, ref, bound, what):
    """As ops_ref.check; references may live on the GPU."""
    O.check(got.cpu(), ref.cpu(), bound.cpu() if isinstance(bound, torch.Tensor) else bound, what)


# ---------------------------------------------------------------- balance

BALANCE = [(1, 1, 1), (1, 4, 8), (5, 10, 512), (7, 3, 5), (64, 2, 64), (65, 8, 256), (100, 32, 1024), (333, 5, 130),
           (1000, 6, 257), (2500, 4, 60), (77, 3, 514), (8300, 2, 16), (9000, 10, 512)]


def balance_case(T, k, E, dt, seed, masked):
    g = gen(seed)
    z = (torch.randn(T, E, generator=g) * 2).to(dt)
    idx = draw_idx(T, k, E, 0.1 if masked else 0.0, seed + 1)
    keep = None
    if masked:
        keep = (torch.rand(T, generator=g) < 0.8).to(torch.uint8)
        z[torch.rand(T, E, generator=g) < 0.2] = -INF          # masked experts
        z[torch.rand(T, generator=g) < 0.1] = -INF             # rows whose mask leaves nothing
        z[keep == 0] = NAN                                     # padding holds anything
        if T > 4:
            z[2], keep[2] = torch.finfo(dt).min, 1             # a mask of the type's lowest value, everywhere
    return z, idx, keep


def run_balance(z, idx, keep, T, k, E):
    losses, counts, prob = Out(2, dtype=F32), Out(E, dtype=torch.int32, fill=-9), Out(E, dtype=F32)
    lse, tokens = Out(T, dtype=F32), Out(1, dtype=torch.int32, fill=-9)
    nb = brx.balance_loss_workspace_bytes(T, k, E)
    brx.balance_loss(z, CODE[z.dtype], idx, T, k, E, losses.t, counts.t, lse.t, tokens.t, ws_of(nb), nb, prob=prob.t, keep=keep)
    return [o.guarded() for o in (losses, counts, prob, lse, tokens)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,k,E", BALANCE)
def test_balance(T, k, E, dt, masked):
    print(f"case balance T={T} k={k} E={E} {dt} masked={masked}", flush=True)
    z, idx, keep = balance_case(T, k, E, dt, T + E, masked)
    zc, ic, kc = z.cuda(), idx.cuda(), None if keep is None else keep.cuda()
    losses, counts, prob, lse, tokens = run_balance(zc, ic, kc, T, k, E)
    on = R.counted(z, keep)
    lowest = T > 4 and masked and bool(on[2])
    zd = z.double()
    zd[~on] = 0
    leaf = zd.clone().requires_grad_(True)
    rl, rc, rp, rs, n = R.balance(torch.where(on[:, None], leaf, torch.full_like(leaf, -INF)), idx, keep, E)
    assert counts.cpu().tolist() == rc.tolist() and int(tokens) == n
    finite = torch.where(torch.isfinite(zd), zd, torch.zeros_like(zd))
    x = (zd.max(1).values[:, None] - zd)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).clamp(max=110.0)   # far down the exponential is 0
    rs = rs.detach()
    span = float(x.max())
    err = (E + 2 * span + 16) * U                      # relative, of a row's sum of exponentials
    b_lse = err + 2 * U * (rs.abs() + finite.abs().max(1).values)
    check(lse, rs, torch.where(on, b_lse, torch.zeros_like(b_lse)), "lse")
    rp = rp.detach()
    check(prob, rp, (2 * err + (T + 16) * U) * rp, "prob")
    ref = rl.detach()
    if n:
        b0 = (2 * err + (T + E + 24) * U) * ref[0]
        check(losses[:1], ref[:1], b0, "balance")
        if not lowest:   # its squared normaliser is past fp32
            check(losses[1:], ref[1:], (2 * rs.abs() * b_lse * on).sum() / n + (T + 16) * U * ref[1], "z loss")
        else:
            assert float(losses[1]) == INF
    else:
        assert losses.tolist() == [0.0, 0.0] and not prob.any()
    # the gradient, with and without the picks'
    dl = torch.tensor([0.7, 0.0 if lowest else 0.3])
    dp = rand(T, k, seed=9)
    dp[~on] = NAN
    for dpicks in (None, dp):
        dz = Out(T, E, dtype=dt)
        brx.balance_loss_backward(zc, CODE[dt], ic, T, k, E, lse, counts, tokens, dl.cuda(), dz.t, keep=kc,
                                  dpicks=None if dpicks is None else dpicks.cuda())
        p = torch.where(on[:, None], torch.exp(zd - rs[:, None]), torch.zeros_like(zd))
        nn = max(n, 1)
        g = float(dl[0].double()) * E * rc.double() / (nn * nn * k)
        zl = torch.where(on, 2 * float(dl[1].double()) * rs / nn, torch.zeros_like(rs))[:, None]
        want = p * (g - (p * g).sum(1, keepdim=True) + zl)
        mag = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True) + zl.abs())
        # p from the stored lse (its error and rounding), the sums, eight more roundings
        bound = (2 * b_lse[:, None] + (2 * x + E + 24) * U + U * rs.abs()[:, None]) * mag
        if dpicks is not None:
            for t in on.nonzero().flatten().tolist():
                for r in range(k):
                    e = int(idx[t, r])
                    if 0 <= e < E:
                        want[t, e] += float(dp[t, r].double())
                        bound[t, e] += (k + 2) * U * abs(float(dp[t, r]))
            bound = bound + U * want.abs()
        check(dz.guarded(), want, bound, "dz")
        if dpicks is None and n and not lowest:   # the closed form is the definition's
            auto, = torch.autograd.grad((rl * dl.double()).sum(), leaf, retain_graph=True)
            assert torch.allclose(torch.where(on[:, None], auto, torch.zeros_like(auto)), want, atol=1e-12)
        again = zc.clone()
        brx.balance_loss_backward(again, CODE[dt], ic, T, k, E, lse, counts, tokens, dl.cuda(), again, keep=kc,
                                  dpicks=None if dpicks is None else dpicks.cuda())   # over z
        assert torch.equal(again, dz.t)


def test_balance_without_tokens_and_without_kept_ones():
    for T, keep in ((0, None), (3, torch.zeros(3, dtype=torch.bool)), (500, torch.zeros(500, dtype=torch.uint8))):
        E, k = 70, 2
        z, idx = torch.full((T, E), NAN).cuda(), torch.zeros(T, k, dtype=torch.int32).cuda()
        losses, counts, prob, lse, tokens = run_balance(z, idx, None if keep is None else keep.cuda(), T, k, E)
        assert not losses.any() and not counts.any() and not prob.any() and not lse.any() and int(tokens) == 0
        dz = Out(T, E, dtype=F32)
        if T:
            brx.balance_loss_backward(z, 1, idx, T, k, E, lse, counts, tokens, torch.ones(2).cuda(), dz.t, keep=keep.cuda())
            assert not dz.guarded().any()


def test_balance_nan_stays_in_its_row():
    """A logit of NaN or +inf in a token that counts shows in that token's lse and gradient, and in the losses, not in others' rows."""
    T, k, E = 9, 2, 40
    z = rand(T, E, seed=3)
    z[4, 7], z[6] = NAN, -INF
    z[6, 3] = NAN
    idx = draw_idx(T, k, E, 0.0, 5).cuda()
    losses, counts, prob, lse, tokens = run_balance(z.cuda(), idx, None, T, k, E)
    ok = torch.tensor([t not in (4, 6) for t in range(T)])
    assert bool(lse.cpu()[ok].isfinite().all()) and bool(lse.cpu()[~ok].isnan().all()) and int(tokens) == T
    assert bool(losses.isnan().all()) and int(counts.sum()) == T * k
    dz = Out(T, E, dtype=F32)
    brx.balance_loss_backward(z.cuda(), 1, idx, T, k, E, lse, counts, tokens, torch.ones(2).cuda(), dz.t)
    assert bool(dz.guarded().cpu()[ok].isfinite().all()) and bool(dz.t.cpu()[~ok].isnan().any(1).all())


def test_balance_of_several_calls():
    """The gradient of losses over two calls' tokens, from the summed counts and tokens."""
    T, k, E = 150, 4, 64
    z, idx = rand(2 * T, E, seed=1), draw_idx(2 * T, k, E, 0.0, 2)
    parts = [run_balance(z[s].cuda(), idx[s].cuda(), None, T, k, E) for s in (slice(0, T), slice(T, 2 * T))]
    whole = run_balance(z.cuda(), idx.cuda(), None, 2 * T, k, E)
    counts, tokens = parts[0][1] + parts[1][1], parts[0][4] + parts[1][4]
    assert torch.equal(counts, whole[1]) and torch.equal(tokens, whole[4])
    dl = torch.tensor([0.5, 0.25]).cuda()
    want, got = torch.empty(2 * T, E, device="cuda"), torch.empty(2 * T, E, device="cuda")
    brx.balance_loss_backward(z.cuda(), 1, idx.cuda(), 2 * T, k, E, whole[3], whole[1], whole[4], dl, want)
    for i, s in enumerate((slice(0, T), slice(T, 2 * T))):
        brx.balance_loss_backward(z[s].cuda(), 1, idx[s].cuda(), T, k, E, parts[i][3], counts, tokens, dl, got[s])
    assert torch.equal(got, want)


# ------------------------------------------------------------- embedding

def draw_ids(T, V, seed, pad=0.15):
    """Ids of a few frequent rows, many rare ones, and padding of every kind."""
    g = gen(seed)
    ids = torch.exp(torch.rand(T, generator=g) * torch.log(torch.tensor(float(V)))).long().clamp(1, V) - 1
    ids = torch.randperm(V, generator=g)[ids].to(torch.int32)
    bad = torch.tensor([-1, V, -2**31, 2**31 - 1], dtype=torch.int32)[torch.randint(0, 4, (T,), generator=g)]
    return torch.where(torch.rand(T, generator=g) < pad, bad, ids)


EMBED = [(1, 1, 1), (1, 7, 8), (5, 1000, 2048), (17, 3, 130), (33, 1024, 65), (40, 1025, 264), (300, 2, 1000),
         (1000, 5000, 72), (513, 40, 2056), (2000, 70000, 31)]


@pytest.mark.parametrize("ot", [BF, F32])
@pytest.mark.parametrize("wt", [BF, F32])
@pytest.mark.parametrize("T,V,d", EMBED)
def test_embed(T, V, d, wt, ot):
    print(f"case embed T={T} V={V} d={d} {wt} {ot}", flush=True)
    ids, scale = draw_ids(T, V, T + V), 1.7
    W = rand(V, d, seed=1, dtype=wt)
    out = Out(T, d, dtype=ot)
    brx.embed(W.cuda(), CODE[wt], V, d, ids.cuda(), T, scale, out.t, CODE[ot])
    ref = R.embed(W.double(), ids, f32(scale))
    check(out.guarded(), ref, U * ref.abs(), "out")
    # the gradient: rows of padding hold NaN
    dout = rand(T, d, seed=2, dtype=ot)
    dout[(ids < 0) | (ids >= V)] = NAN
    ref, mag, n = R.embed_backward(dout.double(), ids, V, f32(scale))
    nb = brx.embed_backward_workspace_bytes(T, V, d)
    dW = Out(V, d, dtype=wt)
    brx.embed_backward(dout.cuda(), CODE[ot], ids.cuda(), T, V, d, scale, dW.t, CODE[wt], ws_of(nb), nb)
    got = dW.guarded()
    assert not got.cpu()[n == 0].any()
    check(got, ref, (n[:, None] + 2) * U * mag, "dW")
    base = rand(V, d, seed=3, dtype=wt)
    add = Out(V, d, dtype=wt)
    add.t.copy_(base)
    brx.embed_backward(dout.cuda(), CODE[ot], ids.cuda(), T, V, d, scale, add.t, CODE[wt], ws_of(nb), nb, flags=brx.ACCUMULATE)
    got = add.guarded()
    assert torch.equal(got.cpu()[n == 0], base[n == 0])
    check(got, ref + base.double(), (n[:, None] + 3) * U * (mag + base.double().abs()), "dW added")


@pytest.mark.parametrize("T,V,d,kind", [(100000, 3000, 24, "mixed"), (70000, 1, 8, "one"), (4100, 1 << 19, 8, "one"),
                                        (65536, (1 << 20) - 1, 4, "mixed"), (5000, 600, 264, "runs"), (16, 9, 8, "one"),
                                        (32, 9, 8, "one"), (300, 50000, 40, "none")])
def test_embed_gradient_of_long_runs_and_many_tokens(T, V, d, kind):
    """Runs of equal ids over many chunks, sorts of two launches, the highest ids."""
    print(f"case embed gradient T={T} V={V} d={d} {kind}", flush=True)
    if kind == "one":
        ids = torch.full((T,), V - 1, dtype=torch.int32)
    elif kind == "none":
        ids = torch.full((T,), -1, dtype=torch.int32)
    elif kind == "runs":   # ids in order: runs that end at, before and behind the chunks' borders
        ids = torch.repeat_interleave(torch.arange(V, dtype=torch.int32), torch.arange(V) % 50)[:T]
        ids = torch.cat([ids, torch.full((T - len(ids),), V - 1, dtype=torch.int32)])
    else:
        ids = draw_ids(T, V, 5)
    dout = rand(T, d, seed=6)
    ref, mag, n = R.embed_backward(dout.double(), ids, V, 0.5)
    nb = brx.embed_backward_workspace_bytes(T, V, d)
    first = None
    for _ in range(2):
        dW = Out(V, d, dtype=F32)
        brx.embed_backward(dout.cuda(), 1, ids.cuda(), T, V, d, 0.5, dW.t, 1, ws_of(nb), nb)
        got = dW.guarded()
        first = got if first is None else first
        assert torch.equal(first, got)
    check(got, ref, (n[:, None] + 2) * U * mag, "dW")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,V,d,kind", [(256, 5001, 33, "mixed"), (257, 5001, 33, "mixed"), (256, (1 << 20) - 1, 3, "mixed"),
                                        (255, 700, 5002, "one"), (272, 9, 8, "one"), (257, 1, 1, "one"), (64, 2049, 130, "none"),
                                        (256, 4097, 24, "pairs")])
def test_embed_gradient_about_the_border_of_one_launch(T, V, d, kind, dt):
    """Few tokens (one launch) and just more: every row between them zero, or left as it was, runs of all lengths."""
    print(f"case embed border T={T} V={V} d={d} {kind} {dt}", flush=True)
    ids = draw_ids(T, V, 8)
    if kind == "one":
        ids = torch.full((T,), V - 1, dtype=torch.int32)
    elif kind == "none":
        ids = torch.full((T,), V, dtype=torch.int32)
    elif kind == "pairs":   # the same id far apart, the first and the last rows
        ids = torch.arange(T, dtype=torch.int32) % (T // 2)
        ids[::7] = V - 1
    dout = rand(T, d, seed=6, dtype=dt)
    ref, mag, n = R.embed_backward(dout.double(), ids, V, -0.5)
    nb = brx.embed_backward_workspace_bytes(T, V, d)
    base = rand(V, d, seed=3, dtype=dt)
    for flags in (0, brx.ACCUMULATE):
        dW = Out(V, d, dtype=dt)
        if flags:
            dW.t.copy_(base)
        brx.embed_backward(dout.cuda(), CODE[dt], ids.cuda(), T, V, d, -0.5, dW.t, CODE[dt], ws_of(nb), nb, flags=flags)
        got, was = dW.guarded().cpu(), base if flags else torch.zeros_like(base)
        assert torch.equal(got[n == 0], was[n == 0])
        check(got, ref + was.double(), (n[:, None] + 3) * U * (mag + was.double().abs()), f"flags {flags}")


def test_embed_past_32_bits_and_without_tokens():
    V, d = (1 << 19) + 7, 4104   # 2^31 elements are behind row 523,287
    assert V * d > 1 << 31
    W = torch.zeros(V, d, dtype=BF, device="cuda")
    ids = torch.tensor([V - 1, 5, V - 2, 523288, V - 1], dtype=torch.int32)
    v = rand(5, d, seed=1, dtype=BF)
    W[ids.long()[[4, 1, 2, 3]].cuda()] = v[1:].cuda()[[3, 0, 1, 2]]
    out = Out(5, d, dtype=BF)
    brx.embed(W, 0, V, d, ids.cuda(), 5, 1.0, out.t, 0)
    assert torch.equal(out.guarded().cpu(), torch.stack([v[4], v[1], v[2], v[3], v[4]]))
    nb = brx.embed_backward_workspace_bytes(5, V, d)
    W.fill_(3.0)
    brx.embed_backward(v.cuda(), 0, ids.cuda(), 5, V, d, 1.0, W, 0, ws_of(nb), nb)
    assert torch.equal(W[V - 2].cpu(), v[2]) and torch.equal(W[523288].cpu(), v[3]) and torch.equal(W[5].cpu(), v[1])
    O.check(W[V - 1].cpu(), v[0].double() + v[4].double(), U * 2 * (v[0].double().abs() + v[4].double().abs()), "row")
    W[ids.long().cuda()] = 0
    assert int(torch.count_nonzero(W)) == 0
    W[:9] = 2.0
    brx.embed_backward(None, 0, None, 0, 9, d, 1.0, W[:9], 0, None, 0)
    assert not W[:9].any()
    W[:9] = 2.0
    brx.embed_backward(None, 0, None, 0, 9, d, 1.0, W[:9], 0, None, 0, flags=brx.ACCUMULATE)
    assert bool((W[:9] == 2.0).all())


# ------------------------------------------------------- vocabulary loss

VOCAB = [(1, 1, 8), (1, 300, 64), (3, 1000, 136), (5, 5003, 2048), (31, 129, 72), (32, 4096, 264), (33, 77, 8),
         (100, 1025, 1032), (130, 257, 520), (300, 5000, 264), (512, 255, 64), (513, 256, 64), (700, 1500, 328),
         (1100, 3001, 136)]


def vocab_case(T, V, d, ignore, seed=1, spread=3.0):
    g = gen(seed + T + V)
    h, W = rand(T, d, seed=seed, dtype=BF), rand(V, d, seed=seed + 1, dtype=BF, scale=spread * d ** -0.5)
    t = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    bad = torch.tensor([-1, V, -100, 2**31 - 1, -2**31], dtype=torch.int32)[torch.randint(0, 5, (T,), generator=g)]
    t = torch.where(torch.rand(T, generator=g) < ignore, bad, t)
    none = (t < 0) | (t >= V)
    h[none] = NAN   # rows without a target hold anything
    up, un = rand(T, seed=seed + 2), 0.1 * rand(T, seed=seed + 3)
    up[none], un[none] = NAN, INF
    return [v.cuda() for v in (h, W, t, up, un)], ~none.cuda()


def run_vocab(h, W, t, T, V, d):
    loss, lse = Out(T, dtype=F32), Out(T, dtype=F32)
    nb = brx.vocab_loss_workspace_bytes(T, V, d)
    brx.vocab_loss(h, W, t, T, V, d, loss.t, lse.t, ws_of(nb), nb)
    return loss.guarded(), lse.guarded()


def check_vocab(T, V, d, ignore, types, what="", spread=3.0):
    (h, W, t, up, un), ok = vocab_case(T, V, d, ignore, spread=spread)
    loss, lse = run_vocab(h, W, t, T, V, d)
    hd, Wd = h.double(), W.double()
    rl, rs, _ = R.vocab(hd, Wd, t)
    bl, bs = torch.zeros_like(rl), torch.zeros_like(rl)
    if bool(ok.any()):
        bl[ok], bs[ok] = R.vocab_bounds(hd[ok], Wd, t[ok])
    check(lse, rs, bs, "lse")
    check(loss, rl, bl, "loss")
    nb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
    for ht, wt, dlse, add in types:
        print(f"  gradient {ht} {wt} add={add}", flush=True)
        dh, dW = Out(T, d, dtype=ht), Out(V, d, dtype=wt)
        base = rand(V, d, seed=8, dtype=wt).cuda() if add else None
        if add:
            dW.t.copy_(base)
        brx.vocab_loss_backward(h, W, t, T, V, d, lse, up, ws_of(nb), nb, dlse=un if dlse else None, dh=dh.t, dhdtype=CODE[ht],
                                dW=dW.t, dwdtype=CODE[wt], flags=brx.ACCUMULATE if add else 0)
        piece = tuple(2.0 ** -8 if x is BF else 2.0 ** -16 for x in (ht, wt))
        rh, bh, rw, bw = R.vocab_grads(hd, Wd, t, lse.double(), up.double(), un.double() if dlse else None, piece)
        got = dh.guarded()
        assert not got[~ok].any(), "rows without a target"
        check(got, rh, bh, "dh")
        if add:
            rw, bw = rw + base.double(), bw + 2 * U * (rw.abs() + base.double().abs())
        got = dW.guarded()
        check(got, rw, bw, "dW")
        # independent roundings add in squares: in 2-norm no more than the types' half steps
        for g, r, x in ((dh.t, rh, ht), (dW.t, rw, wt)):
            if float(r.norm()) > 0:
                off = float((g.double() - r).norm() / r.norm())
                assert off <= (2 * 2.0 ** -8 if x is BF else 2.0 ** -15), off


@pytest.mark.parametrize("ignore", [0.0, 0.4])
@pytest.mark.parametrize("T,V,d", VOCAB)
def test_vocab_loss(T, V, d, ignore):
    print(f"case vocab T={T} V={V} d={d} ignore={ignore}", flush=True)
    check_vocab(T, V, d, ignore, [(BF, BF, True, False), (F32, F32, False, False), (BF, F32, True, True),
                                  (F32, BF, False, True)])


@pytest.mark.parametrize("T,V,d,ignore", [(8200, 8500, 64, 0.3), (33000, 2500, 16, 0.5), (4100, 17000, 72, 0.1),
                                          (20, 70000, 40, 0.2)])
def test_vocab_loss_in_pieces(T, V, d, ignore):
    """More columns than a piece holds, the last piece ragged and with spans of no columns."""
    print(f"case vocab pieces T={T} V={V} d={d}", flush=True)
    check_vocab(T, V, d, ignore, [(BF, BF, True, False), (F32, F32, True, True)])


@pytest.mark.parametrize("n", range(1, 12))
def test_vocab_contractions_of_every_length(n):
    """The buffered contractions' start, turns and end in each tile: hidden sizes and token counts of 1 to 11 steps."""
    for T, V in ((20, 300), (200, 300), (600, 300)):
        for d in (64 * n - 8, 64 * n):
            print(f"case vocab T={T} V={V} d={d}", flush=True)
            check_vocab(T, V, d, 0.0, [(BF, BF, False, False), (F32, F32, False, False)])
    for T in (32 * n - 3, 32 * n, 64 * n):
        check_vocab(T, 4000, 72, 0.0, [(BF, F32, False, False)])


def test_vocab_loss_without_targets_and_without_tokens():
    T, V, d = 40, 500, 64
    (h, W, _, up, un), _ = vocab_case(T, V, d, 0.0)
    t = torch.full((T,), -1, dtype=torch.int32).cuda()
    loss, lse = run_vocab(torch.full_like(h, NAN), W, t, T, V, d)
    assert not loss.any() and not lse.any()
    nb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
    dh, dW = Out(T, d, dtype=BF), Out(V, d, dtype=F32)
    brx.vocab_loss_backward(torch.full_like(h, NAN), W, t, T, V, d, lse, up, ws_of(nb), nb, dlse=un, dh=dh.t, dW=dW.t, dwdtype=1)
    assert not dh.guarded().any() and not dW.guarded().any()
    dW = Out(V, d, dtype=F32)
    brx.vocab_loss_backward(None, None, None, 0, V, d, None, None, None, 0, dW=dW.t, dwdtype=1)
    assert not dW.guarded().any()
    kept = Out(V, d, dtype=F32)
    brx.vocab_loss_backward(None, None, None, 0, V, d, None, None, None, 0, dW=kept.t, dwdtype=1, flags=brx.ACCUMULATE)
    assert bool((kept.guarded() == 7.0).all())


def test_vocab_gradients_apart():
    """Either gradient alone has the bits of both together."""
    for T, V, d in ((20, 300, 72), (200, 900, 136)):
        (h, W, t, up, un), _ = vocab_case(T, V, d, 0.2)
        _, lse = run_vocab(h, W, t, T, V, d)
        nb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
        args = (h, W, t, T, V, d, lse, up)
        for ht, wt in ((BF, BF), (F32, F32)):
            both = torch.empty(T, d, dtype=ht, device="cuda"), torch.empty(V, d, dtype=wt, device="cuda")
            brx.vocab_loss_backward(*args, ws_of(nb), nb, dlse=un, dh=both[0], dhdtype=CODE[ht], dW=both[1], dwdtype=CODE[wt])
            dh, dW = torch.zeros_like(both[0]), torch.zeros_like(both[1])
            brx.vocab_loss_backward(*args, ws_of(nb), nb, dlse=un, dh=dh, dhdtype=CODE[ht])
            brx.vocab_loss_backward(*args, ws_of(nb), nb, dlse=un, dW=dW, dwdtype=CODE[wt])
            assert same((dh, dW), both)


@pytest.mark.parametrize("weighted", [False, True])
def test_vocab_gradients_of_a_mean_have_no_bias(weighted):
    """dloss = 1 / 510 in every row (1 + 2^-8 of a power of two: half a step of bf16): rounded as such, the targets'
    entries of dz, and with them both gradients, would be 2^-8 off along themselves.  As multiples of it they are 1 less
    a probability of about 2^-12, rounded at most to 1; the output's rounding averages over T d = 65280 values and V d."""
    T, V, d = 510, 4096, 128
    h, W = rand(T, d, seed=1, dtype=BF).cuda(), rand(V, d, seed=2, dtype=BF, scale=0.01).cuda()
    t = torch.randint(0, V, (T,), generator=gen(3), dtype=torch.int32).cuda()
    dloss = torch.full((T,), 1 / 510, device="cuda")
    if weighted:
        dloss[:300] = 0          # rows without weight ahead of it
    _, lse = run_vocab(h, W, t, T, V, d)
    dh, dW = torch.full((T, d), 7.0, dtype=BF, device="cuda"), torch.full((V, d), 7.0, dtype=BF, device="cuda")
    nb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
    brx.vocab_loss_backward(h, W, t, T, V, d, lse, dloss, ws_of(nb), nb, dh=dh, dW=dW)
    p = torch.softmax(h.double() @ W.double().t(), 1)
    p[torch.arange(T), t.long()] -= 1
    dz = p * dloss.double()[:, None]
    for got, ref in ((dh, dz @ W.double()), (dW, dz.t().contiguous() @ h.double())):
        along = float(((got.double() - ref) * ref).sum() / ref.square().sum())
        assert abs(along) <= 2.0 ** -10, along


def test_vocab_loss_of_sharp_and_far_logits():
    """Logits of hundreds: the maximum is taken out, the loss of a certain token is small or exact."""
    for T in (9, 200, 600):
        check_vocab(T, 700, 128, 0.1, [(F32, F32, True, False)], spread=150.0)
    T, V, d = 3, 400, 64
    h = torch.zeros(T, d, dtype=BF)
    W = torch.zeros(V, d, dtype=BF)
    h[:, 0], W[17, 0] = 1000.0, 1000.0   # one logit of a million, the others 0
    t = torch.tensor([17, 17, 3], dtype=torch.int32).cuda()
    loss, lse = run_vocab(h.cuda(), W.cuda(), t, T, V, d)
    z = float(h[0, 0]) * float(W[17, 0])
    assert loss.tolist() == [0.0, 0.0, z] and lse.tolist() == [z] * 3


def test_vocab_nan_stays_in_its_row():
    T, V, d = 50, 600, 72
    (h, W, t, up, un), _ = vocab_case(T, V, d, 0.0)
    h[7, 3] = NAN
    loss, lse = run_vocab(h, W, t, T, V, d)
    ok = torch.arange(T) != 7
    assert bool(loss.cpu()[ok].isfinite().all()) and bool(loss[7].isnan()) and bool(lse[7].isnan())
    nb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
    dh = Out(T, d, dtype=F32)
    brx.vocab_loss_backward(h, W, t, T, V, d, lse, up, ws_of(nb), nb, dlse=un, dh=dh.t, dhdtype=1)
    assert bool(dh.guarded().cpu()[ok].isfinite().all()) and bool(dh.t[7].isnan().any())


# ------------------------------------------------------ orthogonalisation

COEF = (3.4445, -4.7750, 2.0315)
ORTH = [(1, 1, 1), (2, 1, 9), (1, 9, 1), (3, 8, 8), (2, 17, 40), (2, 63, 65), (1, 64, 130), (2, 130, 64), (3, 100, 300),
        (2, 300, 100), (1, 257, 513), (1, 520, 264), (2, 136, 1000), (40, 33, 70), (1, 129, 127),
        # a matrix to a block: its longest and their neighbours
        (2, 32, 1792), (1, 1791, 31), (2, 31, 257), (1, 32, 1793), (2, 64, 1024), (1, 1023, 61), (1, 33, 513), (1, 65, 1024),
        (2, 128, 384), (1, 383, 97), (1, 128, 385), (3, 128, 256), (2, 64, 512), (1, 7, 300)]


def size_of(N, K):
    return float(torch.exp2(torch.round(torch.log2(torch.tensor(float(max(N, K)))) / 2)))


def run_orth(G, steps, c, scale, eps):
    n, N, K = G.shape
    out = Out(n, N, K, dtype=BF)
    nb = brx.orthogonalise_workspace_bytes(n, N, K)
    brx.orthogonalise(G, CODE[G.dtype], n, N, K, out.t, ws_of(nb), nb, steps=steps, coefficients=c, scale=scale, eps=eps)
    return out.guarded()


def orth_case(n, N, K, dt, seed=1, scale=1e-3):
    g = rand(n, N, K, seed=seed, scale=scale)
    r = max(1, min(N, K) // 8)
    return (g + torch.bmm(rand(n, N, r, seed=seed + 1), rand(n, r, K, seed=seed + 2, scale=scale))).to(dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,N,K", ORTH)
def test_orthogonalise(n, N, K, dt):
    """One step elementwise, five in Frobenius norm, no step: G / (|G| + eps)."""
    print(f"case orth n={n} N={N} K={K} {dt}", flush=True)
    G = orth_case(n, N, K, dt)
    c, eps, scale = tuple(f32(v) for v in COEF), f32(1e-7), 1.25
    Gd, size = G.double(), size_of(N, K)
    got = run_orth(G.cuda(), 0, COEF, scale, 1e-7)
    ref = R.orthogonalise(Gd, 0, c, scale, eps)
    check(got, ref, 4 * U * ref.abs(), "no step")
    got = run_orth(G.cuda(), 1, COEF, scale, 1e-7)
    check(got, R.orthogonalise(Gd, 1, c, scale, eps), R.orth_one_step_bound(Gd, c, scale, eps, size), "one step")
    got = run_orth(G.cuda(), 5, COEF, 1.0, 1e-7)
    ref = R.orthogonalise(Gd, 5, c, 1.0, eps)
    bound = R.orth_norm_bound(Gd, 5, c, eps, size) + 2.0 ** -8 * ref.flatten(1).norm(dim=1)
    off = (got.cpu().double() - ref).flatten(1).norm(dim=1)
    print(f"  five steps off {float((off / ref.flatten(1).norm(dim=1)).max()):.2e}, bound "
          f"{float((bound / ref.flatten(1).norm(dim=1)).max()):.2e}", flush=True)
    assert bool((off <= bound).all())


@pytest.mark.parametrize("n,N,K", [(200, 60, 72), (200, 72, 60), (70, 200, 264), (70, 264, 200), (70, 500, 520), (66, 520, 500),
                                   (16, 1030, 520), (16, 520, 1030), (8, 1100, 1290), (8, 1290, 1100), (20, 1000, 1010), (20, 1010, 1000)])
def test_orthogonalise_every_tile(n, N, K):
    """Enough matrices for the larger tiles: one step elementwise, in 64 bits on the GPU."""
    print(f"case orth tiles n={n} N={N} K={K}", flush=True)
    G = orth_case(n, N, K, F32, seed=4).cuda()
    c = tuple(f32(v) for v in COEF)
    first = None
    for _ in range(2):
        got = run_orth(G, 1, COEF, 1.0, 1e-7)
        first = got.clone() if first is None else first
        assert torch.equal(got, first)
    for e in range(0, n, max(1, n // 8)):
        g = G[e:e + 1].double()
        check(got[e:e + 1], R.orthogonalise(g, 1, c, 1.0, f32(1e-7)), R.orth_one_step_bound(g, c, 1.0, f32(1e-7), size_of(N, K)),
              f"matrix {e}")


def test_orthogonalise_makes_rows_orthonormal():
    """Singular values of the result lie where the polynomial takes them, and a gradient of few rows keeps its rank."""
    n, N, K = 2, 192, 320
    G = torch.bmm(rand(n, N, 20, seed=1), rand(n, 20, K, seed=2)).cuda()
    got = run_orth(G, 5, COEF, 1.0, 1e-7).double().cpu()
    s = torch.linalg.svdvals(got)
    assert bool((s[:, :20] > 0.6).all()) and bool((s[:, :20] < 1.3).all())
    # what G lacks: bf16 rounding of the result (a matrix with singular values up to 2^-9 (sqrt(N) + sqrt(K)) / sqrt(3)
    # times the rms of a value) and the products' own error
    rms = float(got.square().mean().sqrt())
    assert float(s[:, 20:].max()) <= 2 * 2.0 ** -9 * (N ** 0.5 + K ** 0.5) * rms + float(
        R.orth_norm_bound(G.cpu().double(), 5, COEF, 1e-7, size_of(N, K)).max())


def test_orthogonalise_zeros_infinities_and_scales():
    n, N, K = 5, 72, 136
    G = rand(n, N, K, seed=3)
    G[1] = 0
    G[2, 5, 7] = INF
    G[3, 0, 0] = NAN
    got = run_orth(G.cuda(), 5, COEF, 1.0, 1e-7).cpu()
    assert bool(got[[0, 4]].isfinite().all()) and not got[1].any() and not got[2].isfinite().all() and not got[3].isfinite().all()
    want = run_orth(G[[0, 4]].cuda(), 5, COEF, 1.0, 1e-7).cpu()
    assert torch.equal(got[[0, 4]], want)
    # G and eps times a power of two: G / (|G| + eps) is the same number, also where squares leave fp32's range
    # (an eps that is not scaled alike shows: 1e-30 beside a norm of 8e-23 is 1e-8, enough to round the quotient elsewhere)
    want = run_orth(G[[0, 4]].cuda(), 5, COEF, 1.0, 2.0 ** -24)
    for s in (2.0 ** 80, 2.0 ** -80):
        assert torch.equal(run_orth((G[[0, 4]] * s).cuda(), 5, COEF, 1.0, 2.0 ** -24 * s), want)


@pytest.mark.parametrize("c", [(1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (1.5, -0.5, 0.0), (2.0, -1.5, 1e-30), (0.0, 0.0, 0.0),
                               (2.0, -1.2, 0.2)])
@pytest.mark.parametrize("n,N,K", [(2, 60, 72), (3, 200, 300), (3, 300, 200), (70, 256, 264)])
def test_orthogonalise_other_polynomials(n, N, K, c):
    """Terms apart, coefficients of zero: one step elementwise, three in Frobenius norm."""
    G = orth_case(n, N, K, F32, seed=5)
    c = tuple(f32(v) for v in c)
    got = run_orth(G.cuda(), 1, c, 1.0, 1e-7)
    g = G[:3].double()
    check(got[:3], R.orthogonalise(g, 1, c, 1.0, f32(1e-7)), R.orth_one_step_bound(g, c, 1.0, f32(1e-7), size_of(N, K)), "one step")
    got = run_orth(G.cuda(), 3, c, 1.0, 1e-7)[:3]
    ref = R.orthogonalise(g, 3, c, 1.0, f32(1e-7))
    bound = R.orth_norm_bound(g, 3, c, f32(1e-7), size_of(N, K)) + 2.0 ** -8 * ref.flatten(1).norm(dim=1)
    assert bool(((got.cpu().double() - ref).flatten(1).norm(dim=1) <= bound).all())


def test_orthogonalise_in_place():
    for n, N, K in ((3, 72, 136), (2, 130, 61)):
        G = orth_case(n, N, K, BF).cuda()
        for steps in (0, 1, 5):
            want = run_orth(G, steps, COEF, 1.0, 1e-7)
            own = G.clone()
            nb = brx.orthogonalise_workspace_bytes(n, N, K)
            brx.orthogonalise(own, 0, n, N, K, own, ws_of(nb), nb, steps=steps)
            assert torch.equal(own, want)


@pytest.mark.parametrize("n,N,K", [(3, 4, 300), (2, 7, 1225), (3, 18, 556), (3, 22, 556), (2, 33, 90), (3, 48, 256), (2, 200, 64),
                                   (2, 73, 274), (2, 100, 200), (2, 127, 256)])
def test_orthogonalise_of_equal_singular_values(n, N, K):
    """All diagonals of X X^T are the same number, whose rounding to 11 bits would not average out: after 5 steps up to
    7e-3 of the result, along itself.  In fp32 what is left averages over the values of a row: X's 11 bits in X X^T are
    2^-11 / sqrt(3) of each of K / 2 products or more off, 5e-5 together for K = 64, and a step makes at most
    (|b| + 2 |c|) 2 = 18 times that of a result of 0.7 or more if it keeps it.  The output's rounding, at most 2^-8,
    averages over N K values, 1200 or more.  2^-10 lies between."""
    print(f"case orth equal n={n} N={N} K={K}", flush=True)
    side, long = min(N, K), max(N, K)
    q = torch.linalg.qr(rand(n, long, side, seed=6).double()).Q * 3
    G = (q if N > K else q.transpose(1, 2)).float().contiguous()
    got = run_orth(G.cuda(), 5, COEF, 1.0, 1e-7).cpu().double()
    ref = R.orthogonalise(G.double(), 5, tuple(f32(v) for v in COEF), 1.0, f32(1e-7))
    along = ((got - ref) * ref).sum((1, 2)) / ref.square().sum((1, 2))
    assert float(along.abs().max()) <= 2.0 ** -10, along


@pytest.mark.parametrize("n,N,K", [(2, 130, 300), (2, 301, 131), (2, 200, 1800), (1, 512, 1024), (3, 1040, 520), (16, 264, 530),
                                   (14, 768, 1024), (14, 1024, 765), (28, 520, 1100), (28, 1100, 520)])
def test_orthogonalise_of_equal_singular_values_in_tiles(n, N, K):
    """As above where a matrix is cut into tiles, each of the steps' and of the squares' tiles."""
    print(f"case orth equal n={n} N={N} K={K}", flush=True)
    side, long = min(N, K), max(N, K)
    q = torch.linalg.qr(rand(1, long, side, seed=6).double()).Q * 3
    g = (q if N > K else q.transpose(1, 2)).float().contiguous()
    got = run_orth(g.expand(n, N, K).contiguous().cuda(), 5, COEF, 1.0, 1e-7)
    assert bool((got == got[:1]).all())
    ref = R.orthogonalise(g.cuda().double(), 5, tuple(f32(v) for v in COEF), 1.0, f32(1e-7))
    along = ((got[:1].double() - ref) * ref).sum() / ref.square().sum()
    assert abs(float(along)) <= 2.0 ** -10, along


# --------------------------------------------- graphs, streams, repetition

def every_call(seed):
    """One call of each entry point on small inputs: (name, run, inputs to overwrite, outputs)."""
    calls = []
    e = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    for name, T in (("balance", 40), ("balance_large", 700)):
        k, E = 4, 72
        z, idx = rand(T, E, seed=seed).cuda(), draw_idx(T, k, E, 0.1, seed).cuda()
        losses, counts, prob, lse, tokens = e(2), e(E, dt=i32), e(E), e(T), e(1, dt=i32)
        nb = brx.balance_loss_workspace_bytes(T, k, E)
        ws = ws_of(nb)
        calls.append((name, lambda z=z, idx=idx, T=T, o=(losses, counts, lse, tokens), ws=ws, nb=nb, prob=prob:
                      brx.balance_loss(z, 1, idx, T, 4, 72, *o, ws, nb, prob=prob), [z, idx], [losses, counts, prob, lse, tokens]))
    T, k, E = 300, 4, 72
    z, idx, dp = rand(T, E, seed=seed + 1).cuda(), draw_idx(T, k, E, 0.1, seed + 1).cuda(), rand(T, k, seed=seed + 2).cuda()
    lse = torch.logsumexp(z, 1)
    counts, tokens, dl, dz = torch.arange(E, dtype=i32, device="cuda"), e(1, dt=i32).fill_(T), rand(2, seed=seed).cuda(), e(T, E)
    calls.append(("balance_backward", lambda z=z, idx=idx, T=T, lse=lse, counts=counts, tokens=tokens:
                  brx.balance_loss_backward(z, 1, idx, T, k, E, lse, counts, tokens, dl, dz, dpicks=dp),
                  [z, idx, dp, dl], [dz]))
    T, V, d = 500, 3000, 72
    W, ids, out = rand(V, d, seed=seed, dtype=BF).cuda(), draw_ids(T, V, seed).cuda(), e(T, d)
    calls.append(("embed", lambda W=W, V=V, d=d, T=T, out=out: brx.embed(W, 0, V, d, ids, T, 2.0, out, 1), [W, ids], [out]))
    dout, dW = rand(T, d, seed=seed + 3).cuda(), e(V, d, dt=BF)
    eb = brx.embed_backward_workspace_bytes(T, V, d)
    ews = ws_of(eb)
    calls.append(("embed_backward", lambda V=V, d=d, T=T, dW=dW:
                  brx.embed_backward(dout, 1, ids, T, V, d, 2.0, dW, 0, ews, eb), [dout, ids], [dW]))
    T2 = 70000
    many, dmany, dW2 = draw_ids(T2, V, seed + 4).cuda(), rand(T2, 8, seed=seed + 4).cuda(), e(V, 8)
    mb = brx.embed_backward_workspace_bytes(T2, V, 8)
    mws = ws_of(mb)
    calls.append(("embed_backward_large", lambda V=V: brx.embed_backward(dmany, 1, many, T2, V, 8, 2.0, dW2, 1, mws, mb),
                  [dmany, many], [dW2]))
    for name, T, V, d in (("few", 20, 900, 72), ("more", 200, 900, 72), ("many", 600, 1100, 136), ("pieces", 9000, 7500, 16)):
        (h, W, t, up, un), _ = vocab_case(T, V, d, 0.2, seed=seed)
        loss, lse = e(T), e(T)
        nb = brx.vocab_loss_workspace_bytes(T, V, d)
        ws = ws_of(nb)
        calls.append((f"vocab_{name}", lambda h=h, W=W, t=t, s=(T, V, d), o=(loss, lse), ws=ws, nb=nb:
                      brx.vocab_loss(h, W, t, *s, *o, ws, nb), [h, W, t], [loss, lse]))
        known = e(T)
        known.fill_(8.0)
        dh, dW = e(T, d, dt=BF), e(V, d)
        bb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
        bws = ws_of(bb)
        calls.append((f"vocab_backward_{name}", lambda h=h, W=W, t=t, s=(T, V, d), l=known, up=up, un=un, o=(dh, dW), ws=bws, nb=bb:
                      brx.vocab_loss_backward(h, W, t, *s, l, up, ws, nb, dlse=un, dh=o[0], dW=o[1], dwdtype=1),
                      [h, W, t, up, un], [dh, dW]))
    for n, N, K in ((3, 40, 72), (20, 200, 130)):
        G, out = orth_case(n, N, K, F32, seed=seed).cuda(), e(n, N, K, dt=BF)
        nb = brx.orthogonalise_workspace_bytes(n, N, K)
        ws = ws_of(nb)
        calls.append((f"orth_{N}", lambda G=G, s=(n, N, K), o=out, ws=ws, nb=nb: brx.orthogonalise(G, 1, *s, o, ws, nb), [G], [out]))
    return calls


COUNT = 16


def test_every_call_is_counted():
    assert len(every_call(1)) == COUNT


@pytest.mark.parametrize("which", range(COUNT))
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
            g.replay()
            assert same(bits(outs), want), "a replay differs from the eager call"
            run()   # eager work between the replays
            assert same(bits(outs), want)


@pytest.mark.parametrize("which", range(COUNT))
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


def test_two_calls_under_way_together():
    """Calls of every kind on two streams at once, workspaces of their own: the bits of calls alone."""
    a, b = every_call(11), every_call(12)
    for c in a + b:
        c[1]()
    want = [bits(c[3]) for c in a + b]
    for c in a + b:
        for o in c[3]:
            o.zero_()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for q in s:
        q.wait_stream(torch.cuda.current_stream())
    for x, y in zip(a, b):
        for q, c in zip(s, (x, y)):
            with torch.cuda.stream(q):
                c[1]()
    torch.cuda.synchronize()
    for c, w in zip(a + b, want):
        assert same(c[3], w), c[0]


# ------------------------------------------------------- offsets past 2^31

def test_balance_past_32_bits():
    T, k, E = (1 << 21) + 5, 1, 1024
    z = torch.zeros(T, E, dtype=BF, device="cuda")
    z[-1, 1000], z[-2, 3] = 5.0, -INF
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    losses, counts, prob, lse, tokens = run_balance(z, idx, None, T, k, E)
    assert int(tokens) == T and int(counts[0]) == T
    want = torch.log(torch.tensor([1023 + 2.718281828459045 ** 5, 1023.0, 1024.0], dtype=torch.float64))
    O.check(lse[[-1, -2, -3]].cpu(), want, (E + 40) * U, "lse")
    dl = torch.tensor([0.0, 1.0]).cuda()
    brx.balance_loss_backward(z, 0, idx, T, k, E, lse, counts, tokens, dl, z)
    row = torch.exp(torch.tensor([0.0, 5.0], dtype=torch.float64) - want[0]) * 2 * want[0] / T
    O.check(z[-1, [0, 1000]].cpu(), row, (2 * E + 80) * U * row, "dz")
    assert float(z[-2, 3]) == 0.0 and int(torch.count_nonzero(z[-2])) == E - 1


def test_vocab_loss_past_32_bits():
    T, V, d = 3, 1 << 20, 2056
    assert V * d > 1 << 31
    W = torch.zeros(V, d, dtype=BF, device="cuda")
    rows = torch.tensor([V - 1, V - 2, 5, (1 << 31) // d + 1])
    W[rows.cuda()] = rand(4, d, seed=1, dtype=BF, scale=0.1).cuda()
    h = rand(T, d, seed=2, dtype=BF).cuda()
    t = torch.tensor([V - 1, 77, (1 << 31) // d + 1], dtype=torch.int32).cuda()
    loss, lse = run_vocab(h, W, t, T, V, d)
    z = h.double() @ W[rows.cuda()].double().t()
    want = torch.log(z.exp().sum(1) + V - 4)
    bound = 2 * d * U * (h.double().abs() @ W[rows.cuda()].double().abs().t()).max() + (V + 64) * U
    check(lse, want, bound, "lse")
    check(loss, want - torch.stack([z[0, 0], z[1, 0] * 0, z[2, 3]]), 2 * bound, "loss")
    up = torch.ones(T, device="cuda")
    dh, dW = Out(T, d, dtype=F32), torch.full((V, d), 3.0, dtype=BF, device="cuda")
    nb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
    brx.vocab_loss_backward(h, W, t, T, V, d, lse, up, ws_of(nb), nb, dh=dh.t, dhdtype=1, dW=dW)
    p = torch.exp(z - lse.double()[:, None])
    p[0, 0] -= 1
    p[2, 3] -= 1
    ref = p @ W[rows.cuda()].double()
    check(dh.guarded(), ref, (2.0 ** -16 + 4 * bound) * (p.abs() @ W[rows.cuda()].double().abs()) + 8 * U * ref.abs(), "dh")
    ref = p.t() @ h.double()
    check(dW[rows.cuda()], ref, (2.0 ** -8 + 4 * bound) * (p.abs().t() @ h.double().abs()), "dW")
    q = torch.exp(-lse.double())[:, None]
    rest = (q * h.double()).sum(0)
    check(dW[V // 2], rest, (2.0 ** -8 + 4 * bound) * (q * h.double().abs()).sum(0), "dW of a row of zeros")


def test_orthogonalise_past_32_bits():
    n, N, K = 600, 1900, 1900
    G = torch.zeros(n, N, K, device="cuda")
    few = [0, 497, 598, 599]
    for e in few:
        G[e] = rand(N, K, seed=e).cuda()
    out = torch.full((n, N, K), 3.0, dtype=BF, device="cuda")
    nb = brx.orthogonalise_workspace_bytes(n, N, K)
    brx.orthogonalise(G, 1, n, N, K, out, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb, steps=1)
    c = tuple(f32(v) for v in COEF)
    for e in few:
        g = G[e:e + 1].double()
        check(out[e:e + 1], R.orthogonalise(g, 1, c, 1.0, f32(1e-7)), R.orth_one_step_bound(g, c, 1.0, f32(1e-7), size_of(N, K)),
              f"matrix {e}")
        out[e] = 0
    assert int(torch.count_nonzero(out)) == 0


# ------------------------------------------------------------- all together

def test_a_training_step():
    """Token rows in -> norm -> router, its balance losses and its picks ->
    sparse experts -> residual -> norm -> vocabulary loss over the same table,
    all gradients (the table's from both ends, the router's from the loss and
    from its own losses), and the experts' update orthogonalised, against
    automatic differentiation in 64 bits with the same picks.  Rows between the
    operators are bf16: each of the about twelve roundings on a path is at most
    2^-8 of its value, and independent ones add in squares, so losses and
    gradients are within 12 * 2^-8 in 2-norm."""
    T, V, d, E, k, f = 120, 500, 256, 16, 4, 128
    sh = brx.shape(E, k, d, f, 3)
    table = rand(V, d, seed=1, dtype=BF, scale=0.1)
    Wr, g0, g1 = rand(E, d, seed=2, scale=d ** -0.5), 1 + 0.1 * rand(d, seed=3), 1 + 0.1 * rand(d, seed=4)
    W1, W2 = rand(E, 2 * f, d, seed=6, dtype=BF, scale=d ** -0.5), rand(E, d, f, seed=7, dtype=BF, scale=f ** -0.5)
    ids, targets = draw_ids(T, V, 8, pad=0.0), draw_ids(T, V, 9, pad=0.25)
    n, has = T * k, (targets >= 0) & (targets < V)
    m = int(has.sum())
    c_balance, c_z, c_lse, scale = 0.05, 0.01, 0.002, 10.0
    TB, WR, G0, G1, W1c, W2c, I, TG = (v.cuda() for v in (table, Wr, g0, g1, W1, W2, ids, targets))
    e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    # forward
    x = e(T, d)
    brx.embed(TB, 0, V, d, I, T, scale, x, 1)
    a0 = brx.block_norm_args(T, d, 1, 0, 0, brx.PRE_NORM)
    u, r0 = e(T, d, dt=BF), e(T)
    brx.block_norm(a0, x, None, g_pre=G0, u=u, rstd_r=r0)
    nb = brx.workspace_bytes(sh, T)
    ro = dict(topk_idx=e(T, k, dt=torch.int32), topk_w=e(T, k))
    brx.route(sh, brx.LayerData(router_w=WR, codes=None, scales=None), u, brx.X_BF16, T, ro, ws_of(nb), nb)
    z = u.float() @ WR.t()
    losses, counts, lse_r, tokens = e(2), e(E, dt=torch.int32), e(T), e(1, dt=torch.int32)
    bb = brx.balance_loss_workspace_bytes(T, k, E)
    brx.balance_loss(z, 1, ro["topk_idx"], T, k, E, losses, counts, lse_r, tokens, ws_of(bb), bb)
    off, pos = e(E + 1, dt=torch.int32), e(n, dt=torch.int32)
    sb = brx.sort_workspace_bytes(T, k, E)
    brx.sort_picks(ro["topk_idx"], T, k, E, None, off, None, pos, ws_of(sb), sb)
    xs, gu, ys = e(n, d, dt=BF), e(n, 2 * f, dt=BF), e(n, d, dt=BF)
    brx.dispatch(u, 0, T, k, d, pos, xs, n)
    gb = max(brx.grouped_workspace_bytes(n, E, 2 * f, d), brx.grouped_workspace_bytes(n, E, d, f))
    gws = ws_of(gb)
    brx.grouped_product(xs, W1c, off, n, E, 2 * f, d, gu, 0, gws, gb)
    gl, ul = gu.float()[:, :f], gu.float()[:, f:]
    hh = (gl * torch.sigmoid(gl) * ul).to(BF)
    brx.grouped_product(hh, W2c, off, n, E, d, f, ys, 0, gws, gb)
    y = e(T, d, dt=BF)
    brx.combine(ys, 0, n, pos, ro["topk_w"], T, k, d, y, 0)
    a1 = brx.block_norm_args(T, d, 1, 0, 0, brx.PRE_NORM)
    r, h, sr = e(T, d), e(T, d, dt=BF), e(T)
    brx.block_norm(a1, x, y, g_pre=G1, r=r, u=h, rstd_r=sr)
    loss, lse = e(T), e(T)
    vb = brx.vocab_loss_workspace_bytes(T, V, d)
    brx.vocab_loss(h, TB, TG, T, V, d, loss, lse, ws_of(vb), vb)
    # backward of mean loss + c_lse mean lse^2 + c_balance balance + c_z z loss
    up, un = torch.full((T,), 1.0 / m, device="cuda"), 2 * c_lse / m * lse
    dh, dT = e(T, d, dt=BF), e(V, d)
    vb = brx.vocab_loss_backward_workspace_bytes(T, V, d)
    brx.vocab_loss_backward(h, TB, TG, T, V, d, lse, up, ws_of(vb), vb, dlse=un, dh=dh, dW=dT, dwdtype=1)
    dX, dy, dg1 = e(T, d), e(T, d, dt=BF), e(d)
    wb = brx.block_norm_backward_workspace_bytes(a1)
    brx.block_norm_backward(a1, None, dh, r, y, g_pre=G1, rstd_r=sr, dx=dX, dy=dy, dg_pre=dg1, ws=ws_of(wb), ws_bytes=wb)
    dys, dpk = e(n, d, dt=BF), e(T, k)
    brx.combine_backward(dy, 0, ys, 0, n, pos, ro["topk_w"], T, k, d, dys=dys, dz=dpk)
    dhh, dxs, dW1, dW2 = e(n, f), e(n, d, dt=BF), e(E, 2 * f, d), e(E, d, f)
    brx.grouped_dgrad(dys, W2c, off, n, E, d, f, dhh, 1, gws, gb)
    brx.grouped_wgrad(dys, hh, off, n, E, d, f, dW2, 1, gws, gb)
    sg = torch.sigmoid(gl)
    dgu = torch.cat([dhh * ul * sg * (1 + gl * (1 - sg)), dhh * gl * sg], 1).to(BF)
    brx.grouped_dgrad(dgu, W1c, off, n, E, 2 * f, d, dxs, 0, gws, gb)
    brx.grouped_wgrad(dgu, xs, off, n, E, 2 * f, d, dW1, 1, gws, gb)
    du = e(T, d, dt=BF)
    brx.dispatch_backward(dxs, 0, n, pos, T, k, d, du)
    dz = e(T, E)
    brx.balance_loss_backward(z, 1, ro["topk_idx"], T, k, E, lse_r, counts, tokens, torch.tensor([c_balance, c_z], device="cuda"),
                              dz, dpicks=dpk)
    dWr = dz.t().contiguous() @ u.float()
    du_all = (du.float() + dz @ WR).to(BF)
    dXn, dg0 = e(T, d), e(d)
    wb0 = brx.block_norm_backward_workspace_bytes(a0)
    brx.block_norm_backward(a0, dX, du_all, x, None, g_pre=G0, rstd_r=r0, dx=dXn, dg_pre=dg0, ws=ws_of(wb0), ws_bytes=wb0)
    eb = brx.embed_backward_workspace_bytes(T, V, d)
    brx.embed_backward(dXn, 1, I, T, V, d, scale, dT, 1, ws_of(eb), eb, flags=brx.ACCUMULATE)
    ob = brx.orthogonalise_workspace_bytes(E, 2 * f, d)
    step = e(E, 2 * f, d, dt=BF)
    brx.orthogonalise(dW1, 1, E, 2 * f, d, step, ws_of(ob), ob)
    torch.cuda.synchronize()
    # the same in 64 bits
    L = {q: v.double().clone().requires_grad_(True) for q, v in dict(table=table, Wr=Wr, g0=g0, g1=g1, W1=W1, W2=W2).items()}
    idx = ro["topk_idx"].cpu().long()
    eps = f32(1e-6)
    xd = L["table"][ids.long()] * scale
    ud = O.norm_rows(xd, L["g0"], eps)
    zd = ud @ L["Wr"].t()
    bal, _, _, _, _ = R.balance(zd, idx, None, E)
    wd = torch.softmax(zd.gather(1, idx), 1)
    yd = torch.zeros(T, d, dtype=torch.float64)
    for q in range(k):
        guv = torch.bmm(L["W1"][idx[:, q]], ud[:, :, None])[:, :, 0]
        hv = torch.nn.functional.silu(guv[:, :f]) * guv[:, f:]
        yd = yd + wd[:, q:q + 1] * torch.bmm(L["W2"][idx[:, q]], hv[:, :, None])[:, :, 0]
    hd = O.norm_rows(xd + yd, L["g1"], eps)
    ld, sd, _ = R.vocab(hd, L["table"], targets)
    total = ld.sum() / m + c_lse * sd.square().sum() / m + c_balance * bal[0] + c_z * bal[1]
    names = ("table", "Wr", "g0", "g1", "W1", "W2")
    grads = dict(zip(names, torch.autograd.grad(total, [L[q] for q in names])))
    for q, got, ref in (("loss", loss, ld), ("lse", lse, sd), ("balance", losses, bal), ("table", dT, grads["table"]),
                        ("Wr", dWr, grads["Wr"]), ("g0", dg0, grads["g0"]), ("g1", dg1, grads["g1"]), ("W1", dW1, grads["W1"]),
                        ("W2", dW2, grads["W2"])):
        ref = ref.detach()
        off_by = float((got.cpu().double() - ref).norm() / ref.norm())
        print(f"  {q}: {off_by:.2e}", flush=True)
        assert off_by <= 12 * 2.0 ** -8, f"{q}: off by {off_by:.3e} in 2-norm"
    G, c = dW1.cpu().double(), tuple(f32(v) for v in COEF)
    ref = R.orthogonalise(G, 5, c, 1.0, f32(1e-7))
    bound = R.orth_norm_bound(G, 5, c, f32(1e-7), size_of(2 * f, d)) + 2.0 ** -8 * ref.flatten(1).norm(dim=1)
    assert bool(((step.cpu().double() - ref).flatten(1).norm(dim=1) <= bound).all())
