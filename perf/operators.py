"""Operators around the sparse layer: what is measured, in which sizes.

Four kinds of work, each as a user's program calls it:

- dispatch: picks sorted by expert and the token rows copied to their slots; its gradient.
- combine: the experts' rows weighted and summed back per token; its gradient.
- product: every expert's dense matrix times its sorted rows; both gradients.
- norm: norms after and before a block with the branch's gate and the residual scale; its gradient.

``own`` selects between the plain form (elementary torch operations in 32
bits) and the library's kernels.
"""
import math

import torch

own = False


def _lib():
    import bit_routed_expert_amd as brx
    return brx


EPS = 1e-6
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CODE = {"bf16": 0, "f32": 1}   # STRATA_X_BF16, STRATA_X_F32
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a verify step's five tokens, routed over the full-size layer: launch latency
        dict(name="dispatch_verify", kind="dispatch", T=5, k=10, E=512, d=2048, x="bf16", drop=0.0),
        # a 4096-token prompt chunk of the full-size layer
        dict(name="dispatch_prompt", kind="dispatch", T=4096, k=10, E=512, d=2048, x="bf16", drop=0.0),
        # gradient of the copy: a ragged training batch, fp32 rows, an eighth of the picks over capacity
        dict(name="dispatch_back", kind="dispatch_back", T=4093, k=4, E=64, d=1000, x="f32", drop=0.125),
        # one decoded token: the ten experts' rows onto the shared expert's, fp32 residual stream
        dict(name="combine_decode", kind="combine", T=1, k=10, E=512, d=2048, y="f32", out="f32", base=True, drop=0.0),
        # a prompt chunk; the picks whose expert is not resident are left out
        dict(name="combine_prompt", kind="combine", T=4096, k=10, E=512, d=2048, y="bf16", out="bf16", base=True, drop=0.15),
        # a training batch: gradients of the rows, of the gates and of the picked logits
        dict(name="combine_back", kind="combine_back", T=4096, k=10, E=512, d=2048, y="bf16", out="bf16", drop=0.0),
        # gate and up rows of a verify step's picks: weights read once, one or two rows to an expert
        dict(name="product_verify", kind="product", T=5, k=10, E=512, N=1536, K=2048, y="bf16", drop=0.0),
        # gate and up rows of a prompt chunk: about 80 rows to an expert, unevenly
        dict(name="product_prompt", kind="product", T=4096, k=10, E=512, N=1536, K=2048, y="bf16", drop=0.0),
        # both gradients of a small layer's experts (16 of them) over a long training batch
        dict(name="product_back", kind="product_back", T=16384, k=2, E=16, N=1536, K=2048, y="bf16", dw="f32", drop=0.02),
        # one decoded token: the block's output normed, gated and added, then normed for the next block
        dict(name="norm_decode", kind="norm", T=1, d=2048, x="f32", y="f32", u="bf16", post=True, pre=True, gate="token", sigmoid=True),
        # a prompt chunk with bf16 rows
        dict(name="norm_prompt", kind="norm", T=4096, d=2048, x="bf16", y="bf16", u="bf16", post=True, pre=True, gate="channel", sigmoid=False),
        # a training batch: gradients of both rows, the gate and both gains
        dict(name="norm_back", kind="norm_back", T=8191, d=2048, x="f32", y="bf16", u="bf16", post=True, pre=True, gate="channel", sigmoid=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["dispatch", "dispatch_back", "combine", "combine_back", "product", "product", "product_back",
                       "norm", "norm_back"])
    c = {"kind": kind}
    T = _logint(rng, 1, 8192)
    t = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if kind in ("norm", "norm_back"):
        d = rng.choice([128 * rng.randint(1, 32), 8 * rng.randint(8, 512), rng.randint(64, 4096)])
        gate = rng.choice(["none", "token", "channel"])
        c.update(T=T, d=d, x=t(), y=t(), u=t(), post=rng.random() < 0.75, pre=rng.random() < 0.75, gate=gate,
                 sigmoid=gate != "none" and rng.random() < 0.5)
        return c
    E = _logint(rng, 4, 512)
    k = rng.randint(1, min(E, 12))
    T = min(T, 40960 // k)
    drop = rng.choice([0.0, 0.0, 0.1, 0.5])
    c.update(T=T, k=k, E=E, drop=drop)
    if kind in ("product", "product_back"):
        N, K = 8 * _logint(rng, 8, 256), 8 * _logint(rng, 8, 256)
        c.update(N=N, K=K, y=t())
        if kind == "product_back":
            c.update(dw=t())
            while c["E"] * N * K > 16 * 1536 * 2048 * 4:   # gradients of all the experts: a training batch's sizes
                N = c["N"] = max(64, N // 16 * 8)
                K = c["K"] = max(64, K // 16 * 8)
            c["T"] = min(c["T"], max(1, 32768 // k))
        return c
    d = rng.choice([128 * rng.randint(1, 16), 8 * rng.randint(8, 256), rng.randint(64, 2048)])
    c["d"] = d
    if kind in ("dispatch", "dispatch_back"):
        c["x"] = t()
        if c["x"] == "f32":
            c["T"] = max(1, c["T"] // 2)
    else:
        c.update(y=t(), out=t())
        if c["y"] == "f32":
            c["T"] = max(1, c["T"] // 2)
        if kind == "combine":
            c["base"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs

def _rows(g, n, d, dtype, scale=1.0):
    return (torch.randn(n, d, device="cuda", generator=g) * scale).to(dtype)


def _picks(c, g):
    """Picks of a router with uneven experts: [T][k] int32 ids (-1 for a dropped pick) and their gates."""
    T, k, E = c["T"], c["k"], c["E"]
    popular = torch.randn(E, device="cuda", generator=g) * 0.7
    z = torch.randn(T, E, device="cuda", generator=g) + popular
    top = torch.topk(z, k, dim=1)
    idx = top.indices.to(torch.int32)
    if c["drop"] > 0:
        idx = torch.where(torch.rand(T, k, device="cuda", generator=g) < c["drop"], torch.full_like(idx, -1), idx)
    return idx.contiguous(), torch.softmax(top.values, dim=1).contiguous()


def _sorted(idx, E):
    """counts, offsets, perm, pos of the picks (int32), as the sort gives them."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device).scatter_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(counts, 0)
    slot = torch.arange(n, device=flat.device)
    perm = torch.where(slot < offsets[E], order, torch.full_like(order, -1))
    pos = torch.empty_like(order)
    pos[order] = slot
    pos = torch.where(kept, pos, torch.full_like(pos, -1))
    return counts.int(), offsets.int(), perm.int(), pos.int()


def _empty_int(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed + 1))
    kind = c["kind"]
    s = {"case": c}
    T = c["T"]
    if kind in ("norm", "norm_back"):
        d = c["d"]
        xt, yt, ut = _TYPES[c["x"]], _TYPES[c["y"]], _TYPES[c["u"]]
        s["x"] = _rows(g, T, d, xt, 2.0)
        s["y"] = _rows(g, T, d, yt, 0.5)
        s["g_post"] = 1.0 + 0.2 * torch.randn(d, device="cuda", generator=g) if c["post"] else None
        s["g_pre"] = 1.0 + 0.2 * torch.randn(d, device="cuda", generator=g) if c["pre"] else None
        s["gate"] = {"none": None, "token": torch.randn(T, device="cuda", generator=g),
                     "channel": _rows(g, T, d, yt)}[c["gate"]]
        s["a"], s["b"] = 0.9, 0.5
        rstd_y = torch.empty(T, device="cuda")
        rstd_r = torch.empty(T, device="cuda")
        r = torch.empty(T, d, dtype=xt, device="cuda")
        u = torch.empty(T, d, dtype=ut, device="cuda") if c["pre"] else None
        if kind == "norm":
            s.update(r=r, u=u, rstd_y=rstd_y if c["post"] else None, rstd_r=rstd_r if c["pre"] else None)
            return s
        # what the forward pass left for the gradient: the residual rows and both inverse norms
        yn = s["y"].double()
        ry = torch.rsqrt(yn.square().mean(1) + EPS)
        if c["post"]:
            yn = yn * ry[:, None] * s["g_post"].double()
        if c["gate"] != "none":
            gv = s["gate"].double()
            gv = gv[:, None] if c["gate"] == "token" else gv
            yn = yn * (torch.sigmoid(gv) if c["sigmoid"] else gv)
        s["r"] = (s["a"] * s["x"].double() + s["b"] * yn).to(xt)
        s["rstd_y"] = ry.float() if c["post"] else None
        s["rstd_r"] = torch.rsqrt(s["r"].double().square().mean(1) + EPS).float() if c["pre"] else None
        del s["x"]
        s["dr"] = _rows(g, T, d, xt)
        s["du"] = _rows(g, T, d, ut) if c["pre"] else None
        s["dx"] = torch.empty(T, d, dtype=xt, device="cuda")
        s["dy"] = torch.empty(T, d, dtype=yt, device="cuda")
        s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
        s["dg_post"] = torch.empty(d, device="cuda") if c["post"] else None
        s["dg_pre"] = torch.empty(d, device="cuda") if c["pre"] else None
        s["ws"] = torch.empty(max(16, 4 * 2 * 1024 * d), dtype=torch.uint8, device="cuda")
        return s

    k, E = c["k"], c["E"]
    n = T * k
    idx, w = _picks(c, g)
    if kind == "dispatch":
        d, xt = c["d"], _TYPES[c["x"]]
        s.update(idx=idx, x=_rows(g, T, d, xt), counts=_empty_int(E), offsets=_empty_int(E + 1), perm=_empty_int(n),
                 pos=_empty_int(n), xs=torch.zeros(n, d, dtype=xt, device="cuda"),
                 ws=torch.empty(4 << 20, dtype=torch.uint8, device="cuda"))
        return s
    counts, offsets, perm, pos = _sorted(idx, E)
    if kind == "dispatch_back":
        d, xt = c["d"], _TYPES[c["x"]]
        s.update(pos=pos, dxs=_rows(g, n, d, xt), dx=torch.empty(T, d, dtype=xt, device="cuda"))
    elif kind == "combine":
        d, yt, ot = c["d"], _TYPES[c["y"]], _TYPES[c["out"]]
        s.update(pos=pos, w=w, ys=_rows(g, n, d, yt), base=_rows(g, T, d, ot) if c["base"] else None,
                 out=torch.empty(T, d, dtype=ot, device="cuda"))
    elif kind == "combine_back":
        d, yt, ot = c["d"], _TYPES[c["y"]], _TYPES[c["out"]]
        s.update(pos=pos, w=w, ys=_rows(g, n, d, yt), dout=_rows(g, T, d, ot),
                 dys=torch.zeros(n, d, dtype=yt, device="cuda"), dw=torch.empty(T, k, device="cuda"),
                 dz=torch.empty(T, k, device="cuda"))
    else:
        N, K, yt = c["N"], c["K"], _TYPES[c["y"]]
        bf = torch.bfloat16
        W = torch.empty(E, N, K, dtype=bf, device="cuda")
        for e0 in range(0, E, 64):   # the experts' weights, some at a time
            m = min(64, E - e0)
            W[e0:e0 + m] = (torch.randn(m, N, K, device="cuda", generator=g) / math.sqrt(K)).to(bf)
        s.update(offsets=offsets, W=W, x=_rows(g, n, K, bf), longest=int(counts.max().item()))
        s["ws"] = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        if kind == "product":
            s["out"] = torch.zeros(n, N, dtype=yt, device="cuda")
        else:
            s["dy"] = _rows(g, n, N, bf)
            s["dx"] = torch.zeros(n, K, dtype=yt, device="cuda")
            s["dW"] = torch.empty(E, N, K, dtype=_TYPES[c["dw"]], device="cuda")
    return s


# -------------------------------------------------------------- plain forms

def _picked(rows, pos):
    """rows[pos] in 32 bits as [T][k][d], zeros for dropped picks."""
    p = pos.long()
    v = rows.float()[p.clamp_min(0)]
    return torch.where((p >= 0)[..., None], v, torch.zeros_like(v))


def _plain_dispatch(s):
    c = s["case"]
    k, E = c["k"], c["E"]
    counts, offsets, perm, pos = _sorted(s["idx"], E)
    token = torch.div(perm.long().clamp_min(0), k, rounding_mode="floor")
    xs = s["x"].float()[token]
    if c["drop"]:   # the slots behind the last kept pick stay as they were
        xs = torch.where((perm >= 0)[:, None], xs, s["xs"].float())
    return {"counts": counts, "offsets": offsets, "perm": perm, "pos": pos, "xs": xs.to(s["x"].dtype)}


def _plain_dispatch_back(s):
    c = s["case"]
    return {"dx": _picked(s["dxs"], s["pos"].view(c["T"], c["k"])).sum(1).to(s["dxs"].dtype)}


def _plain_combine(s):
    c = s["case"]
    out = (_picked(s["ys"], s["pos"].view(c["T"], c["k"])) * s["w"][..., None]).sum(1)
    if s["base"] is not None:
        out = out + s["base"].float()
    return {"out": out.to(s["out"].dtype)}


def _plain_combine_back(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    pos = s["pos"].view(T, k)
    dout, w = s["dout"].float(), s["w"]
    dw = (_picked(s["ys"], pos) * dout[:, None, :]).sum(2)
    dz = w * (dw - (w * dw).sum(1, keepdim=True))
    p = pos.reshape(-1).long()
    rows = (w[..., None] * dout[:, None, :]).reshape(T * k, -1)
    spare = torch.empty(T * k + 1, rows.shape[1], device=rows.device)   # one row more, where the dropped picks' rows go
    if s["case"]["drop"]:
        spare[:-1] = s["dys"].float()
    spare[torch.where(p >= 0, p, torch.full_like(p, T * k))] = rows
    return {"dys": spare[:-1].to(s["dys"].dtype), "dw": dw, "dz": dz}


def _slots(s, rows):
    """The rows of each expert, padded to the longest: indices [E][longest] and which of them are rows."""
    off = s["offsets"].long()
    j = torch.arange(s["longest"], device=off.device)
    at = off[:-1, None] + j[None, :]
    real = at < off[1:, None]
    return torch.where(real, at, torch.zeros_like(at)), real


def _expert_of(s, rows):
    """Expert and place in its segment of every row, and which rows belong to one."""
    off = s["offsets"].long()
    at = torch.arange(rows, device=off.device)
    e = torch.searchsorted(off[1:].contiguous(), at, right=True)
    real = at < off[-1]
    e = torch.where(real, e, torch.zeros_like(e))
    return e, torch.where(real, at - off[e], torch.zeros_like(at)), real


def _padded(v, at, real):
    p = v.float()[at]
    return torch.where(real[..., None], p, torch.zeros_like(p))


def _plain_product(s):
    x, W, out = s["x"], s["W"], s["out"]
    rows = x.shape[0]
    e, j, real = _expert_of(s, rows)
    if rows * 4 <= W.shape[0]:   # few rows: only the experts they picked
        y = (W[e].float() * x.float()[:, None, :]).sum(2)
    else:
        at, there = _slots(s, rows)
        y = torch.bmm(_padded(x, at, there), W.float().transpose(1, 2))[e, j] if s["longest"] else out.float()
    if s["case"]["drop"]:   # rows behind the last expert's stay as they were
        y = torch.where(real[:, None], y, out.float())
    return {"y": y.to(out.dtype)}


def _plain_product_back(s):
    x, W, dy, dx, dW = s["x"], s["W"], s["dy"], s["dx"], s["dW"]
    e, j, real = _expert_of(s, x.shape[0])
    if not s["longest"]:
        return {"dx": dx, "dW": torch.zeros_like(dW)}
    at, there = _slots(s, x.shape[0])
    dyp = _padded(dy, at, there)
    gx = torch.bmm(dyp, W.float())[e, j]
    gw = torch.bmm(dyp.transpose(1, 2).contiguous(), _padded(x, at, there))
    if s["case"]["drop"]:
        gx = torch.where(real[:, None], gx, dx.float())
    return {"dx": gx.to(dx.dtype), "dW": gw.to(dW.dtype)}


def _gate_values(s):
    """The gate as it multiplies the branch, and the derivative of that."""
    c = s["case"]
    if s["gate"] is None:
        return None, None
    gv = s["gate"].float()
    gv = gv[:, None] if c["gate"] == "token" else gv
    if not c["sigmoid"]:
        return gv, torch.ones_like(gv)
    sg = 1.0 / (1.0 + torch.exp(-gv))
    return sg, sg * (1.0 - sg)


def _plain_norm(s):
    c = s["case"]
    x, y = s["x"].float(), s["y"].float()
    got = {}
    if c["post"]:
        rstd = 1.0 / torch.sqrt((y * y).mean(1) + EPS)
        y = y * rstd[:, None] * s["g_post"]
        got["rstd_y"] = rstd
    gv, _ = _gate_values(s)
    r = s["a"] * x + s["b"] * (y if gv is None else gv * y)
    got["r"] = r.to(s["r"].dtype)
    if c["pre"]:
        rstd = 1.0 / torch.sqrt((r * r).mean(1) + EPS)
        got["u"] = (r * rstd[:, None] * s["g_pre"]).to(s["u"].dtype)
        got["rstd_r"] = rstd
    return got


def _plain_norm_back(s):
    c = s["case"]
    y, r, dr = s["y"].float(), s["r"].float(), s["dr"].float()
    got = {}
    if c["pre"]:
        du, rs = s["du"].float(), s["rstd_r"][:, None]
        rn = r * rs
        got["dg_pre"] = (du * rn).sum(0)
        gd = du * s["g_pre"]
        dr = dr + rs * (gd - rn * (gd * rn).mean(1, keepdim=True))
    got["dx"] = (s["a"] * dr).to(s["dx"].dtype)
    yn = y * s["rstd_y"][:, None] if c["post"] else y
    n = yn * s["g_post"] if c["post"] else yn
    gv, dg = _gate_values(s)
    db = s["b"] * dr
    if gv is not None:
        t = db * n
        t = t.sum(1, keepdim=True) if c["gate"] == "token" else t
        got["dgate"] = (t * dg).reshape(s["gate"].shape).to(s["gate"].dtype)
        db = db * gv
    if c["post"]:
        got["dg_post"] = (db * yn).sum(0)
        db = db * s["g_post"]
        db = s["rstd_y"][:, None] * (db - yn * (db * yn).mean(1, keepdim=True))
    got["dy"] = db.to(s["dy"].dtype)
    return got


# ------------------------------------------------------- the library's calls

def _own_dispatch(s):
    brx, c = _lib(), s["case"]
    T, k, E, d = c["T"], c["k"], c["E"], c["d"]
    brx.sort_picks(s["idx"], T, k, E, s["counts"], s["offsets"], s["perm"], s["pos"], s["ws"], s["ws"].numel())
    brx.dispatch(s["x"], _CODE[c["x"]], T, k, d, s["pos"], s["xs"], T * k)
    return {"counts": s["counts"], "offsets": s["offsets"], "perm": s["perm"], "pos": s["pos"], "xs": s["xs"]}


def _own_dispatch_back(s):
    c = s["case"]
    _lib().dispatch_backward(s["dxs"], _CODE[c["x"]], c["T"] * c["k"], s["pos"], c["T"], c["k"], c["d"], s["dx"])
    return {"dx": s["dx"]}


def _own_combine(s):
    c = s["case"]
    _lib().combine(s["ys"], _CODE[c["y"]], c["T"] * c["k"], s["pos"], s["w"], c["T"], c["k"], c["d"], s["out"],
                   _CODE[c["out"]], base=s["base"])
    return {"out": s["out"]}


def _own_combine_back(s):
    c = s["case"]
    _lib().combine_backward(s["dout"], _CODE[c["out"]], s["ys"], _CODE[c["y"]], c["T"] * c["k"], s["pos"], s["w"],
                            c["T"], c["k"], c["d"], dys=s["dys"], dw=s["dw"], dz=s["dz"])
    return {"dys": s["dys"], "dw": s["dw"], "dz": s["dz"]}


def _own_product(s):
    c = s["case"]
    _lib().grouped_product(s["x"], s["W"], s["offsets"], c["T"] * c["k"], c["E"], c["N"], c["K"], s["out"],
                           _CODE[c["y"]], s["ws"], s["ws"].numel())
    return {"y": s["out"]}


def _own_product_back(s):
    brx, c = _lib(), s["case"]
    rows, E, N, K = c["T"] * c["k"], c["E"], c["N"], c["K"]
    brx.grouped_dgrad(s["dy"], s["W"], s["offsets"], rows, E, N, K, s["dx"], _CODE[c["y"]], s["ws"], s["ws"].numel())
    brx.grouped_wgrad(s["dy"], s["x"], s["offsets"], rows, E, N, K, s["dW"], _CODE[c["dw"]], s["ws"], s["ws"].numel())
    return {"dx": s["dx"], "dW": s["dW"]}


def _norm_args(s):
    brx, c = _lib(), s["case"]
    return brx.block_norm_args(
        T=c["T"], d=c["d"], x_dtype=_CODE[c["x"]], y_dtype=_CODE[c["y"]], u_dtype=_CODE[c["u"]],
        flags=(brx.POST_NORM if c["post"] else 0) | (brx.PRE_NORM if c["pre"] else 0) |
        {"none": 0, "token": brx.GATE_TOKEN, "channel": brx.GATE_CHANNEL}[c["gate"]] |
        (brx.GATE_SIGMOID if c["sigmoid"] else 0),
        resid_scale=s["a"], branch_scale=s["b"], eps=EPS)


def _own_norm(s):
    _lib().block_norm(_norm_args(s), s["x"], s["y"], gate=s["gate"], g_post=s["g_post"], g_pre=s["g_pre"], r=s["r"],
                      u=s["u"], rstd_y=s["rstd_y"], rstd_r=s["rstd_r"])
    return {n: s[n] for n in ("rstd_y", "r", "u", "rstd_r") if s[n] is not None}


def _own_norm_back(s):
    _lib().block_norm_backward(_norm_args(s), s["dr"], s["du"], s["r"], s["y"], gate=s["gate"], g_post=s["g_post"],
                               g_pre=s["g_pre"], rstd_y=s["rstd_y"], rstd_r=s["rstd_r"], dx=s["dx"], dy=s["dy"],
                               dgate=s["dgate"], dg_post=s["dg_post"], dg_pre=s["dg_pre"], ws=s["ws"],
                               ws_bytes=s["ws"].numel())
    return {n: s[n] for n in ("dg_pre", "dx", "dgate", "dg_post", "dy") if s[n] is not None}


_PLAIN = {"dispatch": _plain_dispatch, "dispatch_back": _plain_dispatch_back, "combine": _plain_combine,
          "combine_back": _plain_combine_back, "product": _plain_product, "product_back": _plain_product_back,
          "norm": _plain_norm, "norm_back": _plain_norm_back}
_OWN = {"dispatch": _own_dispatch, "dispatch_back": _own_dispatch_back, "combine": _own_combine,
        "combine_back": _own_combine_back, "product": _own_product, "product_back": _own_product_back,
        "norm": _own_norm, "norm_back": _own_norm_back}


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


# -------------------------------------------------------------------- work

def work(case):
    """Bytes each read or written once, and multiply-adds counted as two."""
    c = case
    kind, T = c["kind"], c["T"]
    if kind in ("norm", "norm_back"):
        d, n = c["d"], c["T"] * c["d"]
        sx, sy, su = _SIZE[c["x"]], _SIZE[c["y"]], _SIZE[c["u"]]
        gate = {"none": 0, "token": 4 * T, "channel": n * sy}[c["gate"]]
        gains = 4 * d * (c["post"] + c["pre"])
        rstds = 4 * T * (c["post"] + c["pre"])
        if kind == "norm":
            return {"bytes": n * (2 * sx + sy + (su if c["pre"] else 0)) + gate + gains + rstds, "flops": 12 * n}
        return {"bytes": n * (2 * sx + 2 * sy + (su + sx if c["pre"] else 0)) + 2 * gate + 2 * gains + rstds,
                "flops": 30 * n}
    k, E = c["k"], c["E"]
    n = T * k
    kept = int(n * (1.0 - c["drop"]))
    if kind == "dispatch":
        row = c["d"] * _SIZE[c["x"]]
        return {"bytes": 12 * n + 8 * E + 4 + row * (T + kept), "flops": 0}
    if kind == "dispatch_back":
        row = c["d"] * _SIZE[c["x"]]
        return {"bytes": 4 * n + row * (T + kept), "flops": c["d"] * kept}
    if kind == "combine":
        d = c["d"]
        return {"bytes": 8 * n + d * (kept * _SIZE[c["y"]] + T * _SIZE[c["out"]] * (2 if c["base"] else 1)),
                "flops": 2 * d * kept}
    if kind == "combine_back":
        d = c["d"]
        return {"bytes": 16 * n + d * (2 * kept * _SIZE[c["y"]] + T * _SIZE[c["out"]]), "flops": 3 * d * kept}
    N, K = c["N"], c["K"]
    used = E * (1.0 - (1.0 - k * (1.0 - c["drop"]) / E) ** T)   # experts with rows, on average
    weights = int(used) * N * K
    if kind == "product":
        return {"bytes": 4 * (E + 1) + 2 * weights + kept * (2 * K + N * _SIZE[c["y"]]), "flops": 2 * kept * N * K}
    return {"bytes": 4 * (E + 1) + 2 * weights + E * N * K * _SIZE[c["dw"]] +
            kept * (2 * K + 2 * N + K * _SIZE[c["y"]]), "flops": 4 * kept * N * K}


# ------------------------------------------------------------ 64-bit values

def _exact_dispatch(s):
    x, idx, c = s["x"], s["idx"].cpu(), s["case"]
    flat = idx.reshape(-1).tolist()
    by = sorted((e, f) for f, e in enumerate(flat) if 0 <= e < c["E"])
    xs = s["xs"].double().clone()
    if by:
        xs[:len(by)] = x.double()[torch.tensor([f // c["k"] for _, f in by], device=x.device)]
    return {"counts": None, "offsets": None, "perm": None, "pos": None, "xs": xs}


def _exact_sum(rows, pos, w, T, k):
    """Sum over r of w[t][r] * rows[pos[t][r]], one pick of all tokens at a time."""
    total = torch.zeros(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    for r in range(k):
        p = pos.view(T, k)[:, r].long()
        has = (p >= 0).nonzero().flatten()
        v = rows[p[has]].double()
        total[has] += v if w is None else v * w.double()[has, r][:, None]
    return total


def _exact_combine_back(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    pos = s["pos"].view(T, k).long()
    dout, w = s["dout"].double(), s["w"].double()
    dys = s["dys"].double().clone()
    dw = torch.zeros(T, k, dtype=torch.float64, device=dout.device)
    for r in range(k):
        has = (pos[:, r] >= 0).nonzero().flatten()
        p = pos[has, r]
        dw[has, r] = torch.linalg.vecdot(dout[has], s["ys"][p].double())
        dys[p] = w[has, r][:, None] * dout[has]
    jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    return {"dys": dys, "dw": dw, "dz": (jac * dw[:, None, :]).sum(2)}


def _exact_product(s, back):
    off = s["offsets"].tolist()
    x, W = s["x"], s["W"]
    if not back:
        out = s["out"].double().clone()
        for e in range(W.shape[0]):
            if off[e + 1] > off[e]:
                out[off[e]:off[e + 1]] = torch.mm(x[off[e]:off[e + 1]].double(), W[e].double().t().contiguous())
        return {"y": out}
    dx = s["dx"].double().clone()
    dW = torch.zeros(W.shape, dtype=torch.float64, device=W.device)
    for e in range(W.shape[0]):
        if off[e + 1] > off[e]:
            dy = s["dy"][off[e]:off[e + 1]].double()
            dx[off[e]:off[e + 1]] = torch.mm(dy, W[e].double())
            dW[e] = torch.mm(dy.t().contiguous(), x[off[e]:off[e + 1]].double())
    return {"dx": dx, "dW": dW}


def _exact_branch(c, s, y, gate, g_post):
    n = y
    ry = None
    if c["post"]:
        ry = (y.square().sum(1) / y.shape[1] + EPS).rsqrt()
        n = y * ry[:, None] * g_post
    if gate is not None:
        gv = torch.sigmoid(gate) if c["sigmoid"] else gate
        n = n * (gv[:, None] if c["gate"] == "token" else gv)
    return s["b"] * n, ry


def _exact_norm(s):
    c = s["case"]
    up = lambda v: None if v is None else v.double()  # noqa: E731
    branch, ry = _exact_branch(c, s, up(s["y"]), up(s["gate"]), up(s["g_post"]))
    r = s["a"] * s["x"].double() + branch
    got = {"r": r}
    if c["post"]:
        got["rstd_y"] = ry
    if c["pre"]:
        rr = (r.square().sum(1) / r.shape[1] + EPS).rsqrt()
        got.update(u=r * rr[:, None] * up(s["g_pre"]), rstd_r=rr)
    return got


def _exact_norm_back(s):
    """The gradients by differentiating the definition in 64 bits; the residual rows are the stored ones."""
    c = s["case"]
    leaf = lambda v: None if v is None else v.double().detach().requires_grad_(True)  # noqa: E731
    y, gate, g_post, g_pre, r = leaf(s["y"]), leaf(s["gate"]), leaf(s["g_post"]), leaf(s["g_pre"]), leaf(s["r"])
    got = {}
    dr = s["dr"].double()
    if c["pre"]:
        u = r * (r.square().mean(1, keepdim=True) + EPS).rsqrt() * g_pre
        a, b = torch.autograd.grad(u, [r, g_pre], s["du"].double())
        dr = dr + a
        got["dg_pre"] = b
    got["dx"] = s["a"] * dr
    branch, _ = _exact_branch(c, s, y, gate, g_post)
    names = [n for n, v in (("dy", y), ("dgate", gate), ("dg_post", g_post)) if v is not None]
    leaves = [v for v in (y, gate, g_post) if v is not None]
    got.update(zip(names, torch.autograd.grad(branch, leaves, dr)))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    kind, c = case["kind"], case
    if kind == "dispatch":
        got = _exact_dispatch(s)
    elif kind == "dispatch_back":
        got = {"dx": _exact_sum(s["dxs"], s["pos"], None, c["T"], c["k"])}
    elif kind == "combine":
        total = _exact_sum(s["ys"], s["pos"], s["w"], c["T"], c["k"])
        got = {"out": total if s["base"] is None else total + s["base"].double()}
    elif kind == "combine_back":
        got = _exact_combine_back(s)
    elif kind in ("product", "product_back"):
        got = _exact_product(s, kind == "product_back")
    else:
        got = _exact_norm(s) if kind == "norm" else _exact_norm_back(s)
    order = {"norm": ("rstd_y", "r", "u", "rstd_r"), "norm_back": ("dg_pre", "dx", "dgate", "dg_post", "dy")}.get(kind)
    return {n: got[n] for n in order if n in got} if order else got
