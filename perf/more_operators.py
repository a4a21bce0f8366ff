"""Operators at the ends of a training step: what is measured, in which sizes.

Four kinds of work, each as a user's program calls it:

- balance: the router's balance and z losses with the picks counted per expert; the logits' gradient.
- embed: table rows of token ids, scaled; the table's gradient.
- vocab: softmax cross entropy over the vocabulary, from hidden rows and the output matrix; both gradients.
- orth: the experts' updates orthogonalised by Newton-Schulz products.

``own`` selects between the plain form (elementary torch operations in 32
bits) and the library's kernels.
"""
import math

import torch

own = False


def _lib():
    import bit_routed_expert_amd as brx
    return brx


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CODE = {"bf16": 0, "f32": 1}   # STRATA_X_BF16, STRATA_X_F32
_SIZE = {"bf16": 2, "f32": 4}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # of X, (X X^T) X and (X X^T)^2 X in a Newton-Schulz step
ORTH_EPS = 1e-7


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a verify step's five tokens, the full-size router: launch latency
        dict(name="balance_verify", kind="balance", T=5, k=10, E=512, z="f32", keep=1.0),
        # a 32K-token prompt's or batch's router logits
        dict(name="balance_batch", kind="balance", T=32768, k=10, E=512, z="f32", keep=1.0),
        # a padded training batch: the losses' gradient and that of the picked logits, bf16 logits
        dict(name="balance_back", kind="balance_back", T=16384, k=10, E=512, z="bf16", keep=0.9, picks=True),
        # a verify step's five tokens
        dict(name="embed_verify", kind="embed", T=5, V=128000, d=2048, w="bf16", out="f32", pad=0.0),
        # a training batch's gradient over the whole table, token frequencies falling as one over the rank
        dict(name="embed_back", kind="embed_back", T=16384, V=128000, d=2048, w="bf16", out="bf16", pad=0.1),
        # scoring a verify step's five tokens: the output matrix read once
        dict(name="vocab_verify", kind="vocab", T=5, V=128000, d=2048, ignore=0.0),
        # losses of a 4096-token chunk
        dict(name="vocab_chunk", kind="vocab", T=4096, V=128000, d=2048, ignore=0.0),
        # gradients of a 4096-token training batch; a quarter of the tokens (prompts, padding) has no target
        dict(name="vocab_back", kind="vocab_back", T=4096, V=128000, d=2048, ignore=0.25, dh="bf16", dw="bf16"),
        # a ragged batch, an odd vocabulary, gradients kept in 32 bits
        dict(name="vocab_back_f32", kind="vocab_back", T=2047, V=50001, d=1000, ignore=0.1, dh="f32", dw="f32"),
        # the gate and up matrices of the small layer's 16 experts: latency
        dict(name="orth_small", kind="orth", E=16, N=128, K=256, g="bf16"),
        # gate and up rows of 16 full-size experts, gradients in 32 bits
        dict(name="orth_experts", kind="orth", E=16, N=1536, K=2048, g="f32"),
        # the down matrices of 8 full-size experts: more rows than columns
        dict(name="orth_down", kind="orth", E=8, N=2048, K=768, g="bf16"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["balance", "balance_back", "embed", "embed_back", "vocab", "vocab_back", "vocab_back", "orth", "orth"])
    t = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    c = {"kind": kind}
    if kind in ("balance", "balance_back"):
        E = _logint(rng, 4, 512)
        c.update(T=_logint(rng, 1, 32768), k=rng.randint(1, min(E, 12)), E=E, z=t(), keep=rng.choice([1.0, 0.9, 0.5]))
        if kind == "balance_back":
            c["picks"] = rng.random() < 0.5
        return c
    if kind in ("embed", "embed_back"):
        d = rng.choice([128 * rng.randint(1, 16), 8 * rng.randint(8, 256), rng.randint(64, 2048)])
        c.update(T=_logint(rng, 1, 16384), V=_logint(rng, 100, 128000), d=d, w=t(), out=t(), pad=rng.choice([0.0, 0.1]))
        return c
    if kind == "orth":
        E, N, K = _logint(rng, 1, 64), _logint(rng, 16, 2048), _logint(rng, 16, 2048)
        while E > 1 and E * N * K * min(N, K) > 16 * 1536 * 2048 * 1536:
            E = (E + 1) // 2
        c.update(E=E, N=N, K=K, g=t())
        return c
    T, V, d = _logint(rng, 1, 4096), _logint(rng, 64, 128000), 8 * rng.randint(8, 256)
    c.update(T=T, V=V, d=d, ignore=rng.choice([0.0, 0.1, 0.5]))
    if kind == "vocab_back":
        c.update(dh=t(), dw=t())
    return c


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _tokens(g, n, V):
    """Ids whose frequency falls as one over their rank, ranks dealt to ids by a permutation."""
    rank = torch.exp(_rand(g, n).double() * math.log(V)).long().clamp_(1, V) - 1
    return torch.randperm(V, device="cuda", generator=g)[rank].int()


def _weights(g, V, d):
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    for v in range(0, V, 16384):   # some rows at a time
        m = min(16384, V - v)
        W[v:v + m] = (_randn(g, m, d) * (1.5 / math.sqrt(d))).to(torch.bfloat16)
    return W


def _workspace(n):
    """A program allocates its workspace once; no less than any of its calls asks for."""
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed + 1))
    kind = c["kind"]
    s = {"case": c}
    if kind in ("balance", "balance_back"):
        T, k, E = c["T"], c["k"], c["E"]
        z = (_randn(g, T, E) + 0.7 * _randn(g, E)).to(_TYPES[c["z"]])
        idx = torch.topk(z.float(), k, dim=1).indices.int().contiguous()
        keep = None if c["keep"] == 1.0 else (_rand(g, T) < c["keep"])
        s.update(z=z, idx=idx, keep=keep)
        if kind == "balance":
            s.update(losses=torch.empty(2, device="cuda"), counts=torch.empty(E, dtype=torch.int32, device="cuda"),
                     prob=torch.empty(E, device="cuda"), lse=torch.empty(T, device="cuda"),
                     tokens=torch.empty(1, dtype=torch.int32, device="cuda"),
                     ws=_workspace(16 << 20))
            return s
        # what the forward pass left for the gradient
        lse = torch.logsumexp(z.double(), 1)
        counted = torch.ones(T, dtype=torch.bool, device="cuda") if keep is None else keep
        s["lse"] = torch.where(counted, lse, torch.zeros_like(lse)).float()
        s["counts"] = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(
            0, idx.reshape(-1).long(), counted[:, None].expand(T, k).reshape(-1).long()).int()
        s["tokens"] = counted.sum().int().reshape(1)
        s["dlosses"] = torch.tensor([0.01, 0.001], device="cuda")
        s["dpicks"] = _randn(g, T, k) / T if c["picks"] else None
        s["dz"] = torch.empty_like(z)
        return s
    if kind in ("embed", "embed_back"):
        T, V, d = c["T"], c["V"], c["d"]
        ids = _tokens(g, T, V)
        ids = torch.where(_rand(g, T) < c["pad"], torch.full_like(ids, -1), ids)
        s.update(ids=ids, scale=math.sqrt(d))
        if kind == "embed":
            s["W"] = torch.empty(V, d, dtype=_TYPES[c["w"]], device="cuda").normal_(0.0, 1.0 / math.sqrt(d), generator=g)
            s["out"] = torch.empty(T, d, dtype=_TYPES[c["out"]], device="cuda")
        else:
            s["dout"] = _randn(g, T, d).to(_TYPES[c["out"]])
            s["dW"] = torch.empty(V, d, dtype=_TYPES[c["w"]], device="cuda")
            s["ws"] = _workspace(32 * T + 2 * d * T + (16 << 20))
        return s
    if kind == "orth":
        E, N, K = c["E"], c["N"], c["K"]
        # momentum of gradients: a few strong directions in a full-rank rest
        r = max(1, min(N, K) // 16)
        G = _randn(g, E, N, K) + torch.bmm(_randn(g, E, N, r), 3.0 * _randn(g, E, r, K)) / math.sqrt(r)
        s.update(G=(1e-3 * G).to(_TYPES[c["g"]]), out=torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda"),
                 scale=math.sqrt(max(1.0, N / K)))
        s["ws"] = _workspace(16 * E * (N + 64) * (K + 64) + (16 << 20))
        return s
    T, V, d = c["T"], c["V"], c["d"]
    s["h"] = _randn(g, T, d).to(torch.bfloat16)
    s["W"] = _weights(g, V, d)
    targets = _tokens(g, T, V)
    s["targets"] = torch.where(_rand(g, T) < c["ignore"], torch.full_like(targets, -1), targets)
    if kind == "vocab":
        s.update(loss=torch.empty(T, device="cuda"), lse=torch.empty(T, device="cuda"))
        s["ws"] = _workspace(T * (V // 8 + 2 * d) + (16 << 20))
        return s
    # what the forward pass left, and the gradient of the mean loss with a small weight on the squared normaliser
    valid = s["targets"] >= 0
    z = torch.mm(s["h"].float(), s["W"].float().t())
    lse = torch.where(valid, torch.logsumexp(z, 1), torch.zeros(T, device="cuda"))
    del z
    s["lse"] = lse
    n = valid.sum().clamp_min(1)
    s["dloss"] = torch.ones(T, device="cuda") / n
    s["dlse"] = 2e-4 * lse / n
    s["dh"] = torch.empty(T, d, dtype=_TYPES[c["dh"]], device="cuda")
    s["dW"] = torch.empty(V, d, dtype=_TYPES[c["dw"]], device="cuda")
    s["ws"] = _workspace(1 << 30)
    return s


# -------------------------------------------------------------- plain forms

def _counted(s):
    """Rows that count: kept ones."""
    T = s["z"].shape[0]
    return torch.ones(T, dtype=torch.bool, device=s["z"].device) if s["keep"] is None else s["keep"]


def _plain_balance(s):
    c = s["case"]
    k, E = c["k"], c["E"]
    z, on = s["z"].float(), _counted(s)
    m = z.max(1, keepdim=True).values
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = torch.where(on, (m + torch.log(total))[:, 0], torch.zeros_like(m[:, 0]))
    n = on.sum()
    prob = torch.where(on[:, None], e / total, torch.zeros_like(e)).sum(0) / n.clamp_min(1)
    counts = torch.zeros(E, dtype=torch.int64, device=z.device).scatter_add_(
        0, s["idx"].reshape(-1).long(), on[:, None].expand(-1, k).reshape(-1).long())
    balance = E * (counts.float() / (n * k).clamp_min(1) * prob).sum()
    zloss = (lse * lse).sum() / n.clamp_min(1)
    return {"losses": torch.stack([balance, zloss]), "counts": counts.int(), "prob": prob, "lse": lse,
            "tokens": n.int().reshape(1)}


def _plain_balance_back(s):
    c = s["case"]
    k, E = c["k"], c["E"]
    on = _counted(s)[:, None]
    n = s["tokens"].float().clamp_min(1)
    p = torch.exp(s["z"].float() - s["lse"][:, None])
    g = s["dlosses"][0] * E * s["counts"].float() / (n * n * k)
    dz = p * (g - (p * g).sum(1, keepdim=True)) + p * (2.0 * s["dlosses"][1] / n * s["lse"])[:, None]
    if s["dpicks"] is not None:
        dz = dz.scatter_add(1, s["idx"].long(), s["dpicks"])
    return {"dz": torch.where(on, dz, torch.zeros_like(dz)).to(s["z"].dtype)}


def _plain_embed(s):
    ids = s["ids"].long()
    rows = s["W"][ids.clamp_min(0)].float() * s["scale"]
    return {"out": torch.where((ids >= 0)[:, None], rows, torch.zeros_like(rows)).to(s["out"].dtype)}


def _plain_embed_back(s):
    ids = s["ids"].long()
    V, d = s["dW"].shape
    rows = torch.zeros(V + 1, d, device=ids.device)   # one row more, for the ids without a row
    rows.index_add_(0, torch.where(ids >= 0, ids, torch.full_like(ids, V)), s["dout"].float())
    return {"dW": (rows[:V] * s["scale"]).to(s["dW"].dtype)}


def _plain_vocab(s):
    valid = s["targets"] >= 0
    z = torch.mm(s["h"].float(), s["W"].float().t())
    m = z.max(1, keepdim=True).values
    picked = z.gather(1, s["targets"].long().clamp_min(0)[:, None])[:, 0]
    lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
    none = torch.zeros_like(lse)
    return {"loss": torch.where(valid, lse - picked, none), "lse": torch.where(valid, lse, none)}


def _plain_vocab_back(s):
    valid = s["targets"] >= 0
    h, W = s["h"].float(), s["W"].float()
    none = torch.zeros_like(s["dloss"])
    dloss, dlse = torch.where(valid, s["dloss"], none), torch.where(valid, s["dlse"], none)
    dz = torch.exp(torch.mm(h, W.t()) - s["lse"][:, None]) * (dloss + dlse)[:, None]
    dz.scatter_add_(1, s["targets"].long().clamp_min(0)[:, None], -dloss[:, None])
    dz = torch.where(valid[:, None], dz, torch.zeros_like(dz))
    return {"dh": torch.mm(dz, W).to(s["dh"].dtype), "dW": torch.mm(dz.t(), h).to(s["dW"].dtype)}


def _plain_orth(s):
    G = s["G"].float()
    tall = G.shape[1] > G.shape[2]
    X = G.transpose(1, 2).contiguous() if tall else G
    X = X / (torch.sqrt((X * X).sum((1, 2), keepdim=True)) + ORTH_EPS)
    a, b, c = COEFFICIENTS
    for _ in range(5):
        A = torch.bmm(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    X = X.transpose(1, 2).contiguous() if tall else X
    return {"out": (s["scale"] * X).to(torch.bfloat16)}


# ------------------------------------------------------- the library's calls

def _own_balance(s):
    c = s["case"]
    _lib().balance_loss(s["z"], _CODE[c["z"]], s["idx"], c["T"], c["k"], c["E"], s["losses"], s["counts"], s["lse"],
                        s["tokens"], s["ws"], s["ws"].numel(), prob=s["prob"], keep=s["keep"])
    return {n: s[n] for n in ("losses", "counts", "prob", "lse", "tokens")}


def _own_balance_back(s):
    c = s["case"]
    _lib().balance_loss_backward(s["z"], _CODE[c["z"]], s["idx"], c["T"], c["k"], c["E"], s["lse"], s["counts"],
                                 s["tokens"], s["dlosses"], s["dz"], keep=s["keep"], dpicks=s["dpicks"])
    return {"dz": s["dz"]}


def _own_embed(s):
    c = s["case"]
    _lib().embed(s["W"], _CODE[c["w"]], c["V"], c["d"], s["ids"], c["T"], s["scale"], s["out"], _CODE[c["out"]])
    return {"out": s["out"]}


def _own_embed_back(s):
    c = s["case"]
    _lib().embed_backward(s["dout"], _CODE[c["out"]], s["ids"], c["T"], c["V"], c["d"], s["scale"], s["dW"], _CODE[c["w"]],
                          s["ws"], s["ws"].numel())
    return {"dW": s["dW"]}


def _own_vocab(s):
    c = s["case"]
    _lib().vocab_loss(s["h"], s["W"], s["targets"], c["T"], c["V"], c["d"], s["loss"], s["lse"], s["ws"], s["ws"].numel())
    return {"loss": s["loss"], "lse": s["lse"]}


def _own_vocab_back(s):
    c = s["case"]
    _lib().vocab_loss_backward(s["h"], s["W"], s["targets"], c["T"], c["V"], c["d"], s["lse"], s["dloss"], s["ws"],
                               s["ws"].numel(), dlse=s["dlse"], dh=s["dh"], dhdtype=_CODE[c["dh"]], dW=s["dW"],
                               dwdtype=_CODE[c["dw"]])
    return {"dh": s["dh"], "dW": s["dW"]}


def _own_orth(s):
    c = s["case"]
    _lib().orthogonalise(s["G"], _CODE[c["g"]], c["E"], c["N"], c["K"], s["out"], s["ws"], s["ws"].numel(), steps=5,
                         coefficients=COEFFICIENTS, scale=s["scale"], eps=ORTH_EPS)
    return {"out": s["out"]}


_PLAIN = {"balance": _plain_balance, "balance_back": _plain_balance_back, "embed": _plain_embed,
          "embed_back": _plain_embed_back, "vocab": _plain_vocab, "vocab_back": _plain_vocab_back, "orth": _plain_orth}
_OWN = {"balance": _own_balance, "balance_back": _own_balance_back, "embed": _own_embed, "embed_back": _own_embed_back,
        "vocab": _own_vocab, "vocab_back": _own_vocab_back, "orth": _own_orth}


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


# -------------------------------------------------------------------- work

def work(case):
    """Bytes each read or written once, and multiply-adds counted as two."""
    c = case
    kind = c["kind"]
    if kind in ("balance", "balance_back"):
        T, k, E = c["T"], c["k"], c["E"]
        kept = int(T * c["keep"])
        row = E * _SIZE[c["z"]]
        if kind == "balance":
            return {"bytes": kept * (row + 4 * k) + 4 * T + 8 * E + 12, "flops": 4 * kept * E}
        return {"bytes": kept * (row + 4 + (8 * k if c["picks"] else 0)) + T * row + 4 * E + 12, "flops": 6 * kept * E}
    if kind in ("embed", "embed_back"):
        T, V, d = c["T"], c["V"], c["d"]
        kept = int(T * (1.0 - c["pad"]))
        if kind == "embed":
            return {"bytes": 4 * T + d * (min(kept, V) * _SIZE[c["w"]] + T * _SIZE[c["out"]]), "flops": kept * d}
        return {"bytes": 4 * T + d * (kept * _SIZE[c["out"]] + V * _SIZE[c["w"]]), "flops": kept * d}
    if kind == "orth":
        E, N, K = c["E"], min(c["N"], c["K"]), max(c["N"], c["K"])
        # X X^T and its square are symmetric: half of each
        return {"bytes": E * N * K * (_SIZE[c["g"]] + 2), "flops": 5 * E * (N * (N + 1) * (K + N) + 2 * N * N * K)}
    T, V, d = c["T"], c["V"], c["d"]
    kept = int(T * (1.0 - c["ignore"]))
    if kind == "vocab":
        return {"bytes": 2 * d * (V + kept) + 12 * T, "flops": 2 * kept * V * d}
    return {"bytes": 2 * d * (V + kept) + 16 * T + d * (T * _SIZE[c["dh"]] + V * _SIZE[c["dw"]]), "flops": 6 * kept * V * d}


# ------------------------------------------------------------ 64-bit values

def _exact_balance_losses(z, on, idx, k, E):
    """Both losses of the kept rows' logits by the definition, and the counts."""
    rows = z[on]
    n = rows.shape[0]
    if n == 0:
        zero = z.sum() * 0.0
        return zero, zero, torch.zeros(E, dtype=torch.float64, device=z.device)
    prob = torch.softmax(rows, 1).mean(0)
    f = torch.stack([(idx[on] == e).sum() for e in range(E)]).double() / (n * k)
    return E * torch.dot(f, prob), torch.logsumexp(rows, 1).square().mean(), prob


def _exact_balance(s):
    c = s["case"]
    on = _counted(s)
    z = s["z"].double()
    balance, zloss, prob = _exact_balance_losses(z, on, s["idx"], c["k"], c["E"])
    lse = torch.zeros(c["T"], dtype=torch.float64, device=z.device)
    lse[on] = torch.logsumexp(z[on], 1)
    return {"losses": torch.stack([balance, zloss]), "counts": None, "prob": prob, "lse": lse, "tokens": None}


def _exact_balance_back(s):
    c = s["case"]
    z = s["z"].double().requires_grad_(True)
    balance, zloss, _ = _exact_balance_losses(z, _counted(s), s["idx"], c["k"], c["E"])
    w = s["dlosses"].double()
    total = w[0] * balance + w[1] * zloss
    if s["dpicks"] is not None:
        on = _counted(s)
        total = total + (z.gather(1, s["idx"].long())[on] * s["dpicks"].double()[on]).sum()
    return {"dz": torch.autograd.grad(total, z)[0]}


def _exact_vocab(s):
    T = s["h"].shape[0]
    W = s["W"].double().t().contiguous()
    loss, lse = (torch.zeros(T, dtype=torch.float64, device=W.device) for _ in range(2))
    has = (s["targets"] >= 0).nonzero().flatten()
    for some in has.split(1024):
        z = torch.mm(s["h"][some].double(), W)
        lse[some] = torch.logsumexp(z, 1)
        loss[some] = -torch.log_softmax(z, 1)[torch.arange(len(some), device=z.device), s["targets"][some].long()]
    return {"loss": loss, "lse": lse}


def _exact_vocab_back(s):
    """The gradients from the stored normalisers, some rows at a time."""
    T, d = s["h"].shape
    W = s["W"].double()
    Wt = W.t().contiguous()
    dh = torch.zeros(T, d, dtype=torch.float64, device=W.device)
    dW = torch.zeros_like(W)
    has = (s["targets"] >= 0).nonzero().flatten()
    for some in has.split(1024):
        h = s["h"][some].double()
        up, un = s["dloss"][some].double(), s["dlse"][some].double()
        dz = (torch.mm(h, Wt) - s["lse"][some].double()[:, None]).exp_().mul_((up + un)[:, None])
        at = torch.arange(len(some), device=W.device)
        dz[at, s["targets"][some].long()] -= up
        dh[some] = torch.mm(dz, W)
        dW.addmm_(dz.t(), h)
    return {"dh": dh, "dW": dW}


def _exact_orth(s):
    """The polynomial of the other product: a I + b X^T X + c (X^T X)^2 from the right (of the shorter side's matrix)."""
    a, b, c = COEFFICIENTS
    out = torch.empty(s["G"].shape, dtype=torch.float64, device=s["G"].device)
    for e in range(out.shape[0]):
        X = s["G"][e].double()
        X = X / (torch.linalg.matrix_norm(X) + ORTH_EPS)
        X = X.t().contiguous() if X.shape[0] < X.shape[1] else X
        for _ in range(5):
            A = torch.mm(X.t().contiguous(), X)
            P = b * A + c * torch.mm(A, A)
            P.diagonal().add_(a)
            X = torch.mm(X, P)
        out[e] = s["scale"] * (X.t() if out.shape[1] < out.shape[2] else X)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    ids = s["ids"].long() if "ids" in s else None
    if kind == "embed":
        out = torch.zeros(case["T"], case["d"], dtype=torch.float64, device=ids.device)
        has = (ids >= 0).nonzero().flatten()
        out[has] = s["W"][ids[has]].double() * s["scale"]
        return {"out": out}
    if kind == "embed_back":
        dW = torch.zeros(case["V"], case["d"], dtype=torch.float64, device=ids.device)
        has = (ids >= 0).nonzero().flatten()
        dW.index_add_(0, ids[has], s["dout"][has].double() * s["scale"])
        return {"dW": dW}
    return {"balance": _exact_balance, "balance_back": _exact_balance_back, "vocab": _exact_vocab,
            "vocab_back": _exact_vocab_back, "orth": _exact_orth}[kind](s)
