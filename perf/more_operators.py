"""The ends of a training step around the layer: cases, inputs, plain forms and the library's calls.

Three operators, named by a case's "op":
  balance        how evenly the router spreads T tokens, for each of B sequences of T/B tokens: picks of each expert, mean
                 probabilities, the balance loss E/k * sum_e (picks_e / n) * mean_t p[t, e] over the n tokens that a mask
                 leaves, the mean square of log(sum(exp(logits))), and the gradient of both for the logits, added to the
                 gradient that the layer's backward gives
  xent           softmax cross entropy of x W^T over a vocabulary of V rows against one target a token (below 0: none),
                 log(sum(exp)) of each token, and the gradients for x and W of weights on both
  orthogonalize  matrices to nearly orthogonal ones by five steps X <- a X + (b A + c A A) X, A = X X^T, of a matrix
                 divided by its Frobenius norm (on the transpose where there are more rows than columns)
"""
import math

import torch

own = False

DEV = "cuda"
COEF = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ----------------------------------------------------------------- cases
def _balance(name, T, E, k, B=1, masked=0.0, zipf=False):
    c = dict(op="balance", T=T, E=E, k=k, B=B, masked=masked, zipf=zipf)
    if name:
        c["name"] = name
    return c


def _xent(name, T, V, d, grad="", ignored=0.0, z=0.0):
    c = dict(op="xent", T=T, V=V, d=d, grad=grad, ignored=ignored, z=z)
    if name:
        c["name"] = name
    return c


def _ortho(name, mats, rows, cols, src="fp32", empty=0):
    c = dict(op="orthogonalize", mats=mats, rows=rows, cols=cols, src=src, empty=empty)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the tiny layer's router: nothing but latency
        _balance("balance_T512_E8", 512, 8, 2),
        # the DeepSeek-V2-Lite-like layer on four sequences that end in padding
        _balance("balance_T8192_E64_B4", 8192, 64, 6, B=4, masked=0.2),
        # heavy-tailed routing over 128 experts, 32 sequences
        _balance("balance_T32768_E128_B32", 32768, 128, 8, B=32, zipf=True),
        # one sequence of 128k tokens
        _balance("balance_T131072_E64", 131072, 64, 6),
        # the score of one answered token: every row of the projection is read for it
        _xent("xent_T1_V32000", 1, 32000, 2048),
        # the scores of a batch of answers, an odd vocabulary
        _xent("xent_T37_V50257_d4096", 37, 50257, 4096, ignored=0.1),
        # a training step of a small model with fp32 gradients
        _xent("xent_T512_V1000_fp32", 512, 1000, 256, grad="fp32", ignored=0.1),
        # a step's tokens where part is prompt and does not count, with a weight on log(sum(exp)) squared
        _xent("xent_T2000_V32001", 2000, 32001, 2048, grad="bf16", ignored=0.4, z=1e-4),
        # a whole step of the DeepSeek-V2-Lite-like layer's tokens over a large vocabulary
        _xent("xent_T8192_V100000", 8192, 100000, 2048, grad="bf16"),
        # a gate projection with fewer experts than anything else is wide: latency
        _ortho("orthogonalize_1x64x2048", 1, 64, 2048),
        # odd matrices with more rows than columns, one of an expert that saw no token
        _ortho("orthogonalize_5x1001x333", 5, 1001, 333, src="bf16", empty=1),
        # the gate projections of all experts of the DeepSeek-V2-Lite-like layer
        _ortho("orthogonalize_66x1408x2048", 66, 1408, 2048),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["balance", "xent", "xent", "orthogonalize"])
    if op == "balance":
        E = _log(rng, 2, 256)
        B = rng.choice([1, 1, 2, 7, _log(rng, 1, 64)])
        T = B * _log(rng, 1, max(1, 131072 * 64 // (E * B)))
        return _balance(None, T, E, rng.randint(1, min(E, 8)), B, rng.choice([0.0, 0.0, 0.1, 0.6]), rng.random() < 0.25)
    if op == "xent":
        d = 64 * _log(rng, 1, 64)
        V = _log(rng, 2, 120000)
        T = _log(rng, 1, 8192)
        while T * V * d > 8192 * 50000 * 2048:
            T = (T + 1) // 2
        return _xent(None, T, V, d, rng.choice(["", "bf16", "bf16", "fp32"]), rng.choice([0.0, 0.1, 0.5]),
                     rng.choice([0.0, 0.0, 1e-4]))
    mats, rows, cols = _log(rng, 1, 40), _log(rng, 2, 2500), _log(rng, 2, 2500)
    while mats * rows * cols * min(rows, cols) > 40 * 1408 * 1408 * 2048:
        mats = (mats + 1) // 2 if mats > 1 else 1
        rows = rows if mats > 1 else rows // 2
    return _ortho(None, mats, rows, cols, rng.choice(["fp32", "bf16"]), 1 if mats > 2 and rng.random() < 0.3 else 0)


# ----------------------------------------------------------------- inputs
def _gen(seed, n):
    return torch.Generator(device=DEV).manual_seed(seed * 1013 + n)


def _randn(shape, g, std=1.0, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _prepare_balance(st, seed):
    T, E, k, B = st["T"], st["E"], st["k"], st["B"]
    bias = -2.4 * torch.arange(1, E + 1, dtype=torch.float32, device=DEV).log() if st["zipf"] else 0.0
    st["logits"] = _randn((T, E), _gen(seed, 1)) + bias
    st["topk_idx"] = torch.sort(st["logits"], dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
    st["mask"] = None
    if st["masked"]:  # every sequence ends in padding, on average `masked` of it, some wholly
        L = T // B
        kept = (torch.rand(B, 1, generator=_gen(seed, 2), device=DEV) * 2 * st["masked"]).clamp(max=1.0)
        kept = ((1.0 - kept) * L).ceil().long()
        st["mask"] = (torch.arange(L, device=DEV) < kept).reshape(T)
        st["logits"][~st["mask"]] = float("nan")  # what padding holds is nobody's business
    st["dlogits_in"] = _randn((T, E), _gen(seed, 3), 1e-4)  # from the layer's backward
    st["dloss"] = torch.full((B,), 1e-2 / B, device=DEV)
    st["dz"] = torch.full((B,), 1e-3 / B, device=DEV)
    return st


def _prepare_xent(st, seed):
    T, V, d = st["T"], st["V"], st["d"]
    st["W"] = _randn((V, d), _gen(seed, 1), d ** -0.5, torch.bfloat16)
    target = torch.randint(V, (T,), generator=_gen(seed, 2), device=DEV)
    # a trained model's hidden states: some tokens are certain, some are not
    sure = torch.rand(T, 1, generator=_gen(seed, 3), device=DEV) * 1.5 * math.log(V + 1.0)
    x = _randn((T, d), _gen(seed, 4)) + sure * st["W"][target].float()
    st["x"] = x.bfloat16()
    drop = torch.rand(T, generator=_gen(seed, 5), device=DEV) < st["ignored"]
    st["target"] = torch.where(drop, -100, target)
    st["dloss"] = (~drop).float() / max(1, T - int(T * st["ignored"]))
    st["loss"], st["lse"] = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    if st["grad"]:
        dt = torch.float32 if st["grad"] == "fp32" else torch.bfloat16
        st["dx"], st["dW"] = torch.empty(T, d, dtype=dt, device=DEV), torch.empty(V, d, dtype=dt, device=DEV)
    return st


def _prepare_ortho(st, seed):
    M, m, n = st["mats"], st["rows"], st["cols"]
    dt = torch.float32 if st["src"] == "fp32" else torch.bfloat16
    r = min(16, m, n)  # a gradient: a few strong directions over noise
    G = torch.empty(M, m, n, dtype=dt, device=DEV)
    for i in range(M):
        g = _gen(seed, 10 + i)
        G[i] = (_randn((m, r), g) @ _randn((r, n), g) * 0.3 + _randn((m, n), g)) * 1e-3
    for i in range(st["empty"]):
        G[M - 1 - i] = 0.0
    st["G"] = G
    st["O"] = torch.empty(M, m, n, dtype=torch.bfloat16, device=DEV)
    return st


def prepare(case, seed):
    return {"balance": _prepare_balance, "xent": _prepare_xent, "orthogonalize": _prepare_ortho}[case["op"]](dict(case), seed)


# ------------------------------------------------------------- plain form
def _plain_balance(st):
    T, E, k, B = st["T"], st["E"], st["k"], st["B"]
    z, keep = st["logits"].view(B, -1, E), torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"]
    keep = keep.view(B, -1, 1)
    z = torch.where(keep, z, 0.0)
    m = z.amax(2, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(2, keepdim=True)
    p, lse = e / s, m + torch.log(s)
    picks = torch.zeros(T, E, dtype=torch.int32, device=DEV).scatter_(1, st["topk_idx"].long(), 1).view(B, -1, E)
    counts = (picks * keep).sum(1, dtype=torch.int32)
    n = keep.sum(1).clamp(min=1).float()  # [B, 1]
    mean_p = ((p * keep).sum(1, dtype=torch.float64) / n).float()
    loss = (counts.float() * mean_p).sum(1) * (E / k) / n[:, 0]
    zloss = ((lse * lse * keep).sum((1, 2), dtype=torch.float64) / n[:, 0]).float()
    c = counts.float()[:, None] * ((E / k) * st["dloss"][:, None] / (n * n))[:, None]
    grad = p * (c - (p * c).sum(2, keepdim=True)) + (2 * st["dz"][:, None] / n)[:, None] * lse * p
    return {"counts": counts, "mean_p": mean_p, "loss": loss, "zloss": zloss,
            "dlogits": st["dlogits_in"] + torch.where(keep, grad, 0.0).view(T, E)}


def _plain_xent(st):
    T, target = st["T"], st["target"]
    x, W = st["x"].float(), st["W"].float()
    z = x @ W.t()
    m = z.amax(1, keepdim=True)
    use = target >= 0
    at = target.clamp(min=0)[:, None]
    zt = z.gather(1, at)
    e = z.sub_(m).exp_()
    s = e.sum(1, keepdim=True)
    loss = torch.where(use, ((m - zt) + torch.log(s))[:, 0], 0.0)
    lse = (m + torch.log(s))[:, 0]
    out = {"loss": loss, "lse": lse}
    if st["grad"]:
        g = torch.where(use, st["dloss"], 0.0)
        h = 2 * st["z"] * st["dloss"] * lse
        D = e.mul_(((g + h) / s[:, 0])[:, None])
        D.scatter_add_(1, at, -g[:, None])
        out["dx"] = (D @ W).to(st["dx"].dtype)
        out["dW"] = (D.t() @ x).to(st["dW"].dtype)
    return out


def _plain_ortho(st):
    a, b, c = COEF
    X = st["G"].float()
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    tall = st["rows"] > st["cols"]
    if tall:
        X = X.transpose(1, 2)
    for _ in range(STEPS):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return {"O": (X.transpose(1, 2) if tall else X).bfloat16().contiguous()}


def _plain(st):
    return {"balance": _plain_balance, "xent": _plain_xent, "orthogonalize": _plain_ortho}[st["op"]](st)


# -------------------------------------------------------- the library's calls
def _own(st):
    from combine_fp32_softmax_gb300 import moe
    op = st["op"]
    if op == "balance":
        if "ws" not in st:  # the layer's workspace; its widths do not matter here
            st["cfg"] = moe.moe_cfg(st["T"], 64, 64, st["E"], st["k"], 0, 0)
            st["ws"] = moe.alloc_workspace(st["cfg"])
            B, E = st["B"], st["E"]
            st["counts"] = torch.empty(B, E, dtype=torch.int32, device=DEV)
            st["mean_p"] = torch.empty(B, E, device=DEV)
            st["loss"], st["zloss"] = torch.empty(B, device=DEV), torch.empty(B, device=DEV)
            st["dlogits"] = torch.empty(st["T"], E, device=DEV)
        moe.moe_balance_fwd(st["cfg"], st["logits"], st["topk_idx"], st["mask"], st["counts"], st["mean_p"], st["loss"],
                            st["zloss"], st["ws"])
        moe.moe_balance_bwd(st["cfg"], st["logits"], st["counts"], st["mask"], st["dloss"], st["dz"], st["dlogits_in"],
                            st["dlogits"], st["ws"])
        return {n: st[n] for n in ("counts", "mean_p", "loss", "zloss", "dlogits")}
    if op == "xent":
        if "ws" not in st:
            st["ws"] = moe.alloc_xent_workspace(st["T"], st["V"], st["d"], backward=bool(st["grad"]))
        moe.moe_xent_fwd(st["x"], st["W"], st["target"], st["loss"], st["lse"], st["ws"])
        if not st["grad"]:
            return {"loss": st["loss"], "lse": st["lse"]}
        dlse = (2 * st["z"]) * st["dloss"] * st["lse"] if st["z"] else None
        moe.moe_xent_bwd(st["x"], st["W"], st["target"], st["loss"], st["lse"], st["dloss"], dlse, st["dx"], st["dW"],
                         st["ws"])
        return {n: st[n] for n in ("loss", "lse", "dx", "dW")}
    if "ws" not in st:
        st["ws"] = moe.alloc_orthogonalize_workspace(st["mats"], st["rows"], st["cols"])
    moe.moe_orthogonalize(st["G"], st["O"], STEPS, st["ws"])
    return {"O": st["O"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ what it takes
def work(case):
    if case["op"] == "balance":
        T, E, k, B = (case[n] for n in ("T", "E", "k", "B"))
        # logits, picks, mask and the layer's gradient in, gradient out; counts and probabilities once
        return {"bytes": T * (E * 12 + k * 4 + (1 if case["masked"] else 0)) + B * (E * 8 + 16), "flops": 12 * T * E}
    if case["op"] == "xent":
        T, V, d = case["T"], case["V"], case["d"]
        b, f = (V + T) * d * 2 + T * 16, 2 * T * V * d
        if case["grad"]:  # the products for x and W; the logits' product counts once
            return {"bytes": b + T * 4 + (V + T) * d * (4 if case["grad"] == "fp32" else 2), "flops": 3 * f}
        return {"bytes": b, "flops": f}
    M, r, c = case["mats"], case["rows"], case["cols"]
    m, n = min(r, c), max(r, c)
    # X X^T and A A are symmetric: half of each
    return {"bytes": M * r * c * ((4 if case["src"] == "fp32" else 2) + 2),
            "flops": (M - case["empty"]) * STEPS * (m * m * n + m * m * m + 2 * m * m * n)}


# --------------------------------------------------------------- in 64 bits
def _exact_balance(st):
    T, E, k, B = st["T"], st["E"], st["k"], st["B"]
    L = T // B
    out = {"counts": torch.zeros(B, E, dtype=torch.int32, device=DEV),
           "mean_p": torch.zeros(B, E, dtype=torch.float64, device=DEV),
           "loss": torch.zeros(B, dtype=torch.float64, device=DEV),
           "zloss": torch.zeros(B, dtype=torch.float64, device=DEV),
           "dlogits": st["dlogits_in"].double()}
    for b in range(B):
        rows = torch.arange(b * L, (b + 1) * L, device=DEV)
        if st["mask"] is not None:
            rows = rows[st["mask"][rows]]
        n = len(rows)
        if n == 0:
            continue
        z = st["logits"][rows].double()
        p, lse = torch.softmax(z, 1), torch.logsumexp(z, 1)
        cnt = torch.bincount(st["topk_idx"][rows].long().reshape(-1), minlength=E)
        P = p.mean(0)
        share = cnt.double() * E / (k * n)
        out["counts"][b], out["mean_p"][b] = cnt.int(), P
        out["loss"][b], out["zloss"][b] = share @ P, lse.square().mean()
        gp = st["dloss"][b].double() * share / n  # for each probability
        out["dlogits"][rows] += p * (gp - (p @ gp)[:, None]) + (2 * st["dz"][b].double() / n) * lse[:, None] * p
    return out


def _exact_xent(st):
    T, V = st["T"], st["V"]
    x = st["x"].double()
    out = {"loss": torch.zeros(T, dtype=torch.float64, device=DEV), "lse": torch.zeros(T, dtype=torch.float64, device=DEV)}
    W = st["W"].double()
    if st["grad"]:
        out["dx"], out["dW"] = torch.zeros_like(x), torch.zeros_like(W)
    for t in range(0, T, 1024):
        xs, target = x[t:t + 1024], st["target"][t:t + 1024]
        z = xs @ W.t()
        lse = torch.logsumexp(z, 1)
        out["lse"][t:t + 1024] = lse
        rows = (target >= 0).nonzero()[:, 0]
        z -= lse[:, None]
        out["loss"][t + rows] = -z[rows, target[rows]]
        if st["grad"]:
            g = st["dloss"][t:t + 1024].double()
            D = z.exp_().mul_((torch.where(target >= 0, g, 0.0) + 2 * st["z"] * g * lse)[:, None])
            D[rows, target[rows]] -= g[rows]
            out["dx"][t:t + 1024] = D @ W
            out["dW"] += D.t() @ xs
    return out


def _exact_ortho(st):
    out = torch.zeros(st["mats"], st["rows"], st["cols"], dtype=torch.float64, device=DEV)
    eye = torch.eye(min(st["rows"], st["cols"]), dtype=torch.float64, device=DEV)
    for i in range(st["mats"]):
        X = st["G"][i].double()
        X = X / (torch.linalg.vector_norm(X) + EPS)
        for _ in range(STEPS):
            if st["rows"] <= st["cols"]:
                A = X @ X.t()
                X = (COEF[0] * eye + A @ (COEF[1] * eye + COEF[2] * A)) @ X
            else:
                A = X.t() @ X
                X = X @ (COEF[0] * eye + A @ (COEF[1] * eye + COEF[2] * A))
        out[i] = X
    return {"O": out}


def exact(case, seed):
    st = prepare(case, seed)
    return {"balance": _exact_balance, "xent": _exact_xent, "orthogonalize": _exact_ortho}[case["op"]](st)
