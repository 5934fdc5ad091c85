"""The layer for a few tokens and its 4-bit weights: cases, inputs, plain forms and the library's calls.

Five operators, named by a case's "op":
  decode      a whole MoE layer for T <= 64 tokens: softmax top-k of the logits, SwiGLU experts, shared experts, weighted sum
  decode_q4   the same with 4-bit expert weights and one bf16 scale per group of `group` weights along the summed dimension
  linear      y = x W^T for T <= 64 rows of x, bf16 W [n, K]
  linear_q4   the same with 4-bit weights and group scales
  quantize    bf16 matrices to 4 bits and group scales, and back to the bf16 values they stand for

The 4-bit format: W[r, c] = s[c // group, r] * (q[r, c] - 8) with q in 0..15.  Eight columns 8j..8j+7 of a row share four bytes,
columns 0, 2, 4, 6 in the nibbles of the first two (low nibble first) and 1, 3, 5, 7 in the last two.  Scales are [K / group, n],
the rows padded to a multiple of 8.  Quantizing: s = bf16(absmax / 7) of the group, q = 8 + rint(w / s) held to -8..7 (8 where s = 0).
"""
import math

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------- cases
def _decode(name, T, d, f, E, k, S=0, renorm=0, zipf=False, y="bf16", group=0):
    c = dict(op="decode_q4" if group else "decode", T=T, d=d, f=f, E=E, k=k, S=S, renorm=renorm, zipf=zipf, y=y)
    if group:
        c["group"] = group
    if name:
        c["name"] = name
    return c


def _linear(name, T, n, K, y="bf16", group=0):
    c = dict(op="linear_q4" if group else "linear", T=T, n=n, K=K, y=y)
    if group:
        c["group"] = group
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a small layer with a ragged expert width and a shared expert, seven sequences, fp32 sums kept for the caller
        _decode("decode_T7_d256_f320", 7, 256, 320, 6, 2, S=1, renorm=1, y="fp32"),
        # one sequence answering: every token reads its 6 + 2 experts of the DeepSeek-V2-Lite-like layer
        _decode("decode_T1_dsv2lite", 1, 2048, 1408, 64, 6, S=2),
        # a full batch of the same layer: nearly every expert is read for a handful of tokens
        _decode("decode_T64_dsv2lite", 64, 2048, 1408, 64, 6, S=2),
        # the same layers with 4-bit experts: one sequence
        _decode("decode_q4_T1_dsv2lite", 1, 2048, 1408, 64, 6, S=2, group=128),
        # sixteen sequences on the Mixtral-like layer: eight large experts, all read
        _decode("decode_q4_T16_mixtral", 16, 4096, 14336, 8, 2, renorm=1, group=64),
        # heavy-tailed routing: some experts get every token, most of the 128 get none
        _decode("decode_q4_T33_skewed", 33, 4096, 2048, 128, 8, zipf=True, group=32),
        # the gate projection that makes the layer's logits for one token: latency alone
        _linear("linear_T1_gate64", 1, 64, 2048, y="fp32"),
        # a square projection beside the experts for a batch, an odd number of rows and outputs
        _linear("linear_T37_n4097", 37, 4097, 4096),
        # the wide projection of a dense layer for one token
        _linear("linear_q4_T1_n14336", 1, 14336, 4096, group=128),
        # the way back for an odd batch with fine groups
        _linear("linear_q4_T19_K14336", 19, 4096, 14336, y="fp32", group=32),
        # one expert's projection brought to 4 bits
        dict(name="quantize_1408x2048", op="quantize", mats=1, rows=1408, cols=2048, group=128),
        # every gate projection of a layer at load time
        dict(name="quantize_66x1408x2048", op="quantize", mats=66, rows=1408, cols=2048, group=64),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["decode", "decode_q4", "linear", "linear_q4", "quantize"])
    group = rng.choice([32, 64, 128]) if op in ("decode_q4", "linear_q4", "quantize") else 0
    step = max(64, group)
    T = _log(rng, 1, 64)
    y = rng.choice(["bf16", "bf16", "fp32"])
    if op == "quantize":
        return dict(op=op, mats=_log(rng, 1, 40), rows=_log(rng, 8, 2500), cols=step * _log(rng, 1, 2048 // step), group=group)
    if op.startswith("linear"):
        return _linear(None, T, _log(rng, 8, 16000), step * _log(rng, 2, 8192 // step), y, group)
    d = step * _log(rng, 1, 4096 // step)
    f = step * _log(rng, 1, 4096 // step)
    E = _log(rng, 2, 128)
    while (E + 4) * d * f > 66 * 2048 * 1408:  # no more weights than the DeepSeek-V2-Lite-like layer has
        E = max(2, E // 2)
        if E == 2:
            f = max(step, f // 2 // step * step)
    return _decode(None, T, d, f, E, rng.randint(1, min(E, 8)), rng.choice([0, 0, 1, 2, 4]), rng.randint(0, 1),
                   rng.random() < 0.25, y, group)


# ----------------------------------------------------------------- inputs
def _gen(seed, n):
    return torch.Generator(device=DEV).manual_seed(seed * 1009 + n)


def _bf16(shape, g, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def _pad8(n):
    return (n + 7) // 8 * 8


def _pack(w, group):
    """bf16 [M, n, K] -> codes uint8 [M, n, K/2], scales bf16 [M, K/group, pad8(n)]."""
    M, n, K = w.shape
    wg = w.view(M, n, K // group, group).float()
    s = (wg.abs().amax(-1) / 7.0).bfloat16()
    sf = s.float()[..., None]
    q = torch.where(sf > 0, (wg / sf).round().clamp(-8, 7), torch.zeros((), device=w.device)).to(torch.int8).view(M, n, K) + 8
    q = q.to(torch.uint8).view(M, n, K // 8, 8)
    codes = torch.stack([q[..., 0] | q[..., 2] << 4, q[..., 4] | q[..., 6] << 4,
                         q[..., 1] | q[..., 3] << 4, q[..., 5] | q[..., 7] << 4], -1).view(M, n, K // 2)
    scales = torch.zeros(M, K // group, _pad8(n), dtype=torch.bfloat16, device=w.device)
    scales[:, :, :n] = s.transpose(1, 2)
    return codes, scales


def _unpack(codes, scales, n, group):
    """The fp32 values that codes and scales stand for, [M, n, K]."""
    M, _, half = codes.shape
    b = codes.view(M, n, half // 4, 4)
    lo, hi = b & 15, b >> 4
    q = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1], hi[..., 3]], -1)
    q = q.view(M, n, 2 * half // group, group).float() - 8.0
    return (q * scales[:, :, :n].transpose(1, 2).float()[..., None]).view(M, n, 2 * half)


def _weights(st, name, shape, seed, group):
    w = _bf16(shape, seed, 0.02)
    if not group:
        st[name] = w
        return
    parts = [_pack(m[None], group) for m in w]  # matrix by matrix: the fp32 copies stay small
    st[name] = torch.cat([p[0] for p in parts])
    st[name + "s"] = torch.cat([p[1] for p in parts])


def prepare(case, seed):
    st = dict(case)
    group = case.get("group", 0)
    if case["op"] == "quantize":
        M, n, K = case["mats"], case["rows"], case["cols"]
        st["W"] = _bf16((M, n, K), _gen(seed, 1), 0.02)
        st["codes"] = torch.empty(M, n, K // 2, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty(M, K // group, _pad8(n), dtype=torch.bfloat16, device=DEV)
        st["back"] = torch.empty_like(st["W"])
        return st
    T = case["T"]
    ydt = torch.bfloat16 if case["y"] == "bf16" else torch.float32
    if case["op"].startswith("linear"):
        st["x"] = _bf16((T, case["K"]), _gen(seed, 1))
        _weights(st, "W", (1, case["n"], case["K"]), _gen(seed, 2), group)
        st["out"] = torch.empty(T, case["n"], dtype=ydt, device=DEV)
        return st
    d, f, E, N = case["d"], case["f"], case["E"], case["E"] + case["S"]
    st["x"] = _bf16((T, d), _gen(seed, 1))
    st["logits"] = torch.randn(T, E, device=DEV, generator=_gen(seed, 2)) + _bias(case, DEV)
    _weights(st, "W1", (N, f, d), _gen(seed, 3), group)
    _weights(st, "W3", (N, f, d), _gen(seed, 4), group)
    _weights(st, "W2", (N, d, f), _gen(seed, 5), group)
    st["out"] = torch.empty(T, d, dtype=ydt, device=DEV)
    st["idx"] = torch.empty(T, case["k"], dtype=torch.int32, device=DEV)
    st["w"] = torch.empty(T, case["k"], dtype=torch.float32, device=DEV)
    return st


def _bias(case, device):
    """Heavy-tailed load: two times the log of a Zipf(1.2) weight for each expert."""
    r = torch.arange(1, case["E"] + 1, dtype=torch.float32, device=device)
    return -2.4 * r.log() if case["zipf"] else torch.zeros_like(r)


# ------------------------------------------------------------- plain form
def _plain_route(z, k, renorm):
    idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]  # ties keep the lower index
    e = torch.exp(z - z.amax(1, keepdim=True))
    w = (e / e.sum(1, keepdim=True)).gather(1, idx)
    return idx, w / w.sum(1, keepdim=True) if renorm else w


def _plain_values(st, name, experts=None):
    """fp32 weights of the given experts (all of them by default)."""
    pick = (lambda t: t) if experts is None else (lambda t: t.index_select(0, experts))
    if "group" not in st:
        return pick(st[name]).float()
    return _unpack(pick(st[name]), pick(st[name + "s"]), st[name].shape[1], st["group"])


def _plain_decode(st):
    T, k, E, S = st["T"], st["k"], st["E"], st["S"]
    x = st["x"].float()
    idx, w = _plain_route(st["logits"], k, st["renorm"])
    if T * k <= E:  # fewer picks than experts: one matrix per pick (and per shared expert), the rows of its token
        token = torch.arange(T, device=x.device)
        experts = torch.cat([idx.reshape(-1), torch.arange(E, E + S, device=x.device)])
        mine = torch.cat([token.repeat_interleave(k)[:, None] == token, torch.ones(S, T, dtype=torch.bool, device=x.device)])
        gate = mine * torch.cat([w.reshape(-1), w.new_ones(S)])[:, None]
    else:  # every expert on every token, weight 0 where it was not picked
        experts = None
        gate = torch.cat([w.new_zeros(T, E).scatter_(1, idx, w).t(), w.new_ones(S, T)])
    a = x @ _plain_values(st, "W1", experts).transpose(1, 2)
    b = x @ _plain_values(st, "W3", experts).transpose(1, 2)
    h = a / (1 + torch.exp(-a)) * b * gate[:, :, None]
    y = (h @ _plain_values(st, "W2", experts).transpose(1, 2)).sum(0)
    return {"y": y.to(st["out"].dtype), "topk_idx": idx.int(), "topk_w": w}


def _plain(st):
    if st["op"] == "quantize":
        codes, scales = _pack(st["W"], st["group"])
        return {"values": _unpack(codes, scales, st["rows"], st["group"]).bfloat16(), "scales": scales}
    if st["op"].startswith("linear"):
        return {"y": (st["x"].float() @ _plain_values(st, "W")[0].t()).to(st["out"].dtype)}
    return _plain_decode(st)


# -------------------------------------------------------- the library's calls
def _own(st):
    from combine_fp32_softmax_gb300 import moe
    op = st["op"]
    if op == "quantize":
        moe.moe_q4_quantize(st["W"], st["codes"], st["scales"], st["group"])
        moe.moe_q4_dequantize(st["codes"], st["scales"], st["back"], st["group"])
        return {"values": st["back"], "scales": st["scales"]}
    if op.startswith("linear"):
        if "ws" not in st:  # a program allocates its workspace once
            st["ws"] = moe.alloc_linear_workspace(st["T"], st["n"], st["K"])
        if op == "linear":
            moe.moe_linear_fwd(st["x"], st["W"], st["out"], st["ws"])
        else:
            moe.moe_linear_q4_fwd(st["x"], st["W"], st["Ws"], st["group"], st["out"], st["ws"])
        return {"y": st["out"]}
    if "ws" not in st:
        st["cfg"] = moe.moe_cfg(st["T"], st["d"], st["f"], st["E"], st["k"], st["S"], st["renorm"])
        st["ws"] = moe.alloc_decode_workspace(st["cfg"])
    if op == "decode":
        moe.moe_decode_fwd(st["cfg"], st["logits"], st["x"], st["W1"], st["W3"], st["W2"], st["out"], st["idx"], st["w"], st["ws"])
    else:
        moe.moe_decode_q4_fwd(st["cfg"], st["group"], st["logits"], st["x"], st["W1"], st["W1s"], st["W3"], st["W3s"], st["W2"],
                              st["W2s"], st["out"], st["idx"], st["w"], st["ws"])
    return {"y": st["out"], "topk_idx": st["idx"], "topk_w": st["w"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ what it takes
def _picked(case):
    """Experts that at least one of T tokens picks, on average over routings of the case's distribution."""
    if case["T"] == 1:
        return case["k"]
    g = torch.Generator().manual_seed(7)
    z = torch.randn(32, case["T"], case["E"], generator=g) + _bias(case, "cpu")
    hit = torch.zeros(32, case["E"])
    hit.scatter_(1, z.topk(case["k"], dim=2).indices.view(32, -1), 1.0)
    return float(hit.sum(1).mean())


def work(case):
    group = case.get("group", 0)
    per = 0.5 + 2.0 / group if group else 2.0  # bytes of a weight
    if case["op"] == "quantize":
        n = case["mats"] * case["rows"] * case["cols"]
        return {"bytes": n * (2 + 2 * per + 2), "flops": 4 * n}
    T, ysize = case["T"], 2 if case["y"] == "bf16" else 4
    if case["op"].startswith("linear"):
        n, K = case["n"], case["K"]
        return {"bytes": n * K * per + T * K * 2 + T * n * ysize, "flops": 2 * T * n * K}
    d, f, E, k, S = (case[x] for x in ("d", "f", "E", "k", "S"))
    return {"bytes": (_picked(case) + S) * 3 * d * f * per + T * (E * 4 + d * 2 + d * ysize + k * 8),
            "flops": 6 * d * f * T * (k + S)}


# --------------------------------------------------------------- in 64 bits
def _exact_matrix(st, name, e):
    if "group" not in st:
        return st[name][e].double()
    codes, scales, G = st[name][e], st[name + "s"][e].double(), st["group"]
    n, K = codes.shape[0], 2 * codes.shape[1]
    out = torch.empty(n, K, dtype=torch.float64, device=codes.device)
    for c in range(8):  # column 8j + c: byte (c odd ? 2 : 0) + c // 4 of four, high nibble for c % 4 >= 2
        byte = codes[:, (2 if c % 2 else 0) + c // 4::4].int()
        out[:, c::8] = ((byte >> (4 if c % 4 >= 2 else 0)) % 16 - 8).double()
    for j in range(K // G):
        out[:, j * G:(j + 1) * G] *= scales[j, :n, None]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        W, G = st["W"].double(), case["group"]
        M, n, K = W.shape
        scales = torch.zeros(M, K // G, _pad8(n), dtype=torch.float64, device=DEV)
        values = torch.empty_like(W)
        for j in range(K // G):
            block = W[:, :, j * G:(j + 1) * G]
            s = (block.abs().max(dim=2).values / 7).to(torch.bfloat16).double()
            q = torch.round(block / torch.where(s > 0, s, torch.ones_like(s))[:, :, None]).clamp(-8, 7)
            scales[:, j, :n] = s
            values[:, :, j * G:(j + 1) * G] = q * s[:, :, None]
        return {"values": values, "scales": scales}
    x = st["x"].double()
    if case["op"].startswith("linear"):
        return {"y": x @ _exact_matrix(st, "W", 0).t()}
    T, E, k = case["T"], case["E"], case["k"]
    z = st["logits"].double()
    left, picks = z.clone(), []
    for _ in range(k):  # the largest left, the lowest index among equals
        best = (left == left.max(dim=1, keepdim=True).values).int().argmax(dim=1)
        picks.append(best)
        left[torch.arange(T, device=DEV), best] = -math.inf
    idx = torch.stack(picks, 1)
    p = torch.softmax(z, dim=1)
    w = torch.gather(p, 1, idx)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    y = torch.zeros(T, case["d"], dtype=torch.float64, device=DEV)
    for e in range(E + case["S"]):
        if e < E:
            at = (idx == e).nonzero()
            if len(at) == 0:
                continue
            token, scale = at[:, 0], w[at[:, 0], at[:, 1]]
        else:
            token, scale = torch.arange(T, device=DEV), torch.ones(T, dtype=torch.float64, device=DEV)
        xe = x[token]
        a = xe @ _exact_matrix(st, "W1", e).t()
        b = xe @ _exact_matrix(st, "W3", e).t()
        y.index_add_(0, token, (a * torch.sigmoid(a) * b * scale[:, None]) @ _exact_matrix(st, "W2", e).t())
    return {"y": y, "topk_idx": idx.int(), "topk_w": w}
