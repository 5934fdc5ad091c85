"""The layer for a few tokens at its edges: infinite weights, tiles drawn from a counter, one workspace for several
token counts, sums of one sign, waits that run out."""
import time

import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300 import moe
from combine_fp32_softmax_gb300.configs import MoEConfig
from combine_fp32_softmax_gb300.inputs import make_layer_inputs
from oracle import moe_oracle as O
from oracle import q4_oracle as Q
from tests.gpu_util import DEV, np64, relf
from tests.test_gpu_decode import BF16, F32, Layer, check_y, device_error

pytestmark = pytest.mark.gpu

INF = float("inf")


def check_with_infinities(got, ref):
    """The same infinities and NaN as the reference, and its other elements within check_y's bound."""
    g = np64(got)
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    for sign in (1, -1):
        assert np.array_equal(g == sign * np.inf, ref == sign * np.inf)
    ok = np.isfinite(ref)
    check_y("finite part", got[torch.from_numpy(ok).to(got.device)], ref[ok])


# ----------------------------------------------------- infinite weights in W2
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 40])
def test_infinite_weights_of_picked_experts(T, dtype):
    """y is what the formula gives: an infinity of the product's sign, NaN only where two of them meet."""
    cfg = MoEConfig("inf", T, 320, 640, 4, 2, S=1)
    layer = Layer(cfg)
    W2 = layer.host["W2"]
    W2[:, 3, 17] = INF           # in every expert: the sign is that of each token's h
    W2[4, 200, 600] = -INF       # in the shared expert, whose last columns come in another run of sums
    W2[4, 319, 0], W2[4, 319, 639] = INF, INF
    layer.dev[2] = W2.to(DEV)
    y, _, _, ws = layer.run(dtype)
    assert device_error(ws) == (0, 0)
    ref = layer.reference().y
    assert np.isinf(ref).any()
    check_with_infinities(y, ref)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_weights_meet_hidden_values_that_bf16_holds(dtype):
    """h = 2 and -4 exactly, so that the lower parts of h are 0."""
    cfg = MoEConfig("exact", 3, 64, 64, 2, 1, renorm=1)
    layer = Layer(cfg, logits=torch.tensor([[1.0, 0.0], [0.0, 1.0], [1.0, 0.0]]))
    x = torch.zeros(3, 64)
    x[:, 0] = 1.0
    W1, W3, W2 = torch.zeros(2, 64, 64), torch.zeros(2, 64, 64), torch.ones(2, 64, 64)
    W1[:, :, 0] = 128.0                                  # silu(128) = 128 in fp32
    W3[0, :, 0], W3[1, :, 0] = 1 / 64, -1 / 32
    W2[:, 5, 9], W2[:, 6, 33] = INF, -INF
    W2[:, 7, 1], W2[:, 7, 2] = INF, -INF                 # NaN
    layer.x = x.to(BF16)
    layer.host = dict(zip(("W1", "W3", "W2"), (w.to(BF16) for w in (W1, W3, W2))))
    layer.dev = [layer.host[n].to(DEV) for n in ("W1", "W3", "W2")]
    y, _, _, ws = layer.run(dtype)
    assert device_error(ws) == (0, 0)
    got = y.float().cpu()
    assert got[:, 5].tolist() == [INF, -INF, INF] and got[:, 6].tolist() == [-INF, INF, -INF]
    assert torch.isnan(got[:, 7]).all()
    assert got[:, 0].tolist() == [128.0, -256.0, 128.0]


# --------------------------------------------- one workspace, several counts
@pytest.mark.parametrize("group", [0, 64])
def test_a_workspace_for_64_tokens_serves_any_count(group):
    full = Layer(MoEConfig("batch", 64, 256, 320, 8, 2, S=1), group=group)
    ws = full.workspace()
    x, z = full.x.to(DEV), full.logits.to(DEV)
    for T in (64, 1, 21, 20, 7, 64, 33):
        part = Layer.__new__(Layer)
        part.cfg, part.group, part.dev = full.cfg.with_(T=T), group, full.dev
        got = part.run(ws=ws, x=x, logits=z)          # x and logits with more rows than T
        assert device_error(ws) == (0, 0)
        want = part.run(x=x[:T].clone(), logits=z[:T].clone())
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a, b), T


# ------------------------------------------------------------ fp32 precision
# The tensor core cuts its running sum of positive terms off below 2^-23 of it, once for each 16 columns.  Sums restart
# after at most 16 instructions (4 bits: with every group, 8 at most), so that 16 2^-23 = 2^-19 of a sum of positive terms
# is lost at most; the sums of those runs and groups are added rounded to nearest, 2^-24 each, K / 32 of them at most.
def cut(K):
    return 2.0 ** -19 + -(-K // 32) * 2.0 ** -24


@pytest.mark.parametrize("T,n,K", [(1, 4096, 4096), (9, 257, 14336), (64, 2048, 4096)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_fp32_linear_sums_of_one_sign(T, n, K, group):
    g = torch.Generator(device=DEV).manual_seed(T + K)
    x = torch.randn(T, K, generator=g, device=DEV).abs().to(BF16)
    W = torch.randn(n, K, generator=g, device=DEV).abs().to(BF16)
    y, ws = torch.empty(T, n, device=DEV), moe.alloc_linear_workspace(T, n, K)
    if group:
        codes, scales = moe.q4_empty(1, n, K, group)
        moe.moe_q4_quantize(W, codes, scales, group)
        moe.moe_linear_q4_fwd(x, codes, scales, group, y, ws)
        W = torch.from_numpy(Q.values(codes, scales, group)[0]).to(DEV)
    else:
        moe.moe_linear_fwd(x, W, y, ws)
    assert device_error(ws) == (0, 0)
    ref = x.double() @ W.double().T
    assert ((y.double() - ref).abs() / ref).max().item() <= cut(K)


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T", [1, 33])
def test_fp32_layer_sums_of_one_sign(T, group):
    """x, W1, W3, W2 >= 0: a relative error of a comes through silu at most 1.28 times, b's and h's once; 16 roundings
    for silu, the gate's weight and the sum over the slots."""
    cfg = MoEConfig("positive", T, 1024, 1408, 5, 2, S=1, renorm=1)
    inp = make_layer_inputs(cfg, 3)
    layer = Layer(cfg, 3, group=group)
    W = {n: getattr(inp, n).abs() for n in ("W1", "W3", "W2")}
    layer.x = inp.x.abs()
    if group:
        q = {n: Q.quantize(w, group) for n, w in W.items()}
        layer.dev = [t.to(DEV) for n in W for t in q[n]]
        W = {n: Q.values(*q[n], group) for n in W}
    else:
        layer.dev = [W[n].to(DEV) for n in W]
    layer.host = W
    y, _, _, ws = layer.run(F32)
    assert device_error(ws) == (0, 0)
    ref = layer.reference().y
    assert (ref > 0).all()
    assert (np.abs(np64(y) - ref) / ref).max() <= 2.28 * cut(1024) + cut(1408) + 16 * 2.0 ** -24


def layer_with_16_bit_hidden_values(layer):
    """The layer in fp64 but for h, which is the sum of two bf16 values."""
    c, x, out = layer.cfg, O.f64(layer.x), np.zeros((layer.cfg.T, layer.cfg.d))
    W1, W3, W2 = (O.f64(layer.host[n]) for n in ("W1", "W3", "W2"))
    r = O.route(layer.logits, c.k, c.renorm)
    for t in range(c.T):
        for j in range(c.k + c.S):
            e, w = (r.sel[t, j], r.w[t, j]) if j < c.k else (c.E + j - c.k, 1.0)
            a = W1[e] @ x[t]
            h = torch.from_numpy(w * a / (1 + np.exp(-a)) * (W3[e] @ x[t]))
            high = h.to(BF16).double()
            out[t] += W2[e] @ (high + (h - high).to(BF16).double()).numpy()
    return out


@pytest.mark.parametrize("T", [1, 9, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_fp32_q4_layer_keeps_24_bits_of_the_hidden_values(T, group):
    """Errors of random sign, relative to y's norm.  A group's sum loses at most half of 8 2^-23 on average, half of that
    again as the sum grows: 2.4e-7 for a, b and y each, and a few roundings of 2^-24: below 1.5e-6 together.  An h of
    16 bits would be off by 2e-6 and more."""
    layer = Layer(MoEConfig("three_parts", T, 512, 768, 5, 2, S=1), group=group)
    y, _, _, ws = layer.run(F32)
    assert device_error(ws) == (0, 0)
    ref = layer.reference().y
    assert relf(layer_with_16_bit_hidden_values(layer), ref) > 1.6e-6
    assert relf(np64(y), ref) <= 1.5e-6


@pytest.mark.parametrize("T,n,K", [(1, 2048, 65536), (64, 512, 16384)])
def test_bf16_linear_sums_of_one_sign_over_many_columns(T, n, K):
    """A bf16 y: the tensor core's sum runs over all of K and loses at most 2^-23 for each 16 columns; then y's own
    rounding, 2^-8 at most."""
    g = torch.Generator(device=DEV).manual_seed(K)
    x = torch.randn(T, K, generator=g, device=DEV).abs().to(BF16)
    W = torch.randn(n, K, generator=g, device=DEV).abs().to(BF16)
    y, ws = torch.empty(T, n, dtype=BF16, device=DEV), moe.alloc_linear_workspace(T, n, K)
    moe.moe_linear_fwd(x, W, y, ws)
    assert device_error(ws) == (0, 0)
    ref = x.double() @ W.double().T
    err = (y.double() - ref) / ref
    assert err.abs().max().item() <= 2.0 ** -8 + K / 16 * 2.0 ** -23
    assert abs(err.mean().item()) <= K / 16 * 2.0 ** -23 + 2.0 ** -8 / (T * n) ** 0.5


# --------------------------------------------- tiles drawn from a counter
def matrix(W, scales, e, group):
    """fp64 values of matrix e of device weights."""
    if not group:
        return W[e].double()
    word, q = W[e].view(torch.int32), torch.empty(W.shape[1], 2 * W.shape[2], dtype=torch.float64, device=DEV)
    for i, c in enumerate(Q.NIBBLE_COLUMN):
        q[:, c::8] = ((word >> (4 * i)) & 15).double() - 8
    return q * scales[e, :, :W.shape[1]].double().T.repeat_interleave(group, 1)


def drawn_layer(group):
    """The layer on the GPU, and its weights with their scales."""
    T, d = (16, 1792) if group else (64, 1536)
    cfg = MoEConfig("drawn", T, d, 1408, 32, 4, S=2)
    g = torch.Generator(device=DEV).manual_seed(d)
    W = [(torch.randn(34, *s, generator=g, device=DEV) * s[1] ** -0.5).to(BF16)
         for s in ((1408, d), (1408, d), (d, 1408))]
    z = torch.randn(T, 32, generator=g, device=DEV)
    for t in range(T):                                    # every expert has as many tokens
        z[t, (4 * t + torch.arange(4, device=DEV)) % 32] += 20
    layer = Layer.__new__(Layer)
    layer.cfg, layer.group, layer.logits = cfg, group, z
    layer.x = torch.randn(T, d, generator=g, device=DEV).to(BF16)
    if group:
        layer.dev = []
        for w in W:
            q = moe.q4_empty(*w.shape, group)
            moe.moe_q4_quantize(w, *q, group)
            layer.dev += q
        pairs = list(zip(layer.dev[::2], layer.dev[1::2]))
    else:
        layer.dev, pairs = W, [(w, None) for w in W]
    return layer, pairs


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [0, 64, 128])
def test_whole_tiles_drawn_by_the_CTAs(group, dtype):
    """More than one turn of whole tiles for 152 SMs in either product: 374 tiles of 24 K blocks and 204 of 22 (bf16),
    374 of 7 and 238 of 6 (4 bits).  Who draws what differs from call to call and from grid to grid; the bits do not."""
    layer, pairs = drawn_layer(group)
    T, d, z = layer.cfg.T, layer.cfg.d, layer.logits
    ws, out = layer.workspace(), layer.outputs(dtype)
    want = [t.clone() for t in layer.run(dtype, ws=ws, out=out)[:3]]
    r = O.route(z.cpu(), 4)
    assert np.array_equal(want[1].cpu().numpy(), r.sel)
    ref, x = torch.zeros(T, d, dtype=torch.float64, device=DEV), layer.x.double()
    for e in range(34):
        token, slot = np.nonzero(r.sel == e) if e < 32 else (np.arange(T), None)
        w = torch.from_numpy(r.w[token, slot] if e < 32 else np.ones(T)).to(DEV)[:, None]
        token = torch.from_numpy(token).to(DEV)
        a, b = (x[token] @ matrix(*pairs[i], e, group).T for i in (0, 1))
        ref.index_add_(0, token, w * a * torch.sigmoid(a) * b @ matrix(*pairs[2], e, group).T)
    check_y("y", want[0], ref.cpu().numpy())
    trash = torch.empty(1 << 26, device=DEV)
    try:
        for limit in (0, 1, 37, 151, 0):
            moe.moe_set_grid_limit(limit)
            for _ in range(20 if limit != 1 else 1):
                out[0].fill_(float("nan"))
                trash.zero_()                             # weights from memory
                layer.run(dtype, ws=ws, out=out)
                for a, b in zip(out, want):
                    assert torch.equal(a, b), limit
            assert device_error(ws) == (0, 0)
    finally:
        moe.moe_set_grid_limit(0)
    for _ in range(200):
        layer.run(dtype, ws=ws, out=out)
    assert device_error(ws) == (0, 0)
    for a, b in zip(out, want):
        assert torch.equal(a, b)


# ------------------------------------------------------- waits that run out
ROUTED, PARTS, MEETING_1, MEETING_2 = 1, 2, 3, 4


def gives_up(drop, ws, call):
    """A call that waits for a count which never comes ends within seconds, with the error set."""
    begin = time.monotonic()
    try:
        moe.moe_debug_drop_decode_count(drop)
        call()
        code, info = device_error(ws)
    finally:
        moe.moe_debug_drop_decode_count(0)
    assert code == moe.MOE_ERR_TIMEOUT, (code, info)
    assert 0.5 < time.monotonic() - begin < 20
    return info >> 24


# tiles of the second product cut, and of the first
GIVE_UP = [MoEConfig("cut_out", 30, 64, 1408, 4, 2), MoEConfig("cut_hidden", 30, 2048, 64, 4, 2)]


@pytest.mark.parametrize("cfg", GIVE_UP, ids=lambda c: c.name)
@pytest.mark.parametrize("drop", [ROUTED, PARTS, MEETING_1, MEETING_2])
@pytest.mark.parametrize("group,dtype", [(0, F32), (0, BF16), (64, F32)])
def test_a_layer_call_whose_wait_runs_out_ends_with_an_error(cfg, drop, group, dtype):
    layer = Layer(cfg, group=group)
    ws, out = layer.workspace(), layer.outputs(dtype)
    want = [t.clone() for t in layer.run(dtype, ws=ws, out=out)[:3]]
    site = gives_up(drop, ws, lambda: layer.run(dtype, ws=ws, out=out))
    if drop == ROUTED:
        assert site == 0x20
    moe.moe_decode_ws_init(cfg, ws)
    layer.run(dtype, ws=ws, out=out)
    assert device_error(ws) == (0, 0)
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("group", [0, 128])
def test_a_linear_call_whose_wait_runs_out_ends_with_an_error(group):
    g = torch.Generator().manual_seed(9)
    x, W = torch.randn(30, 4096, generator=g).to(BF16).to(DEV), torch.randn(300, 4096, generator=g).to(BF16).to(DEV)
    q = moe.q4_empty(1, 300, 4096, 128)
    moe.moe_q4_quantize(W, *q, 128)
    y, ws = torch.empty(30, 300, device=DEV), moe.alloc_linear_workspace(30, 300, 4096)

    def call():
        if group:
            moe.moe_linear_q4_fwd(x, *q, group, y, ws)
        else:
            moe.moe_linear_fwd(x, W, y, ws)
    call()
    want = y.clone()
    assert gives_up(PARTS, ws, call) == 0x29
    moe.moe_linear_ws_init(30, 300, 4096, ws)
    call()
    assert device_error(ws) == (0, 0) and torch.equal(y, want)


@pytest.mark.parametrize("drop", [MEETING_1, MEETING_2])
@pytest.mark.parametrize("group", [0, 64])
def test_calls_with_drawn_tiles_whose_wait_runs_out_end_with_an_error(group, drop):
    """After the first product the producers are ahead, in the second one's tiles."""
    layer, _ = drawn_layer(group)
    ws, out = layer.workspace(), layer.outputs(BF16)
    want = [t.clone() for t in layer.run(BF16, ws=ws, out=out)[:3]]
    gives_up(drop, ws, lambda: layer.run(BF16, ws=ws, out=out))
    moe.moe_decode_ws_init(layer.cfg, ws)
    layer.run(BF16, ws=ws, out=out)
    assert device_error(ws) == (0, 0)
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_counts_that_nobody_waits_for_change_nothing():
    layer = Layer(MoEConfig("few", 20, 256, 320, 8, 2, S=1))   # routed by every CTA itself
    want = layer.run(F32)
    try:
        moe.moe_debug_drop_decode_count(ROUTED)
        got = layer.run(F32)
    finally:
        moe.moe_debug_drop_decode_count(0)
    assert device_error(got[3]) == (0, 0)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    with pytest.raises(moe.MoeError):
        moe.moe_debug_drop_decode_count(5)
