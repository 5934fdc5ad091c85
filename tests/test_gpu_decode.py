"""The layer for a few tokens, its linear form and the 4-bit weights on the GPU, against fp64 references.

Tolerances.  bf16 y: half a bf16 step of the reference element, 2^-8 |ref|, plus the fp32 part.  fp32 part of an
element: a sum of K products rounded to fp32 as it grows is off by at most K 2^-23 sum|terms| and, the roundings'
signs being as good as random, by a few times sqrt(K) 2^-23 sum|terms| / sqrt(K) of its rms; 1e-4 of the output's rms
and a relative Frobenius error of 2e-5 hold both that and the layer's 16-bit hidden values (2^-17 relative each)."""
import math

import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300 import moe
from combine_fp32_softmax_gb300.configs import MoEConfig
from combine_fp32_softmax_gb300.inputs import make_layer_inputs
from oracle import moe_oracle as O
from oracle import q4_oracle as Q
from tests.gpu_util import DEV, guarded_empty, np64, relf

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def check_y(name, got, ref):
    rms = float(np.sqrt(np.mean(ref ** 2))) if ref.size else 0.0
    half = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    err = np.abs(np64(got) - ref)
    bound = half * np.abs(ref) + 1e-4 * rms
    assert (err <= bound).all(), f"{name}: {int((err > bound).sum())} of {err.size} beyond, worst {err.max():.3e} " \
                                 f"at rms {rms:.3e}"
    if got.dtype == F32:
        assert relf(np64(got), ref) <= 2e-5, f"{name}: relF {relf(np64(got), ref):.3e}"


def device_error(ws):
    torch.cuda.synchronize()
    return moe.moe_get_device_error(ws)


# ------------------------------------------------------------------- 4 bits
@pytest.mark.parametrize("mats,rows,cols", [(1, 1, 128), (1, 7, 256), (3, 33, 384), (2, 64, 2048), (1, 100, 1408)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_and_back_bit_exact(mats, rows, cols, group):
    g = torch.Generator().manual_seed(rows * cols + group)
    W = (torch.randn(mats, rows, cols, generator=g) * 0.02).to(BF16)
    W[0, 0, :group] = 0                      # a group of zeros: scale 0, codes 8
    W[0, 0, 0] = -0.0
    W[-1, -1, -1] = 40.0                     # an outlier takes its group's scale
    if rows > 4:
        W[0, 3, 0] = float("nan")            # groups with no finite scale come back as NaN
        W[0, 4, 1] = -float("inf")
        W[0, 5, :group] = 1e-39              # a subnormal scale
    codes = guarded_empty((mats, rows, cols // 2), torch.uint8)
    scales = guarded_empty((mats, cols // group, -(-rows // 8) * 8), BF16)
    back = guarded_empty((mats, rows, cols), BF16)
    scales.fill_(float("nan"))
    moe.moe_q4_quantize(W.to(DEV), codes, scales, group)
    want_codes, want_scales = Q.quantize(W, group)
    assert torch.equal(codes.cpu(), want_codes)
    assert torch.equal(scales.cpu().view(torch.int16)[~torch.isnan(want_scales)],
                       want_scales.view(torch.int16)[~torch.isnan(want_scales)])
    assert torch.equal(torch.isnan(scales.cpu()), torch.isnan(want_scales))
    moe.moe_q4_dequantize(codes, scales, back, group)
    want = torch.from_numpy(Q.values(want_codes, want_scales, group)).float().to(BF16)
    assert torch.equal(torch.nan_to_num(back.cpu(), nan=1e9), torch.nan_to_num(want, nan=1e9))


# ------------------------------------------------------------------- linear
def run_linear(x, W, dtype, group=0, ws=None):
    T, (n, K) = x.shape[0], W.shape
    if ws is None:
        ws = guarded_empty((moe.moe_linear_workspace_bytes(T, n, K),), torch.uint8, label="ws")
        moe.moe_linear_ws_init(T, n, K, ws)
    y = guarded_empty((T, n), dtype)
    y.fill_(float("nan"))
    if group:
        codes, scales = Q.quantize(W[None], group)
        moe.moe_linear_q4_fwd(x.to(DEV), codes.to(DEV), scales.to(DEV), group, y, ws)
        ref = Q.values(codes, scales, group)[0]
    else:
        moe.moe_linear_fwd(x.to(DEV), W.to(DEV), y, ws)
        ref = O.f64(W)
    assert device_error(ws) == (0, 0)
    return y, O.f64(x) @ ref.T


LINEAR = [(1, 1, 64), (1, 8, 128), (2, 63, 192), (7, 64, 64), (8, 65, 320), (9, 130, 1408), (16, 200, 256),
          (17, 129, 2048), (31, 1000, 576), (33, 4097, 512), (48, 257, 1024), (64, 640, 704), (64, 64, 4096), (1, 5000, 2048),
          (3, 70, 14336)]


@pytest.mark.parametrize("T,n,K", LINEAR)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_linear_matches_reference(T, n, K, dtype):
    g = torch.Generator().manual_seed(T * n + K)
    y, ref = run_linear(torch.randn(T, K, generator=g).to(BF16), torch.randn(n, K, generator=g).to(BF16), dtype)
    check_y("y", y, ref)


@pytest.mark.parametrize("T,n,K", LINEAR)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_q4_matches_reference(T, n, K, group):
    K = -(-K // max(64, group)) * max(64, group)
    g = torch.Generator().manual_seed(T * n + K + group)
    y, ref = run_linear(torch.randn(T, K, generator=g).to(BF16), torch.randn(n, K, generator=g).to(BF16),
                        F32 if T % 2 else BF16, group)
    check_y("y", y, ref)


@pytest.mark.parametrize("group", [0, 64])
def test_linear_rows_are_independent(group):
    """A row of x with NaN or Inf leaves the other rows' bits alone."""
    g = torch.Generator().manual_seed(5)
    x, W = torch.randn(11, 512, generator=g).to(BF16), torch.randn(96, 512, generator=g).to(BF16)
    clean, _ = run_linear(x, W, F32, group)
    x[4, 17], x[9, 300] = float("nan"), float("inf")
    dirty, _ = run_linear(x, W, F32, group)
    rest = [t for t in range(11) if t not in (4, 9)]
    assert torch.equal(clean[rest], dirty[rest])
    assert torch.isnan(dirty[4]).all() and not torch.isfinite(dirty[9]).any()


# -------------------------------------------------------------------- layer
CFGS = [
    MoEConfig("one", 1, 64, 64, 1, 1),
    MoEConfig("t1", 1, 256, 320, 8, 2, S=1),
    MoEConfig("t2_ek", 2, 128, 192, 4, 4, renorm=1),
    MoEConfig("t5_wide", 5, 512, 704, 16, 6, S=2),
    MoEConfig("t7_mid", 7, 256, 320, 6, 2, S=1, renorm=1),
    MoEConfig("t8_E256_k8_S4", 8, 64, 64, 256, 8, S=4),
    MoEConfig("t9", 9, 192, 448, 10, 3),
    MoEConfig("t33_zipf", 33, 256, 192, 32, 4, zipf=True),
    MoEConfig("t64_skew", 64, 128, 256, 4, 2, S=1, zipf=True),
    MoEConfig("t64_E256", 64, 128, 128, 256, 8, S=4),
    MoEConfig("t1_long", 1, 2048, 1408, 8, 6, S=2),
    MoEConfig("t40_long", 40, 1024, 2816, 3, 1, S=1),
]


class Layer:
    """Host inputs of one layer, device copies (bf16 or 4 bits) and the fp64 result."""

    def __init__(self, cfg, seed=1, group=0, logits=None):
        self.cfg, self.group, inp = cfg, group, make_layer_inputs(cfg, seed)
        self.x, self.logits = inp.x, inp.logits if logits is None else logits
        W = {n: getattr(inp, n) * 4 for n in ("W1", "W3", "W2")}
        if group:
            q = {n: Q.quantize(w, group) for n, w in W.items()}
            self.dev = [t.to(DEV) for n in ("W1", "W3", "W2") for t in q[n]]
            W = {n: Q.values(*q[n], group) for n in q}
        else:
            self.dev = [W[n].to(DEV) for n in ("W1", "W3", "W2")]
        self.host = W

    def reference(self):
        c = self.cfg
        return O.layer_fwd(self.x, self.logits, self.host["W1"], self.host["W3"], self.host["W2"], k=c.k, S=c.S,
                           renorm=c.renorm)

    def outputs(self, dtype):
        c = self.cfg
        y = guarded_empty((c.T, c.d), dtype, label="y")
        y.fill_(float("nan"))
        return y, guarded_empty((c.T, c.k), torch.int32, label="topk_idx"), guarded_empty((c.T, c.k), F32, label="topk_w")

    def workspace(self):
        ws = guarded_empty((moe.moe_decode_workspace_bytes(self.cfg),), torch.uint8, label="ws")
        ws.fill_(0xFF)  # nothing but the initialised words may matter
        moe.moe_decode_ws_init(self.cfg, ws)
        return ws

    def run(self, dtype=F32, ws=None, out=None, x=None, logits=None, stream=None):
        ws = self.workspace() if ws is None else ws
        y, idx, w = self.outputs(dtype) if out is None else out
        x = self.x.to(DEV) if x is None else x
        logits = self.logits.to(DEV) if logits is None else logits
        if self.group:
            moe.moe_decode_q4_fwd(self.cfg, self.group, logits, x, *self.dev, y, idx, w, ws, stream=stream)
        else:
            moe.moe_decode_fwd(self.cfg, logits, x, *self.dev, y, idx, w, ws, stream=stream)
        return y, idx, w, ws


def _check(layer, dtype):
    y, idx, w, ws = layer.run(dtype)
    assert device_error(ws) == (0, 0)
    ref = layer.reference()
    assert np.array_equal(idx.cpu().numpy(), ref.routing.sel)
    np.testing.assert_allclose(np64(w), ref.routing.w, rtol=4e-6)
    check_y("y", y, ref.y)


@pytest.mark.parametrize("cfg", CFGS, ids=lambda c: c.name)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_matches_oracle(cfg, dtype):
    _check(Layer(cfg), dtype)


@pytest.mark.parametrize("cfg", CFGS, ids=lambda c: c.name)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_q4_layer_matches_oracle(cfg, group):
    if group == 128:
        cfg = cfg.with_(d=-(-cfg.d // 128) * 128, f=-(-cfg.f // 128) * 128)
    _check(Layer(cfg, group=group), F32 if group != 64 else BF16)


def test_ties_go_to_the_lower_expert_and_match_the_router():
    cfg = MoEConfig("ties", 16, 128, 128, 12, 3, renorm=1)
    z = torch.randint(-1, 2, (16, 12), generator=torch.Generator().manual_seed(3)).float()
    z[0], z[1, ::2] = 0.0, -0.0
    layer = Layer(cfg, logits=z)
    _check(layer, F32)
    _, idx, w, _ = layer.run()
    ridx, rw = torch.empty_like(idx), torch.empty_like(w)
    moe.moe_route(cfg, z.to(DEV), ridx, rw, moe.alloc_workspace(cfg, DEV))
    assert torch.equal(idx, ridx) and torch.equal(w, rw)


@pytest.mark.parametrize("group", [0, 32])
def test_experts_that_nobody_picked_are_not_used(group):
    cfg = MoEConfig("poison", 3, 128, 192, 16, 2, S=1)
    layer = Layer(cfg, group=group)
    ref = layer.reference()
    unused = sorted(set(range(16)) - set(ref.routing.sel.ravel().tolist()))
    for t in layer.dev:
        if t.dtype == BF16:
            t[unused] = float("nan")
    y, _, _, ws = layer.run()
    assert device_error(ws) == (0, 0)
    check_y("y", y, ref.y)


def test_non_finite_logits_are_reported_and_stay_with_their_token():
    cfg = MoEConfig("nan", 9, 128, 192, 8, 2, S=1)
    layer = Layer(cfg)
    ref = layer.reference()
    layer.logits[5, 3] = float("nan")
    y, idx, w, ws = layer.run()
    assert device_error(ws) == (moe.MOE_ERR_NONFINITE, 5)
    rest = [t for t in range(9) if t != 5]
    assert np.array_equal(idx.cpu().numpy()[rest], ref.routing.sel[rest])
    check_y("y", y[rest], ref.y[rest])
    moe.moe_decode_ws_init(cfg, ws)
    layer.logits[5, 3] = 0.5
    layer.run(ws=ws)
    assert device_error(ws) == (0, 0)


@pytest.mark.parametrize("group", [0, 64])
def test_tokens_with_nan_or_inf_leave_the_others_alone(group):
    cfg = MoEConfig("nanx", 12, 256, 320, 5, 2, S=1)
    layer = Layer(cfg, group=group)
    clean, *_ = layer.run()
    x = layer.x.clone()
    x[2, 7], x[11, 200] = float("nan"), float("inf")
    dirty, _, _, ws = layer.run(x=x.to(DEV))
    assert device_error(ws) == (0, 0)
    rest = [t for t in range(12) if t not in (2, 11)]
    assert torch.equal(clean[rest], dirty[rest])
    assert torch.isnan(dirty[2]).all() and not torch.isfinite(dirty[11]).any()


def test_magnitudes_from_tiny_to_large():
    """Activations whose hidden values span most of bf16's exponents; the gate far into both tails of silu."""
    cfg = MoEConfig("scale", 6, 128, 128, 4, 2)
    layer = Layer(cfg)
    layer.x = (layer.x.float() * torch.tensor([1e-18, 1e-6, 1.0, 60.0, 4e3, 1e9])[:, None]).to(BF16)
    y, _, _, ws = layer.run()
    assert device_error(ws) == (0, 0)
    ref = layer.reference().y
    for t in range(6):  # each token on its own scale
        check_y(f"token {t}", y[t:t + 1], ref[t:t + 1])


@pytest.mark.parametrize("group", [0, 64])
def test_same_bits_every_time_and_for_every_grid(group):
    layer = Layer(MoEConfig("det", 21, 512, 704, 16, 4, S=2), group=group)
    ws = layer.workspace()
    want = layer.run(ws=ws)
    try:
        for limit in (0, 0, 0, 1, 7, 100, 0):
            moe.moe_set_grid_limit(limit)
            got = layer.run(ws=ws)
            assert device_error(ws) == (0, 0)
            for a, b in zip(got[:3], want[:3]):
                assert torch.equal(a, b), limit
    finally:
        moe.moe_set_grid_limit(0)


@pytest.mark.parametrize("cfg", [MoEConfig("few_out", 21, 512, 704, 16, 4, S=2), MoEConfig("one_tile", 2, 64, 1408, 4, 2),
                                 MoEConfig("wide_out", 3, 2048, 64, 8, 2)], ids=lambda c: c.name)
@pytest.mark.parametrize("group", [0, 64])
def test_hundreds_of_calls_in_a_row(cfg, group):
    """Waits whose order varies from call to call: products with fewer ranges than CTAs leave CTAs without work in one
    product or the other."""
    layer = Layer(cfg, group=group)
    ws, out = layer.workspace(), layer.outputs(F32)
    x, z = layer.x.to(DEV), layer.logits.to(DEV)
    want = [t.clone() for t in layer.run(ws=ws, out=out, x=x, logits=z)[:3]]
    for _ in range(8):
        for t in out:
            t.zero_()
        for _ in range(50):
            layer.run(ws=ws, out=out, x=x, logits=z)
        assert device_error(ws) == (0, 0)
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("group", [0, 64])
def test_graph_replays_with_new_inputs(group):
    cfg = MoEConfig("graph", 5, 256, 320, 8, 2, S=1)
    layer = Layer(cfg, group=group)
    ws, out = layer.workspace(), layer.outputs(F32)
    x, z = layer.x.to(DEV), layer.logits.to(DEV)
    layer.run(ws=ws, out=out, x=x, logits=z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        layer.run(ws=ws, out=out, x=x, logits=z)
    for seed in (7, 8, 9):
        other = make_layer_inputs(cfg, seed)
        x.copy_(other.x)
        z.copy_(other.logits)
        graph.replay()
        assert device_error(ws) == (0, 0)
        want = layer.run(x=x, logits=z)
        for a, b in zip(out, want[:3]):
            assert torch.equal(a, b), seed


def test_calls_follow_their_stream():
    """Inputs made on a side stream just before the call, outputs read on it just after."""
    cfg = MoEConfig("stream", 4, 512, 704, 8, 2)
    layer = Layer(cfg)
    want = layer.run()
    s = torch.cuda.Stream()
    ws, out = layer.workspace(), layer.outputs(F32)
    x, z = torch.zeros_like(layer.x, device=DEV), layer.logits.to(DEV)
    src = layer.x.to(DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        x.copy_(src)
        layer.run(ws=ws, out=out, x=x, logits=z)
        got = out[0].clone()
    s.synchronize()
    assert torch.equal(got, want[0])


def test_workspace_serves_other_calls_of_its_shape_in_a_row():
    """Many different routings through one workspace: nothing of one call is left for the next."""
    cfg = MoEConfig("reuse", 30, 128, 192, 64, 6, zipf=True)
    layer = Layer(cfg)
    ws = layer.workspace()
    for seed in range(6):
        inp = make_layer_inputs(cfg, 100 + seed)
        layer.x, layer.logits = inp.x, inp.logits
        y, _, _, _ = layer.run(ws=ws)
        assert device_error(ws) == (0, 0)
        check_y("y", y, layer.reference().y)


@pytest.mark.parametrize("group", [0, 128])
def test_weights_beyond_two_to_the_31(group):
    """The last of 256 experts of a layer whose arrays hold more than 2^31 weights."""
    cfg = MoEConfig("huge", 2, 4096, 2176, 256, 1)
    per = cfg.d * cfg.f
    assert 255 * per > 1 << 31
    z = torch.full((2, 256), -9.0)
    z[0, 255], z[1, 254] = 3.0, 3.0
    small = Layer(cfg.with_(name="two", E=2), group=group, logits=z[:, 254:])
    dev = []
    for t in small.dev:
        big = torch.empty((256, *t.shape[1:]), dtype=t.dtype, device=DEV)
        big[254:] = t
        dev.append(big)
    layer = Layer.__new__(Layer)
    layer.cfg, layer.group, layer.x, layer.logits, layer.dev = cfg, group, small.x, z, dev
    y, idx, w, ws = layer.run()
    assert device_error(ws) == (0, 0)
    assert idx.cpu().tolist() == [[255], [254]]
    p = math.exp(3) / (math.exp(3) + 255 * math.exp(-9))
    ref = small.reference()
    check_y("y", y, ref.y / ref.routing.w * p)


# Widths that end 64, 128 or 192 columns into a stage of 256, experts with 1, 16, 17 and more than 32 rows.
ENDS = [MoEConfig("ends_64", 21, 320, 576, 3, 2, S=1), MoEConfig("ends_128", 40, 128, 640, 2, 1, S=1),
        MoEConfig("ends_192", 17, 448, 192, 16, 3), MoEConfig("ends_0", 64, 512, 256, 24, 2, S=1, zipf=True)]


@pytest.mark.parametrize("cfg", ENDS, ids=lambda c: c.name)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_q4_layer_of_either_type_wherever_the_columns_end(cfg, dtype, group):
    if group == 128:
        cfg = cfg.with_(d=-(-cfg.d // 128) * 128, f=-(-cfg.f // 128) * 128)
    _check(Layer(cfg, group=group), dtype)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_q4_hundreds_of_calls_in_a_row_of_either_type(group, dtype):
    layer = Layer(MoEConfig("many", 37, 384, 640, 16, 4, S=1, zipf=True), group=group)
    ws, out = layer.workspace(), layer.outputs(dtype)
    x, z = layer.x.to(DEV), layer.logits.to(DEV)
    want = [t.clone() for t in layer.run(dtype, ws=ws, out=out, x=x, logits=z)[:3]]
    for _ in range(4):
        for _ in range(50):
            layer.run(dtype, ws=ws, out=out, x=x, logits=z)
        assert device_error(ws) == (0, 0)
        for a, b in zip(out, want):
            assert torch.equal(a, b)


# An fp32 y.  The tensor core cuts its running sum off at 2^-23 of it or less for each instruction, always towards zero:
# over 16 of them (the most that are added up before the sums are rounded to nearest) at most 16 2^-23 = 1.9e-6 of a sum
# that only grows, half of that where it grows evenly.  The layer's second product adds as much again; roundings to
# nearest have signs as good as random and are far below.  So 4e-6 for the layer and 2e-6 for the linear form.
@pytest.mark.parametrize("T", [1, 9, 40, 64])
def test_fp32_sums_stay_exact_over_many_columns(T):
    layer = Layer(MoEConfig("deep", T, 3840, 1920, 7, 3))
    y, _, _, ws = layer.run(F32)
    assert device_error(ws) == (0, 0)
    assert relf(np64(y), layer.reference().y) <= 4e-6


@pytest.mark.parametrize("T,n,K", [(1, 40000, 4096), (9, 20000, 4096), (64, 20000, 8192)])
def test_fp32_linear_sums_stay_exact_over_many_columns(T, n, K):
    g = torch.Generator().manual_seed(K)
    x, W = torch.randn(T, K, generator=g).to(BF16), torch.randn(n, K, generator=g).to(BF16)
    y = torch.empty(T, n, dtype=F32, device=DEV)
    moe.moe_linear_fwd(x.to(DEV), W.to(DEV), y, moe.alloc_linear_workspace(T, n, K))
    ref = x.to(DEV).double() @ W.to(DEV).double().T
    assert ((y.double() - ref).norm() / ref.norm()).item() <= 2e-6
