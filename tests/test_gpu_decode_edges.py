"""The layer for a few tokens at its edges: infinite weights, tiles drawn from a counter, one workspace for several
token counts, sums of one sign, waits that run out."""
import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300 import moe
from combine_fp32_softmax_gb300.configs import MoEConfig
from oracle import moe_oracle as O
from tests.gpu_util import DEV, np64
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
