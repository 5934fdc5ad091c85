"""What the binding of the calls for a few tokens refuses before it calls the library: arrays and workspaces that are
too small, too large or of another type.  Host tensors that say they are on the GPU stand in, and a call that passes
raises Called instead of reaching the library."""
import pytest
import torch

from combine_fp32_softmax_gb300 import build as B
from combine_fp32_softmax_gb300 import moe
from combine_fp32_softmax_gb300.configs import MoEConfig

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
CFG = MoEConfig("small", 5, 128, 192, 6, 2, S=1)
T, D, F, E, K, N = 5, 128, 192, 6, 2, 7
G = 64


class Called(Exception):
    pass


class OnGpu(torch.Tensor):
    is_cuda = True


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def empty_q4(*a):
    return [t.as_subclass(OnGpu) for t in moe.q4_empty(*a, device="cpu")]


@pytest.fixture(autouse=True)
def lib(monkeypatch):
    import os
    if not os.path.exists(B.LIB_PATH):
        B.build()

    def call(name, *args):
        raise Called(name)
    monkeypatch.setattr(moe, "_call", call)
    monkeypatch.setattr(moe, "_stream", lambda s: None)


def layer_args(**other):
    a = dict(logits=zeros(T, E), x=zeros(T, D, dtype=BF16), W1=zeros(N, F, D, dtype=BF16),
             W3=zeros(N, F, D, dtype=BF16), W2=zeros(N, D, F, dtype=BF16), y=zeros(T, D),
             topk_idx=zeros(T, K, dtype=I32), topk_w=zeros(T, K),
             ws=zeros(moe.moe_decode_workspace_bytes(CFG), dtype=U8))
    a.update(other)
    return a


def q4_args(**other):
    a = {n: t for n, t in layer_args().items() if n not in ("W1", "W3", "W2")}
    for n, rows, cols in (("W1", F, D), ("W3", F, D), ("W2", D, F)):
        a[n + "q"], a[n + "s"] = empty_q4(N, rows, cols, G)
    a.update(other)
    return a


LAYER_BAD = [("logits", zeros(T, E - 1)), ("logits", zeros(T, E, dtype=BF16)), ("logits", zeros(2 * T, E + 1)),
             ("x", zeros(T, D)), ("x", zeros(T - 1, D, dtype=BF16)),
             ("y", zeros(T, D - 64)), ("y", zeros(T, 2 * D)),
             ("topk_idx", zeros(T, K, dtype=torch.int64)), ("topk_idx", zeros(T, 1, dtype=I32)),
             ("topk_w", zeros(T, K, dtype=BF16)), ("topk_w", zeros(T - 1, K)),
             ("ws", zeros(256, dtype=U8))]


@pytest.mark.parametrize("name,bad", LAYER_BAD + [
    ("W1", zeros(N - 1, F, D, dtype=BF16)), ("W3", zeros(N, F, D)), ("W2", zeros(N, D, F - 64, dtype=BF16))])
def test_layer_refuses(name, bad):
    with pytest.raises(ValueError, match=f"^{name}: "):
        moe.moe_decode_fwd(CFG, **layer_args(**{name: bad}))


@pytest.mark.parametrize("name,bad", LAYER_BAD + [
    ("W1q", zeros(N - 1, F, D // 2, dtype=U8)), ("W3q", zeros(N, F, D // 2, dtype=I32)),
    ("W2q", zeros(N, D, F, dtype=U8)), ("W1s", zeros(N, D // G, F)),
    ("W3s", zeros(N, D // 32, F, dtype=BF16)), ("W2s", zeros(N, F // G, D - 8, dtype=BF16))])
def test_q4_layer_refuses(name, bad):
    with pytest.raises(ValueError, match=f"^{name}: "):
        moe.moe_decode_q4_fwd(CFG, G, **q4_args(**{name: bad}))


def test_right_arrays_pass_and_either_type_of_y_does():
    for y in (zeros(T, D), zeros(T, D, dtype=BF16)):
        with pytest.raises(Called):
            moe.moe_decode_fwd(CFG, **layer_args(y=y))
        with pytest.raises(Called):
            moe.moe_decode_q4_fwd(CFG, G, **q4_args(y=y))


def test_buffers_for_more_tokens_serve_fewer():
    big = dict(logits=zeros(64, E), x=zeros(64, D, dtype=BF16), y=zeros(64, D),
               topk_idx=zeros(64, K, dtype=I32), topk_w=zeros(64 * K))
    with pytest.raises(Called):
        moe.moe_decode_fwd(CFG, **layer_args(**big))
    with pytest.raises(Called):
        moe.moe_decode_q4_fwd(CFG, G, **q4_args(**big))


def test_a_workspace_for_more_tokens_serves_fewer():
    sizes = [moe.moe_decode_workspace_bytes(moe.moe_cfg(t, D, F, E, K, 1, 0)) for t in range(1, 65)]
    assert sizes == sorted(sizes)
    with pytest.raises(Called):
        moe.moe_decode_fwd(CFG, **layer_args(ws=zeros(sizes[-1], dtype=U8)))
    with pytest.raises(ValueError, match="^ws: "):
        moe.moe_decode_fwd(CFG, **layer_args(ws=zeros(sizes[0], dtype=U8)))


def test_workspaces_too_small_are_not_cleared():
    with pytest.raises(ValueError, match="^ws: "):
        moe.moe_decode_ws_init(CFG, zeros(256, dtype=U8))
    with pytest.raises(ValueError, match="^ws: "):
        moe.moe_linear_ws_init(1, 8, 64, zeros(256, dtype=U8))


@pytest.mark.parametrize("name,bad", [("x", zeros(2, 64)), ("W", zeros(8, 64)), ("ws", zeros(256, dtype=U8))])
def test_linear_refuses(name, bad):
    a = dict(x=zeros(2, 64, dtype=BF16), W=zeros(8, 64, dtype=BF16), y=zeros(2, 8),
             ws=zeros(moe.moe_linear_workspace_bytes(2, 8, 64), dtype=U8))
    with pytest.raises(Called):
        moe.moe_linear_fwd(**a)
    a[name] = bad
    with pytest.raises(ValueError, match=f"^{name}: "):
        moe.moe_linear_fwd(**a)


@pytest.mark.parametrize("name,bad", [("x", zeros(2, 64)), ("Wq", zeros(8, 32, dtype=I32)),
                                      ("Ws", zeros(2, 8)), ("ws", zeros(256, dtype=U8))])
def test_linear_q4_refuses(name, bad):
    codes, scales = empty_q4(1, 8, 64, 32)
    a = dict(x=zeros(2, 64, dtype=BF16), Wq=codes, Ws=scales, group=32, y=zeros(2, 8),
             ws=zeros(moe.moe_linear_workspace_bytes(2, 8, 64), dtype=U8))
    with pytest.raises(Called):
        moe.moe_linear_q4_fwd(**a)
    a[name] = bad
    with pytest.raises(ValueError, match=f"^{name}: "):
        moe.moe_linear_q4_fwd(**a)


@pytest.mark.parametrize("name,bad", [("W", zeros(8, 64)), ("codes", zeros(8, 32, dtype=torch.int8)),
                                      ("scales", zeros(2, 8))])
def test_quantize_refuses_types(name, bad):
    codes, scales = empty_q4(1, 8, 64, 32)
    a = dict(W=zeros(8, 64, dtype=BF16), codes=codes, scales=scales, group=32)
    for fn in (moe.moe_q4_quantize, moe.moe_q4_dequantize):
        with pytest.raises(Called):
            fn(**a)
        with pytest.raises(ValueError, match=f"^{name}: "):
            fn(**{**a, name: bad})


def test_host_tensors_and_strides_are_refused():
    for bad in (torch.zeros(T, D, dtype=BF16), zeros(T, 2 * D, dtype=BF16)[:, ::2]):
        with pytest.raises(ValueError, match="CUDA|contiguous"):
            moe.moe_decode_fwd(CFG, **layer_args(x=bad))
    for bad in (torch.zeros(N, F, D, dtype=BF16), zeros(N, D, F, dtype=BF16).transpose(1, 2)):
        with pytest.raises(ValueError, match="CUDA|contiguous"):
            moe.moe_decode_fwd(CFG, **layer_args(W1=bad))


@pytest.mark.parametrize("name", ["logits", "x", "W1", "W3", "W2", "topk_idx", "topk_w", "ws"])
def test_missing_arrays_reach_the_library(name):
    """None becomes a null pointer, which the library refuses."""
    with pytest.raises(Called):
        moe.moe_decode_fwd(CFG, **layer_args(**{name: None}))
    names = [name] if name[0] != "W" else [name + "q", name + "s"]
    for n in names:
        with pytest.raises(Called):
            moe.moe_decode_q4_fwd(CFG, G, **q4_args(**{n: None}))


def test_both_forms_of_a_configuration():
    c = moe.moe_cfg(T, D, F, E, K, 1, 0)
    assert moe.moe_decode_workspace_bytes(c) == moe.moe_decode_workspace_bytes(CFG) > 0
    with pytest.raises(Called):
        moe.moe_decode_fwd(c, **layer_args())
    c.T = T + 1                                    # the same object with another number of tokens
    with pytest.raises(ValueError, match="^logits: "):
        moe.moe_decode_fwd(c, **layer_args())
