"""What the calls of a training step's ends refuse, beside test_step_ends_cpu.py."""
import ctypes

import pytest
import torch

from combine_fp32_softmax_gb300 import moe
from tests.test_step_ends_cpu import OK, balance_args, balance_bwd_args, cfg, host, lib, xent_args  # noqa: F401

BF16, U8 = torch.bfloat16, torch.uint8


def at(address):
    return ctypes.c_void_p(address)


# ----------------------------------------------------------------- binding
def test_binding_names_what_is_missing(host):  # noqa: F811
    for fn, make, names in ((moe.moe_balance_fwd, balance_args, ("logits", "topk_idx", "counts", "mean_p", "loss", "zloss", "ws")),
                            (moe.moe_balance_bwd, balance_bwd_args, ("logits", "counts", "dloss", "dzloss", "dlogits", "ws")),
                            (moe.moe_xent_fwd, lambda **o: xent_args(False, **o), ("x", "W", "target", "loss", "lse", "ws")),
                            (moe.moe_xent_bwd, lambda **o: xent_args(True, **o),
                             ("x", "W", "target", "loss", "lse", "dloss", "ws"))):
        for name in names:
            with pytest.raises(ValueError, match=f"^{name}: "):
                fn(**make(**{name: None}))
    ws = torch.zeros(moe.moe_orthogonalize_workspace_bytes(1, 9, 5), dtype=U8)
    good = dict(G=torch.zeros(9, 5), O=torch.zeros(9, 5, dtype=BF16), ws=ws)
    for name in good:
        with pytest.raises(ValueError, match=f"^{name}: "):
            moe.moe_orthogonalize(**{**good, name: None}, steps=5)


# ----------------------------------------------------------------- library
# One call's arrays far apart; a result moved onto an input or another result, at either of its ends, is refused.
def apart(n):
    return [(1 << 30) + (i << 24) for i in range(n)]


def test_balance_refuses_results_in_other_arrays(lib):  # noqa: F811
    c = cfg(T=12, E=8, k=2)
    logits, picks, mask, counts, mean_p, loss, zloss = names = apart(7)
    sizes = dict(zip(names, (4 * 12 * 8, 4 * 12 * 2, 12, 4 * 3 * 8, 4 * 3 * 8, 4 * 3, 4 * 3)))

    def fwd(**moved):
        a = dict(counts=counts, mean_p=mean_p, loss=loss, zloss=zloss)
        a.update(moved)
        return lib.moe_balance_fwd(ctypes.byref(c), at(logits), at(picks), at(mask), 3, at(a["counts"]), at(a["mean_p"]),
                                   at(a["loss"]), at(a["zloss"]), OK, None)

    for name, own in (("counts", counts), ("mean_p", mean_p), ("loss", loss), ("zloss", zloss)):
        for other in names:
            if other != own:
                last = other + (sizes[other] - 1) // 16 * 16   # the other's last 16 bytes
                first = other - (sizes[own] - 1) // 16 * 16    # its first ones
                assert [fwd(**{name: p}) for p in (other, last, first)] == [moe.MOE_ERR_ARG] * 3, name

    read = {mask: 12, counts: 4 * 3 * 8, loss: 4 * 3, zloss: 4 * 3}   # the gradients of both losses in their places
    for other, n in read.items():
        for p in (other, other + (n - 1) // 16 * 16, other - (4 * 12 * 8 - 16)):
            assert lib.moe_balance_bwd(ctypes.byref(c), at(logits), at(counts), at(mask), 3, at(loss), at(zloss), None, at(p), OK,
                                       None) == moe.MOE_ERR_ARG


def test_xent_refuses_results_in_other_arrays(lib):  # noqa: F811
    T, V, d = 10, 20, 64
    x, W, target, loss, lse, dloss, dlse, dx, dW = apart(9)
    sizes = {x: 2 * T * d, W: 2 * V * d, target: 8 * T, loss: 4 * T, lse: 4 * T, dloss: 4 * T, dlse: 4 * T, dx: 4 * T * d, dW: 2 * V * d}

    def places(own, other):
        return other, other + (sizes[other] - 1) // 16 * 16, other - (sizes[own] - 1) // 16 * 16

    for other in (x, W, target, lse):
        for p in places(loss, other):
            assert lib.moe_xent_fwd(T, V, d, at(x), at(W), at(target), moe.MOE_I64, at(p), at(lse), OK, None) == moe.MOE_ERR_ARG
    for other in (x, W, target, loss):
        for p in places(lse, other):
            assert lib.moe_xent_fwd(T, V, d, at(x), at(W), at(target), moe.MOE_I64, at(loss), at(p), OK, None) == moe.MOE_ERR_ARG

    def bwd(dx, dW):
        return lib.moe_xent_bwd(T, V, d, at(x), at(W), at(target), moe.MOE_I64, at(loss), at(lse), at(dloss), at(dlse), at(dx),
                                moe.MOE_Y_F32, at(dW), moe.MOE_Y_BF16, OK, None)

    for other in (x, W, target, loss, lse, dloss, dlse):
        for p in places(dx, other):
            assert bwd(p, dW) == moe.MOE_ERR_ARG
        for p in places(dW, other):
            assert bwd(dx, p) == moe.MOE_ERR_ARG
    for p in places(dW, dx):
        assert bwd(dx, p) == moe.MOE_ERR_ARG
