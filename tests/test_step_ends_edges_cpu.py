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
