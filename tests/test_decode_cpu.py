"""The layer for a few tokens and the 4-bit format without a GPU: refusals on the host before any CUDA call, and the
reference of the packed format against a hand-worked block."""
import ctypes

import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300 import build as B
from combine_fp32_softmax_gb300 import moe
from oracle import q4_oracle as Q

OK = ctypes.c_void_p(1 << 20)          # never dereferenced: the checks run first
ODD = ctypes.c_void_p((1 << 20) + 8)   # 8-byte aligned only
WS_ODD = ctypes.c_void_p((1 << 20) + 16)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        B.build()
    return moe.lib()


def _cfg(**kw):
    base = dict(T=8, d_model=256, d_ff=384, E=8, k=2, n_shared=0, renorm=0)
    base.update(kw)
    return ctypes.byref(moe.moe_cfg(*[base[n] for n, _ in moe.moe_cfg._fields_]))


def _decode(lib, cfg, ptrs=(OK,) * 6, y_type=0, out=(OK, OK), ws=OK):
    return lib.moe_decode_fwd(cfg, *ptrs, y_type, *out, ws, None)


def _decode_q4(lib, cfg, group=64, ptrs=(OK,) * 9, y_type=0, out=(OK, OK), ws=OK):
    return lib.moe_decode_q4_fwd(cfg, group, *ptrs, y_type, *out, ws, None)


@pytest.mark.parametrize("bad", [dict(T=0), dict(T=65), dict(E=0), dict(E=257), dict(k=0), dict(k=9, E=16),
                                 dict(k=5, E=4), dict(d_model=96), dict(d_ff=100), dict(n_shared=5), dict(renorm=2)])
def test_decode_refuses_shapes(lib, bad):
    c = _cfg(**bad)
    assert lib.moe_decode_workspace_bytes(c) == 0
    assert lib.moe_decode_ws_init(c, OK, None) == moe.MOE_ERR_SHAPE
    assert _decode(lib, c) == moe.MOE_ERR_SHAPE
    assert _decode_q4(lib, c) == moe.MOE_ERR_SHAPE


def test_decode_refuses_pointers_and_types(lib):
    c = _cfg()
    assert lib.moe_decode_workspace_bytes(c) % 256 == 0 and lib.moe_decode_workspace_bytes(c) > 0
    for i in range(6):
        for p, rc in ((None, moe.MOE_ERR_ARG), (ODD, moe.MOE_ERR_ALIGN)):
            assert _decode(lib, c, ptrs=(OK,) * i + (p,) + (OK,) * (5 - i)) == rc
    for i in range(9):
        for p, rc in ((None, moe.MOE_ERR_ARG), (ODD, moe.MOE_ERR_ALIGN)):
            assert _decode_q4(lib, c, ptrs=(OK,) * i + (p,) + (OK,) * (8 - i)) == rc
    for out in ((None, OK), (OK, None)):
        assert _decode(lib, c, out=out) == moe.MOE_ERR_ARG
    assert _decode(lib, c, y_type=2) == moe.MOE_ERR_ARG and _decode(lib, c, y_type=-1) == moe.MOE_ERR_ARG
    assert _decode(lib, c, ws=None) == moe.MOE_ERR_ARG and _decode(lib, c, ws=WS_ODD) == moe.MOE_ERR_ALIGN
    assert lib.moe_decode_fwd(None, *(OK,) * 6, 0, OK, OK, OK, None) == moe.MOE_ERR_ARG


@pytest.mark.parametrize("group", [0, -64, 16, 48, 256])
def test_decode_q4_refuses_groups(lib, group):
    assert _decode_q4(lib, _cfg(), group=group) == moe.MOE_ERR_SHAPE


def test_decode_q4_refuses_widths_that_groups_do_not_divide(lib):
    assert _decode_q4(lib, _cfg(d_model=320), group=128) == moe.MOE_ERR_SHAPE
    assert _decode_q4(lib, _cfg(d_ff=320), group=128) == moe.MOE_ERR_SHAPE


@pytest.mark.parametrize("T,n,K", [(0, 8, 64), (65, 8, 64), (1, 0, 64), (1, 8, 0), (1, 8, 32), (1, 8, 96), (1, 8, -64),
                                   (1, 0x7FFFFF00, 64)])
def test_linear_refuses_shapes(lib, T, n, K):
    assert lib.moe_linear_workspace_bytes(T, n, K) == 0
    assert lib.moe_linear_ws_init(T, n, K, OK, None) == moe.MOE_ERR_SHAPE
    assert lib.moe_linear_fwd(T, n, K, OK, OK, OK, 0, OK, None) == moe.MOE_ERR_SHAPE
    assert lib.moe_linear_q4_fwd(T, n, K, 32, OK, OK, OK, OK, 0, OK, None) == moe.MOE_ERR_SHAPE


def test_linear_refuses_pointers_types_and_groups(lib):
    assert lib.moe_linear_fwd(1, 8, 64, None, OK, OK, 0, OK, None) == moe.MOE_ERR_ARG
    assert lib.moe_linear_fwd(1, 8, 64, OK, ODD, OK, 0, OK, None) == moe.MOE_ERR_ALIGN
    assert lib.moe_linear_fwd(1, 8, 64, OK, OK, OK, 3, OK, None) == moe.MOE_ERR_ARG
    assert lib.moe_linear_fwd(1, 8, 64, OK, OK, OK, 0, WS_ODD, None) == moe.MOE_ERR_ALIGN
    assert lib.moe_linear_q4_fwd(1, 8, 64, 64, OK, OK, None, OK, 0, OK, None) == moe.MOE_ERR_ARG
    assert lib.moe_linear_q4_fwd(1, 8, 64, 128, OK, OK, OK, OK, 0, OK, None) == moe.MOE_ERR_SHAPE
    assert lib.moe_linear_q4_fwd(1, 8, 64, 16, OK, OK, OK, OK, 0, OK, None) == moe.MOE_ERR_SHAPE


@pytest.mark.parametrize("mats,rows,cols,group", [(0, 8, 64, 64), (1, 0, 64, 64), (1, 8, 0, 64), (1, 8, 96, 64),
                                                  (1, 8, 64, 128), (1, 8, 64, 0), (1, 8, 64, 8), (1, 0x7FFFFF00, 64, 64)])
def test_q4_refuses_shapes(lib, mats, rows, cols, group):
    assert lib.moe_q4_quantize(OK, OK, OK, mats, rows, cols, group, None) == moe.MOE_ERR_SHAPE
    assert lib.moe_q4_dequantize(OK, OK, OK, mats, rows, cols, group, None) == moe.MOE_ERR_SHAPE


def test_q4_refuses_pointers(lib):
    for fn in (lib.moe_q4_quantize, lib.moe_q4_dequantize):
        for i in range(3):
            assert fn(*((OK,) * i + (None,) + (OK,) * (2 - i)), 1, 8, 64, 64, None) == moe.MOE_ERR_ARG
            assert fn(*((OK,) * i + (ODD,) + (OK,) * (2 - i)), 1, 8, 64, 64, None) == moe.MOE_ERR_ALIGN


def test_binding_refuses_sizes_and_host_tensors(lib):
    x, y = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(3, 8)
    W = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # rows of x and y differ
        moe.moe_linear_fwd(x, W, y, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):  # W of another size
        moe.moe_linear_fwd(x, W[:7], y[:2], torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):  # host tensors
        moe.moe_linear_fwd(x, W, y[:2], torch.zeros(256, dtype=torch.uint8))
    codes, scales = moe.q4_empty(1, 8, 64, 32, device="cpu")
    assert codes.shape == (1, 8, 32) and scales.shape == (1, 2, 8)
    with pytest.raises(ValueError):
        moe.moe_q4_quantize(W, codes, scales[:, :1], 32)
    with pytest.raises(moe.MoeError):
        moe.alloc_linear_workspace(65, 8, 64, device="cpu")
    with pytest.raises(moe.MoeError):
        moe.alloc_decode_workspace(moe.moe_cfg(65, 256, 256, 8, 2, 0, 0), device="cpu")


def test_packed_format_by_hand():
    q = np.arange(8, dtype=np.int64)[None] + 1      # columns 0..7 hold 1..8
    # nibbles 0..3: columns 0, 2, 4, 6 = 1, 3, 5, 7; nibbles 4..7: columns 1, 3, 5, 7 = 2, 4, 6, 8
    assert Q.pack(q).tolist() == [[0x31, 0x75, 0x42, 0x86]]
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (3, 5, 64))
    assert np.array_equal(Q.unpack(Q.pack(q)), q)


def test_quantize_reference_keeps_half_a_step():
    w = torch.randn(2, 9, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    codes, scales = Q.quantize(w, 64)
    s = scales.double().numpy()[:, :, :9].transpose(0, 2, 1).repeat(64, axis=2)
    # half a step, and the largest magnitude up to 7 s (1 + 2^-8), s being rounded to bf16
    assert (np.abs(Q.values(codes, scales, 64) - w.double().numpy()) <= s * (0.5 + 7 * 2.0 ** -8)).all()
    assert not scales[:, :, 9:].any()


def test_quotient_of_the_quantizer_rounds_like_the_division():
    """x * r, one Newton step and the addition of 1.5 * 2^23 in fp32 give rint(x / s), ties to even, for every pair of
    bf16 significands in the range and every r within 1 ulp of 1 / s (fused operations emulated in fp64, where their
    one rounding is to fp32).  absmax * fl(1/7), rounded to bf16, is the quotient by 7."""
    f32, f64 = np.float32, np.float64
    top = torch.arange(128, 256).float() / 128
    assert torch.equal((top * torch.tensor(1 / 7)).to(torch.bfloat16), (top.double() / 7).to(torch.bfloat16))
    for ms, off in ((m, o) for m in range(128, 256) for o in (-1, 0, 1)):
        s = f32(ms / 128)
        r = f32(1) / s
        r = np.nextafter(r, f32(9 * off)) if off else r
        x = np.concatenate([np.arange(128, 256) / 128 * 2.0 ** e for e in range(-12, 4)]).astype(f32)
        x = x[x <= 7.1 * s]
        x = np.concatenate([x, -x])
        y = x * r
        rest = (x.astype(f64) - y.astype(f64) * f64(s)).astype(f32)
        y = (rest.astype(f64) * f64(r) + y.astype(f64)).astype(f32)
        got = ((y + f32(12582912 + 8)).view(np.uint32) & 15).astype(np.int64) - 8
        num, den = np.rint(x.astype(f64) * 2 ** 20).astype(np.int64), int(f64(s) * 2 ** 20)
        low, rem = num // den, num % den
        want = low + ((2 * rem > den) | ((2 * rem == den) & (low % 2 != 0)))
        assert np.array_equal(got, want), ms
