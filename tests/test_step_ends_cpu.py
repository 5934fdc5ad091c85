"""The ends of a training step without a GPU: the oracle against torch's float64 autograd, what the library's entry points
refuse before any CUDA call, and what the binding refuses before it calls the library."""
import ctypes

import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300 import build as B
from combine_fp32_softmax_gb300 import moe
from oracle import step_oracle as S

OK = ctypes.c_void_p(1 << 20)            # never dereferenced: checks run first
ODD = ctypes.c_void_p((1 << 20) + 8)     # not 16-byte aligned
WS_ODD = ctypes.c_void_p((1 << 20) + 16)  # not 256-byte aligned
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        B.build()
    return moe.lib()


def cfg(T=12, E=8, k=2):
    return moe.moe_cfg(T, 64, 64, E, k, 0, 0)


# ------------------------------------------------------------------ oracle
def test_oracle_balance_against_autograd():
    rng = np.random.default_rng(0)
    T, E, k, B_ = 24, 7, 3, 3
    z = rng.standard_normal((T, E))
    idx = np.argsort(-z, axis=1)[:, :k]
    mask = rng.random(T) < 0.6
    mask[8:16] = False                     # a sequence without tokens
    dl, dz = rng.standard_normal(B_), rng.standard_normal(B_)
    t = torch.tensor(z, requires_grad=True)
    total, losses, zls = 0.0, [], []
    for b in range(B_):
        rows = torch.arange(b * 8, b * 8 + 8)[torch.tensor(mask[b * 8:b * 8 + 8])]
        if len(rows) == 0:
            losses.append(0.0)
            zls.append(0.0)
            continue
        p = torch.softmax(t[rows], 1)
        f = torch.zeros(E, dtype=torch.float64)
        for r in rows:
            for e in idx[r]:
                f[e] += E / (k * len(rows))
        loss, zl = (f * p.mean(0)).sum(), torch.logsumexp(t[rows], 1).square().mean()
        losses.append(loss.item())
        zls.append(zl.item())
        total = total + dl[b] * loss + dz[b] * zl
    total.backward()
    counts, mean_p, loss, zloss = S.balance_fwd(z, idx, B_, mask)
    assert np.allclose(loss, losses, rtol=1e-12) and np.allclose(zloss, zls, rtol=1e-12)
    assert counts.sum() == k * mask.sum() and not counts[1].any()
    assert np.allclose(S.balance_bwd(z, idx, B_, dl, dz, None, mask), t.grad.numpy(), atol=1e-14)


def test_oracle_xent_against_autograd():
    rng = np.random.default_rng(1)
    T, V, d = 9, 13, 5
    x, W = rng.standard_normal((T, d)), rng.standard_normal((V, d))
    target = rng.integers(0, V, T)
    target[[2, 5]] = -100
    dl, dh = rng.standard_normal(T), rng.standard_normal(T)
    tx, tW = torch.tensor(x, requires_grad=True), torch.tensor(W, requires_grad=True)
    z = tx @ tW.t()
    loss = torch.nn.functional.cross_entropy(z, torch.tensor(target), ignore_index=-100, reduction="none")
    lse = torch.logsumexp(z, 1)
    (loss @ torch.tensor(dl) + lse @ torch.tensor(dh)).backward()
    rl, rs = S.xent_fwd(x, W, target)
    assert np.allclose(rl, loss.detach().numpy()) and np.allclose(rs, lse.detach().numpy())
    D = S.xent_grad(x, W, target, dl, dh)
    assert np.allclose(D @ W, tx.grad.numpy(), atol=1e-13) and np.allclose(D.T @ x, tW.grad.numpy(), atol=1e-13)


@pytest.mark.parametrize("shape", [(6, 10), (10, 6), (8, 8), (1, 5), (1, 1)])
def test_oracle_orthogonalize_acts_on_singular_values(shape):
    G = np.random.default_rng(2).standard_normal(shape)
    u, s, vt = np.linalg.svd(G, full_matrices=False)
    s = s / (np.sqrt((s ** 2).sum()) + 1e-7)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert np.allclose(S.orthogonalize(G, 5), (u * s) @ vt, atol=1e-12)
    assert not S.orthogonalize(np.zeros(shape), 5).any()


# ----------------------------------------------------------------- library
def test_balance_refuses(lib):
    c = cfg()
    fwd = [OK, OK, OK, 1, OK, OK, OK, OK, OK, None]   # logits, picks, mask, seqs, counts, mean_p, loss, zloss, ws, stream
    bwd = [OK, OK, OK, 1, OK, OK, OK, OK, OK, None]   # logits, counts, mask, seqs, dloss, dzloss, in, out, ws, stream

    def call(fn, args, i=None, v=None, cc=c):
        a = list(args)
        if i is not None:
            a[i] = v
        return fn(ctypes.byref(cc), *a)

    for i in (0, 1, 4, 5, 6, 7, 8):
        assert call(lib.moe_balance_fwd, fwd, i, None) == moe.MOE_ERR_ARG
    for i in (0, 1, 4, 5, 7, 8):                      # the mask and the gradient to add to may be NULL
        assert call(lib.moe_balance_bwd, bwd, i, None) == moe.MOE_ERR_ARG
    for fn, args in ((lib.moe_balance_fwd, fwd), (lib.moe_balance_bwd, bwd)):
        for i in (0, 1, 2, 4, 5, 6, 7):
            assert call(fn, args, i, ODD) == moe.MOE_ERR_ALIGN
        assert call(fn, args, 8, WS_ODD) == moe.MOE_ERR_ALIGN
        for seqs in (0, -1, 5, 13, 24):
            assert call(fn, args, 3, seqs) == moe.MOE_ERR_SHAPE
        for bad in (cfg(T=0), cfg(E=257), cfg(E=0), cfg(k=9, E=16), cfg(k=3, E=2)):
            assert call(fn, args, cc=bad) == moe.MOE_ERR_SHAPE
    bwd[0] = ctypes.c_void_p(1 << 22)
    size = 4 * c.T * c.E
    for at in ((1 << 22), (1 << 22) + size - 16, (1 << 22) - size + 16,   # the logits, or a part of them
               (1 << 20) + size - 16, (1 << 20) - size + 16):             # a part of the gradient to add to
        assert call(lib.moe_balance_bwd, bwd, 7, ctypes.c_void_p(at)) == moe.MOE_ERR_ARG


@pytest.mark.parametrize("T,V,d", [(0, 10, 64), (10, 0, 64), (10, 10, 0), (10, 10, 32), (10, 10, 96), ((1 << 22) + 1, 10, 64),
                                   (10, (1 << 22) + 1, 64), (10, 10, 65600), (-1, 10, 64)])
def test_xent_refuses_shapes(lib, T, V, d):
    assert lib.moe_xent_workspace_bytes(T, V, d, 1) == 0
    assert lib.moe_xent_fwd(T, V, d, OK, OK, OK, 1, OK, OK, OK, None) == moe.MOE_ERR_SHAPE
    assert lib.moe_xent_bwd(T, V, d, OK, OK, OK, 1, OK, OK, OK, OK, OK, 0, OK, 0, OK, None) == moe.MOE_ERR_SHAPE


def test_xent_refuses_pointers_and_types(lib):
    fwd = [10, 20, 64, OK, OK, OK, 1, OK, OK, OK, None]
    for i in (3, 4, 5, 7, 8, 9):
        assert lib.moe_xent_fwd(*fwd[:i], None, *fwd[i + 1:]) == moe.MOE_ERR_ARG
        assert lib.moe_xent_fwd(*fwd[:i], ODD if i < 9 else WS_ODD, *fwd[i + 1:]) == moe.MOE_ERR_ALIGN
    for tt in (2, -1):
        assert lib.moe_xent_fwd(*fwd[:6], tt, *fwd[7:]) == moe.MOE_ERR_ARG
    A, C = ctypes.c_void_p(1 << 21), ctypes.c_void_p(1 << 22)
    bwd = [10, 20, 64, OK, OK, OK, 1, OK, OK, OK, OK, A, 0, C, 1, OK, None]
    for i in (3, 4, 5, 7, 8, 9, 15):
        assert lib.moe_xent_bwd(*bwd[:i], None, *bwd[i + 1:]) == moe.MOE_ERR_ARG
    for i in (3, 4, 5, 7, 8, 9, 10, 11, 13):
        assert lib.moe_xent_bwd(*bwd[:i], ODD, *bwd[i + 1:]) == moe.MOE_ERR_ALIGN
    assert lib.moe_xent_bwd(*bwd[:15], WS_ODD, None) == moe.MOE_ERR_ALIGN
    for i in (12, 14):
        assert lib.moe_xent_bwd(*bwd[:i], 2, *bwd[i + 1:]) == moe.MOE_ERR_ARG
    for i, at in ((11, (1 << 20) + 1024), (13, (1 << 20) + 1024), (11, (1 << 20) - 2048), (13, (1 << 21) + 2048)):
        shared = list(bwd)                            # with x and W, or with each other
        shared[i] = ctypes.c_void_p(at)
        assert lib.moe_xent_bwd(*shared) == moe.MOE_ERR_ARG
    none = list(bwd)
    none[11] = none[13] = None                        # nothing to compute
    assert lib.moe_xent_bwd(*none) == moe.MOE_ERR_ARG
    assert lib.moe_xent_ws_init(None, None) == moe.MOE_ERR_ARG
    assert lib.moe_xent_ws_init(WS_ODD, None) == moe.MOE_ERR_ALIGN


def test_xent_workspace(lib):
    """The forward needs little; pieces of the vocabulary keep the backward's from growing with the vocabulary."""
    fwd = moe.moe_xent_workspace_bytes(8192, 100000, 2048, False)
    assert 0 < fwd <= 8192 * (2 * 391 * 8 + 4) + 1024
    big, huge = (moe.moe_xent_workspace_bytes(8192, V, 2048) for V in (100000, 4000000))
    assert big < 1 << 30
    assert huge - big < 8192 * 8 * 2 * (4000000 // 256 + 1)   # the forward's pairs alone
    assert moe.moe_xent_workspace_bytes(1, 1, 64) > 0


@pytest.mark.parametrize("mats,rows,cols", [(0, 8, 8), (1, 0, 8), (1, 8, 0), (-1, 8, 8), (65537, 8, 8), (1, 32769, 8),
                                            (1, 8, 32769), (65536, 32768, 32768)])
def test_orthogonalize_refuses_shapes(lib, mats, rows, cols):
    assert lib.moe_orthogonalize_workspace_bytes(mats, rows, cols) == 0
    assert lib.moe_orthogonalize(mats, rows, cols, OK, 0, ctypes.c_void_p(1 << 21), 5, OK, None) == moe.MOE_ERR_SHAPE


def test_orthogonalize_refuses_arguments(lib):
    out = ctypes.c_void_p(1 << 21)
    good = [1, 8, 8, OK, 0, out, 5, OK, None]
    for steps in (0, -1, 17):
        assert lib.moe_orthogonalize(*good[:6], steps, *good[7:]) == moe.MOE_ERR_SHAPE
    assert lib.moe_orthogonalize(*good[:4], 2, *good[5:]) == moe.MOE_ERR_ARG
    for i in (3, 5, 7):
        assert lib.moe_orthogonalize(*good[:i], None, *good[i + 1:]) == moe.MOE_ERR_ARG
        assert lib.moe_orthogonalize(*good[:i], ODD if i < 7 else WS_ODD, *good[i + 1:]) == moe.MOE_ERR_ALIGN
    for at in (1 << 20, (1 << 20) + 240, (1 << 20) - 112):  # in place, or sharing its end or beginning
        assert lib.moe_orthogonalize(*good[:5], ctypes.c_void_p(at), *good[6:]) == moe.MOE_ERR_ARG


# ----------------------------------------------------------------- binding
class Called(Exception):
    pass


@pytest.fixture
def host(lib, monkeypatch):
    """Host tensors count as being on the current device; a call that passes raises Called."""
    def call(name, *args):
        raise Called(name)
    monkeypatch.setattr(moe, "_call", call)
    monkeypatch.setattr(moe, "_stream", lambda s: None)
    monkeypatch.setattr(moe, "_device", lambda: -1)


def balance_args(**other):
    c = cfg()
    a = dict(cfg=c, logits=torch.zeros(12, 8), topk_idx=torch.zeros(12, 2, dtype=I32), mask=None,
             counts=torch.zeros(3, 8, dtype=I32), mean_p=torch.zeros(3, 8), loss=torch.zeros(3), zloss=torch.zeros(3),
             ws=torch.zeros(moe.moe_workspace_bytes(c), dtype=U8))
    a.update(other)
    return a


def balance_bwd_args(**other):
    a = {n: t for n, t in balance_args().items() if n in ("cfg", "logits", "mask", "counts", "ws")}
    a.update(dloss=torch.zeros(3), dzloss=torch.zeros(3), dlogits_in=None, dlogits=torch.zeros(12, 8))
    a.update(other)
    return a


def test_binding_of_the_balance_loss(host):
    for fn, make in ((moe.moe_balance_fwd, balance_args), (moe.moe_balance_bwd, balance_bwd_args)):
        with pytest.raises(Called):
            fn(**make())
        for mask in (torch.zeros(12, dtype=torch.bool), torch.zeros(12, dtype=U8)):
            with pytest.raises(Called):
                fn(**make(mask=mask))
        for bad in (dict(logits=torch.zeros(8, 12)), dict(logits=torch.zeros(12, 8, dtype=BF16)),
                    dict(counts=torch.zeros(3, 8)), dict(counts=torch.zeros(2, 8, dtype=I32)),
                    dict(mask=torch.zeros(12)), dict(mask=torch.zeros(11, dtype=torch.bool)),
                    dict(ws=torch.zeros(64, dtype=U8)), dict(logits=torch.zeros(8, 12).t())):
            with pytest.raises(ValueError):
                fn(**make(**bad))
    for bad in (dict(topk_idx=torch.zeros(12, 2, dtype=torch.int64)), dict(mean_p=torch.zeros(3, 7)), dict(zloss=torch.zeros(2))):
        with pytest.raises(ValueError):
            moe.moe_balance_fwd(**balance_args(**bad))
    for bad in (dict(dlogits_in=torch.zeros(12, 7)), dict(dlogits=torch.zeros(11, 8)), dict(dzloss=torch.zeros(3, 1))):
        with pytest.raises(ValueError):
            moe.moe_balance_bwd(**balance_bwd_args(**bad))
    with pytest.raises(Called):
        moe.moe_balance_bwd(**balance_bwd_args(dlogits_in=torch.zeros(12, 8)))


def xent_args(backward, **other):
    a = dict(x=torch.zeros(6, 64, dtype=BF16), W=torch.zeros(9, 64, dtype=BF16), target=torch.zeros(6, dtype=torch.int64),
             loss=torch.zeros(6), lse=torch.zeros(6), ws=torch.zeros(moe.moe_xent_workspace_bytes(6, 9, 64, backward), dtype=U8))
    if backward:
        a.update(dloss=torch.zeros(6), dlse=None, dx=torch.zeros(6, 64), dW=torch.zeros(9, 64, dtype=BF16))
    a.update(other)
    return a


def test_binding_of_the_cross_entropy(host):
    for fn, backward in ((moe.moe_xent_fwd, False), (moe.moe_xent_bwd, True)):
        for good in ({}, dict(target=torch.zeros(6, dtype=I32))):
            with pytest.raises(Called):
                fn(**xent_args(backward, **good))
        for bad in (dict(x=torch.zeros(6, 64)), dict(x=torch.zeros(6, 128, dtype=BF16)), dict(W=torch.zeros(9, 64)),
                    dict(target=torch.zeros(6)), dict(target=torch.zeros(5, dtype=I32)), dict(loss=torch.zeros(6, dtype=BF16)),
                    dict(lse=torch.zeros(6, 1)), dict(ws=torch.zeros(256, dtype=U8)), dict(x=torch.zeros(384, dtype=BF16)),
                    dict(W=torch.zeros(64, 9, dtype=BF16).t()), dict(x=torch.zeros(6, 128, dtype=BF16)[:, ::2])):
            with pytest.raises(ValueError):
                fn(**xent_args(backward, **bad))
    for good in (dict(dx=None), dict(dW=None), dict(dlse=torch.zeros(6))):
        with pytest.raises(Called):
            moe.moe_xent_bwd(**xent_args(True, **good))
    for bad in (dict(dx=torch.zeros(6, 64, dtype=torch.float16)), dict(dx=torch.zeros(5, 64)), dict(dW=torch.zeros(9, 65)),
                dict(dloss=torch.zeros(6, dtype=torch.float64)), dict(dlse=torch.zeros(7))):
        with pytest.raises(ValueError):
            moe.moe_xent_bwd(**xent_args(True, **bad))
    with pytest.raises(moe.MoeError):
        moe.alloc_xent_workspace(6, 9, 65, device="cpu")


def test_binding_of_orthogonalize(host):
    ws = torch.zeros(moe.moe_orthogonalize_workspace_bytes(2, 9, 5), dtype=U8)
    for dt in (F32, BF16):
        with pytest.raises(Called):
            moe.moe_orthogonalize(torch.zeros(2, 9, 5, dtype=dt), torch.zeros(2, 9, 5, dtype=BF16), 5, ws)
    with pytest.raises(Called):
        moe.moe_orthogonalize(torch.zeros(9, 5), torch.zeros(9, 5, dtype=BF16), 5, ws)
    for G, out, w in ((torch.zeros(2, 9, 5), torch.zeros(2, 9, 5), ws), (torch.zeros(2, 9, 5), torch.zeros(9, 5, dtype=BF16), ws),
                      (torch.zeros(2, 9, 5, dtype=torch.float16), torch.zeros(2, 9, 5, dtype=BF16), ws),
                      (torch.zeros(5), torch.zeros(5, dtype=BF16), ws), (torch.zeros(2, 5, 9).transpose(1, 2), torch.zeros(2, 9, 5, dtype=BF16), ws),
                      (torch.zeros(2, 9, 5), torch.zeros(2, 9, 5, dtype=BF16), ws[:256])):
        with pytest.raises(ValueError):
            moe.moe_orthogonalize(G, out, 5, w)
    with pytest.raises(moe.MoeError):
        moe.alloc_orthogonalize_workspace(1, 40000, 8, device="cpu")


def test_binding_refuses_host_tensors(lib, monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        moe.moe_xent_fwd(**xent_args(False))
    with pytest.raises(ValueError, match="current device"):
        moe.moe_balance_fwd(**balance_args())
