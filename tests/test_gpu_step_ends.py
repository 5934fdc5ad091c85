"""The ends of a training step on the GPU against the fp64 oracle: balance loss, cross entropy over a vocabulary,
orthogonalised matrices.

Tolerances, derived from the kernels' stated roundings:
  * a logit: its sum loses at most 2^-23 of S = sum |x||W| for each 16 columns of a tensor core's run, and 2^-24 of S for
    each addition of runs; runs have up to 768 columns and are held to the bound of 512, the stricter one: dz = (2^-18 + d 2^-33) max S;
  * lse: dz, the error of the exponentials, sum and log (2^-20 together: the exponential is within 2 + |z| ulp of terms that
    add up to the sum), and its own rounding; loss: 2 dz and the same;
  * D: relative 2 dz + 2^-20 + 2^-23 |lse| for the exponential, plus its rounding, 2^-8 in bf16 and 2^-24 as three
    bf16 values; a product of it: that part of sum |D||W|, the tensor core's loss over the K of one run (2^-23 for each 16
    terms), and the result's own rounding, 2^-8 or 2^-24."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300 import moe
from oracle import moe_oracle as O
from oracle import step_oracle as S
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def put(t, label="in"):
    """A device copy between guard regions."""
    d = U.guarded_empty(tuple(t.shape), t.dtype, label)
    d.copy_(t)
    return d


def workspace(nbytes, init):
    ws = U.guarded_empty((nbytes,), torch.uint8, "ws")
    ws.fill_(0xFF)  # NaN in every type: nothing may depend on what a workspace held
    init(ws)
    return ws


# ----------------------------------------------------------------- balance
def balance_inputs(T, E, k, B, masked, seed=0, scale=1.0):
    z = torch.randn(T, E, generator=gen(seed)) * scale
    idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k].int()
    mask = None
    if masked == "tail":
        keep = torch.randint(0, T // B + 1, (B, 1), generator=gen(seed + 1))
        mask = (torch.arange(T // B) < keep).reshape(T)
    elif masked == "none left":
        mask = torch.zeros(T, dtype=torch.bool)
    elif masked == "random":
        mask = torch.rand(T, generator=gen(seed + 1)) < 0.5
    if mask is not None:
        z[~mask] = float("nan")
        idx[~mask] = 1 << 30
    return z, idx, mask


def run_balance(z, idx, mask, B, dloss, dz, add, in_place=False):
    T, E = z.shape
    cfg = moe.moe_cfg(T, 64, 64, E, idx.shape[1], 0, 0)
    ws = workspace(moe.moe_workspace_bytes(cfg), lambda w: moe.moe_ws_init(cfg, w))
    g = {n: put(t) if t is not None else None for n, t in dict(z=z, idx=idx, mask=mask, dloss=dloss, dz=dz, add=add).items()}
    counts, mean_p = U.guarded_empty((B, E), I32), U.guarded_empty((B, E), F32)
    loss, zloss = U.guarded_empty((B,), F32), U.guarded_empty((B,), F32)
    out = g["add"] if in_place else U.guarded_empty((T, E), F32)
    moe.moe_balance_fwd(cfg, g["z"], g["idx"], g["mask"], counts, mean_p, loss, zloss, ws)
    moe.moe_balance_bwd(cfg, g["z"], counts, g["mask"], g["dloss"], g["dz"], g["add"], out, ws)
    return counts, mean_p, loss, zloss, out, ws


@pytest.mark.parametrize("T,E,k,B,masked", [
    (1, 1, 1, 1, None), (1, 5, 3, 1, None), (7, 8, 2, 7, None), (64, 2, 2, 1, "random"), (512, 8, 2, 1, None),
    (513, 33, 3, 1, "random"), (700, 64, 6, 7, "tail"), (1000, 65, 8, 2, "tail"), (1000, 128, 8, 1, None),
    (2048, 129, 5, 4, "random"), (999, 256, 8, 3, None), (96, 16, 4, 2, "none left"), (33 * 40, 20, 4, 40, "tail"),
    (20000, 64, 6, 1, "random"), (40000, 8, 2, 5, "tail"), (4096, 8, 2, 4096, "random")])
def test_balance(T, E, k, B, masked):
    z, idx, mask = balance_inputs(T, E, k, B, masked)
    dloss, dz = torch.randn(B, generator=gen(5)), torch.randn(B, generator=gen(6))
    add = torch.randn(T, E, generator=gen(7))
    counts, mean_p, loss, zloss, out, ws = run_balance(z, idx, mask, B, dloss, dz, add)
    assert U.device_error(ws) == (0, 0)
    zn, mn = z.numpy(), None if mask is None else mask.numpy()
    rc, rp, rl, rz = S.balance_fwd(np.nan_to_num(zn), np.where(idx.numpy() < E, idx.numpy(), 0), B, mn)
    assert np.array_equal(counts.cpu().numpy(), rc)
    # p: the router's own bound (4e-6 relative); a block adds up to T / 608 + 32 of them in fp32, and its sum is rounded
    tol = 4e-6 + (T / 608 / 8 + 8) * 2.0 ** -24
    assert np.all(np.abs(U.np64(mean_p) - rp) <= tol * rp + 1e-30)
    assert np.all(np.abs(U.np64(loss) - rl) <= tol * np.abs(rl))
    # lse is off by 2^-24 (|m| + |log s|) and the log's own error; |lse| <= |m| + log E
    big = np.abs(np.nan_to_num(zn)).max() + np.log(E)
    assert np.all(np.abs(U.np64(zloss) - rz) <= 8 * 2.0 ** -23 * big * (big + 1) + tol * rz)
    ref = S.balance_bwd(np.nan_to_num(zn), np.where(idx.numpy() < E, idx.numpy(), 0), B, dloss.numpy(), dz.numpy(),
                        add.numpy(), mn)
    # the two terms of a gradient, each 1e-5 of its largest possible size: a softmax to 4e-6, a dot of E terms, lse
    n = np.array([len(S._rows(T, B, b, mn)) for b in range(B)]).repeat(T // B)[:, None]
    c = np.abs(dloss.numpy())[:, None] * rc.max(1, keepdims=True) * E / k
    size = (c.repeat(T // B, 0) / np.maximum(n, 1) + 2 * np.abs(dz.numpy()).repeat(T // B)[:, None] * big) / np.maximum(n, 1)
    assert np.all(np.abs(U.np64(out) - ref) <= 2.0 ** -24 * np.abs(ref) + 2e-5 * size)


def test_balance_adds_in_place_and_without():
    z, idx, mask = balance_inputs(300, 64, 6, 3, "tail")
    d, add = torch.ones(3), torch.randn(300, 64, generator=gen(1))
    a = run_balance(z, idx, mask, 3, d, d, add)[4]
    b = run_balance(z, idx, mask, 3, d, d, add, in_place=True)[4]
    assert torch.equal(a, b)
    none = run_balance(z, idx, mask, 3, d, d, None)[4]
    assert torch.equal(none[~mask.to(none.device)], torch.zeros_like(none[~mask.to(none.device)]))
    assert torch.equal(a[~mask.to(a.device)].cpu(), add[~mask])  # tokens that do not count: as they were


def test_balance_gradient_that_is_not_finite_leaves_padding_alone():
    z, idx, mask = balance_inputs(300, 64, 6, 3, "random")
    d, add = torch.tensor([float("nan"), 1.0, float("inf")]), torch.randn(300, 64, generator=gen(1))
    out = run_balance(z, idx, mask, 3, d, d, add)[4].cpu()
    assert torch.equal(out[~mask], add[~mask])
    assert out[:100][mask[:100]].isnan().all() and out[100:200].isfinite().all()


def test_balance_same_bits_and_grid():
    z, idx, mask = balance_inputs(30000, 64, 6, 2, "random")
    d = torch.ones(2)
    a = run_balance(z, idx, mask, 2, d, d, None)
    moe.moe_set_grid_limit(5)
    try:
        b = run_balance(z, idx, mask, 2, d, d, None)
    finally:
        moe.moe_set_grid_limit(0)
    assert all(torch.equal(x, y) for x, y in zip(a[:5], b[:5]))


def test_balance_reports_bad_logits_and_picks():
    z, idx, _ = balance_inputs(200, 16, 2, 1, None)
    z[77, 3] = float("inf")
    d = torch.ones(1)
    *_, out, ws = run_balance(z, idx, None, 1, d, d, None)
    assert U.device_error(ws) == (moe.MOE_ERR_NONFINITE, 77)
    assert not out[77].any()
    z, idx, _ = balance_inputs(200, 16, 2, 1, None)
    idx[5, 1] = 16
    counts, *_, ws = run_balance(z, idx, None, 1, d, d, None)
    assert U.device_error(ws) == (moe.MOE_ERR_ARG, 5)
    assert int(counts.sum()) == 399


def test_balance_gradient_against_differences():
    T, E, k, B = 12, 6, 2, 2
    z, idx, mask = balance_inputs(T, E, k, B, None, seed=3)
    dl, dz = torch.tensor([0.7, -1.3]), torch.tensor([0.2, 0.5])
    got = U.np64(run_balance(z, idx, mask, B, dl, dz, None)[4])

    def f(zz):
        _, _, l, zl = S.balance_fwd(zz, idx.numpy(), B)
        return (l * dl.double().numpy()).sum() + (zl * dz.double().numpy()).sum()

    base = z.double().numpy()
    for t in range(T):
        for e in range(E):
            h = np.zeros_like(base)
            h[t, e] = 1e-5
            d = (f(base + h) - f(base - h)) / 2e-5
            assert abs(got[t, e] - d) <= 1e-5


# ----------------------------------------------------------- cross entropy
def xent_inputs(T, V, d, ignored=0.0, seed=0, sure=12.0):
    W = (torch.randn(V, d, generator=gen(seed)) * d ** -0.5).to(BF16)
    target = torch.randint(V, (T,), generator=gen(seed + 1))
    x = torch.randn(T, d, generator=gen(seed + 2)) + torch.rand(T, 1, generator=gen(seed + 3)) * sure * W[target].float()
    target[torch.rand(T, generator=gen(seed + 4)) < ignored] = -100
    return x.to(BF16), W, target


def logit_error(x, W):
    """Per token: bound on the error of its logits."""
    return (2.0 ** -18 + x.shape[1] * 2.0 ** -33) * (np.abs(x) @ np.abs(W).T).max(1)


def run_xent(x, W, target, backward=False, dloss=None, dlse=None, dx=None, dW=None, ws=None):
    T, d = x.shape
    V = W.shape[0]
    g = [put(t) for t in (x, W, target)]
    loss, lse = U.guarded_empty((T,), F32), U.guarded_empty((T,), F32)
    if ws is None:
        ws = workspace(moe.moe_xent_workspace_bytes(T, V, d, backward), moe.moe_xent_ws_init)
    moe.moe_xent_fwd(*g, loss, lse, ws)
    if not backward:
        return loss, lse, ws
    gx = None if dx is None else U.guarded_empty((T, d), dx, "dx")
    gW = None if dW is None else U.guarded_empty((V, d), dW, "dW")
    for t in (gx, gW):
        if t is not None:
            t.fill_(float("nan"))
    moe.moe_xent_bwd(*g, loss, lse, put(dloss), None if dlse is None else put(dlse), gx, gW, ws)
    return loss, lse, gx, gW, ws


def check_fwd(x, W, target, loss, lse):
    xn, Wn, tn = U.np64(x), U.np64(W), target.numpy().astype(np.int64)
    rl, rs = S.xent_fwd(xn, Wn, tn)
    dz = logit_error(xn, Wn)
    assert np.all(np.abs(U.np64(lse) - rs) <= dz + 2.0 ** -20 + 2.0 ** -23 * np.abs(rs))
    use = tn >= 0
    assert np.all(U.np64(loss)[~use] == 0)
    # log s and m - z are within an ulp each of what they stand for, and exp's error goes into s - 1 alone
    assert np.all(np.abs(U.np64(loss) - rl)[use] <= (2 * dz * np.minimum(1, rl) + 2.0 ** -20 * rl + 2.0 ** -22)[use])
    return dz, rs


def check_bwd(x, W, target, dloss, dlse, lse, dz, dx, dW, T, V):
    xn, Wn, tn = U.np64(x), U.np64(W), target.numpy().astype(np.int64)
    D = S.xent_grad(xn, Wn, tn, dloss.double().numpy(), None if dlse is None else dlse.double().numpy())
    g = np.where(tn >= 0, np.abs(dloss.double().numpy()), 0) + (0 if dlse is None else np.abs(dlse.double().numpy()))
    rel = (2 * dz + 2.0 ** -20 + 2.0 ** -23 * np.abs(lse))[:, None]
    # the target's own entry is off by that part of 1 - p, and by 2^-22 of the weight
    one = np.zeros_like(D)
    use = tn >= 0
    one[np.arange(T)[use], tn[use]] = (2.0 ** -22 * g)[use]
    for name, got, other, K, prod in (("dx", dx, Wn, V, lambda m: m @ np.abs(Wn)), ("dW", dW, xn, T, lambda m: m.T @ np.abs(xn))):
        if got is None:
            continue
        exact = D @ Wn if name == "dx" else D.T @ xn
        half = got.dtype == BF16
        run = 2.0 ** -23 * (-(-K // 16)) if half else 2.0 ** -18 + 3 * K * 2.0 ** -33
        bound = prod(np.abs(D) * (rel + (2.0 ** -8 if half else 2.0 ** -24) + run) + one)
        bound += (2.0 ** -8 if half else 2.0 ** -24) * np.abs(exact)
        err = np.abs(U.np64(got) - exact)
        assert np.all(err <= bound + 1e-30), (name, float((err / (bound + 1e-30)).max()))


@pytest.mark.parametrize("T,V,d", [(1, 1, 64), (1, 2, 64), (1, 1000, 256), (3, 255, 64), (5, 257, 128), (64, 5003, 320),
                                   (128, 300, 2048), (129, 513, 192), (300, 1000, 1024), (517, 4097, 576)])
def test_xent_fwd(T, V, d):
    x, W, target = xent_inputs(T, V, d, 0.2)
    loss, lse, ws = run_xent(x, W, target)
    check_fwd(x, W, target, loss, lse)
    assert U.device_error(ws) == (0, 0)


@pytest.mark.parametrize("wide", [I32, torch.int64])
@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, None), (None, BF16)],
                         ids=lambda t: "/".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("T,V,d", [(1, 1, 64), (1, 1000, 256), (65, 129, 64), (130, 1000, 192), (300, 2049, 320)])
def test_xent_bwd(T, V, d, types, wide):
    x, W, target = xent_inputs(T, V, d, 0.3, seed=T)
    target = target.to(wide)
    dloss = torch.rand(T, generator=gen(9)) / T
    dlse = torch.randn(T, generator=gen(10)) * 1e-3 if types[0] is not None else None
    loss, lse, dx, dW, ws = run_xent(x, W, target, True, dloss, dlse, *types)
    dz, rs = check_fwd(x, W, target, loss, lse)
    check_bwd(x, W, target, dloss, dlse, rs, dz, dx, dW, T, V)
    assert U.device_error(ws) == (0, 0)


def test_xent_pieces_of_the_vocabulary():
    """More columns than a piece holds: sums over pieces, the last one narrow."""
    T, V, d = 40000, 17000, 64
    x, W, target = xent_inputs(T, V, d, 0.1)
    dloss = torch.full((T,), 1.0 / T)
    for dt in (BF16, F32):
        loss, lse, dx, dW, ws = run_xent(x, W, target, True, dloss, None, dt, dt)
        # the formula on the GPU in fp64 (the oracle's arrays would not fit a test's time)
        xd, Wd, tg = x.to(U.DEV).double(), W.to(U.DEV).double(), target.to(U.DEV)
        z = xd @ Wd.t()
        ls = torch.logsumexp(z, 1)
        use = (tg >= 0).nonzero()[:, 0]
        assert (lse.double() - ls).abs().max() < 1e-4
        D = torch.exp(z - ls[:, None]) * torch.where(tg >= 0, 1.0 / T, 0.0)[:, None]
        D[use, tg[use]] -= 1.0 / T
        bar = 2.0 ** -8 * 1.5 if dt == BF16 else 2.0 ** -17
        for got, ref in ((dx, D @ Wd), (dW, D.t() @ xd)):
            assert ((got.double() - ref).norm() / ref.norm()).item() <= bar
        del z, D
        assert U.device_error(ws) == (0, 0)


@pytest.mark.parametrize("weight", [1 + 2.0 ** -8 * 0.999, 1 / 900])
def test_xent_even_weights_add_no_common_error(weight):
    """More tokens than D is kept in two values for, all of one weight: its rounding (half a step at worst, 2^-8) would be
    the error of every target's entry.  The entries beside them are small (V = 6000), so both gradients are off by
    little more than their own rounding, spread evenly up to half a step."""
    T, V, d = 900, 6000, 64
    x, W, target = xent_inputs(T, V, d, 0.1, sure=0.0)
    dloss = torch.full((T,), weight)
    loss, lse, dx, dW, ws = run_xent(x, W, target, True, dloss, None, BF16, BF16)
    D = S.xent_grad(U.np64(x), U.np64(W), target.numpy().astype(np.int64), dloss.double().numpy(), None)
    for got, exact in ((dx, D @ U.np64(W)), (dW, D.T @ U.np64(x))):
        assert U.relf(U.np64(got), exact) <= 2.0 ** -8 / 3 ** 0.5
    assert U.device_error(ws) == (0, 0)


def test_xent_loss_of_nearly_certain_tokens():
    """Losses of 1e-7 to 1 keep their relative precision: s - 1 is summed without the largest term's 1.  Off by 2 dz of
    itself for the logits, the exponentials' 2^-19 (2 + |z| ulp of small terms, |z| below 24) and 2^-24 for each of at most
    128 additions."""
    T, V, d = 2100, 500, 64
    x, W, target = xent_inputs(T, V, d, sure=30.0)
    loss, lse, ws = run_xent(x, W, target)
    rl, _ = S.xent_fwd(U.np64(x), U.np64(W), target.numpy())
    dz = logit_error(U.np64(x), U.np64(W))
    some = (rl > 1e-7) & (rl < 1)
    assert some.sum() > 500
    assert np.all(np.abs(U.np64(loss) - rl)[some] <= ((2 * dz + 2.0 ** -19 + 2.0 ** -17) * rl)[some])


@pytest.mark.parametrize("kind", ["none of the sample", "lse alone", "far apart", "tiny", "signs"])
def test_xent_units_of_odd_weights(kind):
    """D's rows are kept in units near one number that a sample of tokens sets: it may find nothing, or numbers whose
    squares fp32 does not hold."""
    T, V, d = 2100, 500, 64
    x, W, target = xent_inputs(T, V, d, 0.1)
    dloss, dlse = torch.rand(T, generator=gen(9)) + 0.5, None
    if kind == "none of the sample":  # tokens spread evenly over all are looked at
        target[(torch.arange(1024) * T) // 1024] = -1
    elif kind == "lse alone":
        dloss, dlse = torch.zeros(T), torch.randn(T, generator=gen(10))
    elif kind == "far apart":
        dloss *= 10.0 ** torch.randint(-25, 26, (T,), generator=gen(11)).float()
    elif kind == "tiny":
        dloss *= 1e-30
    else:
        dloss *= torch.randint(0, 2, (T,), generator=gen(11)) * 2.0 - 1.0
    loss, lse, dx, dW, ws = run_xent(x, W, target, True, dloss, dlse, BF16, BF16)
    dz, rs = check_fwd(x, W, target, loss, lse)
    check_bwd(x, W, target, dloss, dlse, rs, dz, dx, dW, T, V)
    assert U.device_error(ws) == (0, 0)


def test_xent_certain_tokens_keep_their_precision():
    """Targets so likely that lse and the logit agree to many digits: loss and gradient are those of the rest."""
    T, V, d = 16, 700, 256
    x, W, target = xent_inputs(T, V, d, sure=0.0)
    x = (x.float() + 40.0 * W[target].float()).to(BF16)
    loss, lse, dx, dW, ws = run_xent(x, W, target, True, torch.ones(T), None, F32, F32)
    rl, _ = S.xent_fwd(U.np64(x), U.np64(W), target.numpy())
    assert rl.max() < 1e-6
    dz = logit_error(U.np64(x), U.np64(W))
    assert np.all(np.abs(U.np64(loss) - rl) <= 2 * dz * rl + 2.0 ** -22)


def test_xent_rows_without_weight_add_nothing():
    """NaN and infinities in tokens that do not count stay there."""
    T, V, d = 200, 777, 128
    x, W, target = xent_inputs(T, V, d, 0.5)
    off = target < 0
    ref = run_xent(torch.where(off[:, None], torch.zeros((), dtype=BF16), x), W, target, True, torch.ones(T), None, F32, F32)
    x[off] = float("nan")
    x[off.nonzero()[0, 0]] = float("inf")
    loss, lse, dx, dW, ws = run_xent(x, W, target, True, torch.ones(T), None, F32, F32)
    assert torch.equal(dW, ref[3]) and torch.equal(dx, ref[2]) and torch.equal(loss, ref[0])
    assert not dx[off.to(dx.device)].any()
    # all of them: nothing left
    *_, dx, dW, ws = run_xent(x, W, torch.full((T,), -1), True, torch.ones(T), None, BF16, BF16)
    assert not dx.any() and not dW.any()


def test_xent_target_outside_the_vocabulary():
    T, V, d = 10, 100, 64
    x, W, target = xent_inputs(T, V, d)
    target[7] = V
    loss, lse, dx, dW, ws = run_xent(x, W, target, True, torch.ones(T), None, F32, F32)
    assert U.device_error(ws) == (moe.MOE_ERR_ARG, 7)
    assert loss[7] == 0 and not dx[7].any()


def test_xent_same_bits_grid_graph_and_stream():
    T, V, d = 300, 3001, 256
    x, W, target = xent_inputs(T, V, d, 0.2)
    dloss = torch.full((T,), 1.0 / T)
    ref = run_xent(x, W, target, True, dloss, None, BF16, F32)[:4]
    moe.moe_set_grid_limit(3)
    try:
        got = run_xent(x, W, target, True, dloss, None, BF16, F32)[:4]
    finally:
        moe.moe_set_grid_limit(0)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    g = [put(t) for t in (x, W, target)]
    dl = put(dloss)
    out = [torch.empty_like(t) for t in ref]
    ws = moe.alloc_xent_workspace(T, V, d)
    side = torch.cuda.Stream()

    def step():
        moe.moe_xent_fwd(*g, out[0], out[1], ws)
        moe.moe_xent_bwd(*g, out[0], out[1], dl, None, out[2], out[3], ws)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_xent_gradient_against_differences():
    T, V, d = 4, 9, 64
    x, W, target = xent_inputs(T, V, d, sure=2.0)
    target[1] = -1
    dl, dh = torch.tensor([1.0, 0.5, -2.0, 0.25]), torch.tensor([0.1, 0.3, 0.0, -0.7])
    *_, dx, dW, ws = run_xent(x, W, target, True, dl, dh, F32, F32)

    def f(xx, WW):
        l, s = S.xent_fwd(xx, WW, target.numpy())
        return (l * dl.double().numpy()).sum() + (s * dh.double().numpy()).sum()

    xn, Wn = U.np64(x), U.np64(W)
    rng = np.random.default_rng(0)
    for _ in range(40):
        ux, uW = rng.standard_normal(xn.shape), rng.standard_normal(Wn.shape)
        d = (f(xn + 1e-5 * ux, Wn + 1e-5 * uW) - f(xn - 1e-5 * ux, Wn - 1e-5 * uW)) / 2e-5
        got = (U.np64(dx) * ux).sum() + (U.np64(dW) * uW).sum()
        size = np.abs(U.np64(dx) * ux).sum() + np.abs(U.np64(dW) * uW).sum()
        assert abs(got - d) <= 2.0 ** -14 * size


# --------------------------------------------------------- orthogonalised
def run_ortho(G, steps=5, ws=None):
    mats, rows, cols = G.shape if G.dim() == 3 else (1, *G.shape)
    if ws is None:
        ws = workspace(moe.moe_orthogonalize_workspace_bytes(mats, rows, cols), moe.moe_orthogonalize_ws_init)
    out = U.guarded_empty(tuple(G.shape), BF16, "O")
    out.fill_(float("nan"))
    moe.moe_orthogonalize(put(G), out, steps, ws)
    return out, ws


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("mats,rows,cols,steps", [
    (1, 1, 1, 5), (1, 1, 100, 5), (3, 100, 1, 5), (2, 7, 9, 1), (2, 63, 65, 5), (1, 64, 2048, 5), (3, 128, 128, 5),
    (2, 129, 257, 5), (2, 257, 129, 5), (2, 333, 1001, 3), (2, 1001, 333, 5), (1, 300, 300, 5), (1, 520, 264, 5),
    (1, 700, 520, 2), (5, 256, 512, 5), (1, 16, 3000, 5), (1, 128, 5000, 5), (2, 3001, 100, 5), (130, 20, 30, 5),
    (40, 128, 300, 5), (1, 128, 9000, 1)])
def test_orthogonalize(mats, rows, cols, steps, dt):
    G = (torch.randn(mats, rows, cols, generator=gen(1)) * 1e-3).to(dt)
    G[0] += (torch.randn(rows, 1, generator=gen(2)) @ torch.randn(1, cols, generator=gen(3)) * 2e-3).to(dt)
    got, ws = run_ortho(G, steps)
    assert U.device_error(ws) == (0, 0)
    for i in sorted({0, mats // 2, mats - 1}):
        ref = S.orthogonalize(U.np64(G[i]), steps)
        # what fp16 between the products leaves, and the result's rounding to bf16
        bar = S.orthogonalize_spread(U.np64(G[i]), steps) + 2.0 ** -8
        assert U.relf(U.np64(got[i]), ref) <= bar
        if min(rows, cols) >= 64:
            # the same roundings in other places at most: where fp32 sums move a value over the middle of two
            like = U.relf(S.orthogonalize_rounded(U.np64(G[i]), steps), ref)
            assert U.relf(U.np64(got[i]), ref) <= 1.25 * like + 2.0 ** -12
    if steps == 5 and min(rows, cols) > 1:
        s = np.linalg.svd(U.np64(got[0]), compute_uv=False)
        assert s.max() < 1.3


def test_orthogonalize_scales_zeros_and_bad_matrices():
    rows, cols = 96, 160
    base = torch.randn(rows, cols, generator=gen(4))
    scales = [1.0, 0.0, 1e-20, 1e15, 1e-9, 1e-4]
    G = torch.stack([base * s for s in scales] + [base.clone(), base.clone()])
    G[-2, 3, 5] = float("nan")
    G[-1, 90, 159] = float("inf")
    got, ws = run_ortho(G)
    for i, s in enumerate(scales):
        ref = S.orthogonalize(U.np64(G[i]), 5)
        if s == 0.0:
            assert not got[i].any()
        else:
            assert U.relf(U.np64(got[i]), ref) <= S.orthogonalize_spread(U.np64(G[i]), 5) + 2.0 ** -8, s
    assert got[-2:].isnan().all()
    assert U.device_error(ws) == (0, 0)


@pytest.mark.parametrize("rows,cols", [(96, 160), (300, 200)])
@pytest.mark.parametrize("steps,top", [(1, 1e-9), (5, 1e-9), (10, 2e-14), (16, 1e-17)])
def test_orthogonalize_small_norms(rows, cols, steps, top):
    """Norms far below eps: X starts small and grows 3.4-fold a step, through all of fp16's range.  (Scales at which the
    last step just comes near 1: further steps map [0.7, 1.2] into itself with slopes above 1 and amplify any error.)"""
    scales = [top, top / 30, top / 1000, top * 1e-6]
    base = torch.randn(rows, cols, generator=gen(7))
    got, ws = run_ortho(torch.stack([base * s for s in scales]), steps)
    for i, s in enumerate(scales):
        g = U.np64(base * s)
        assert U.relf(U.np64(got[i]), S.orthogonalize(g, steps)) <= 2.0 ** -8, s  # bf16's rounding and fp16's
    assert U.device_error(ws) == (0, 0)


def test_orthogonalize_same_bits_grid_graph():
    G = torch.randn(3, 300, 500, generator=gen(5))
    ref, _ = run_ortho(G)
    moe.moe_set_grid_limit(3)
    try:
        got, ws = run_ortho(G)
    finally:
        moe.moe_set_grid_limit(0)
    assert torch.equal(ref, got)
    g, out = put(G), torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out, 5, ws)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref, out)
    one, _ = run_ortho(G[1])  # a matrix by itself: the same
    assert torch.equal(ref[1], one)


@pytest.mark.parametrize("rows,cols", [(1300, 1400), (1401, 1290)])
def test_orthogonalize_many_large(rows, cols):
    """Enough tiles for CTA pairs, whose symmetric products are stored from the diagonal on only; an empty matrix and a
    bad one between the others leave them alone."""
    mats = 10
    G = torch.randn(mats, rows, cols, generator=gen(6))
    G[3] = 0
    G[7, 5, 5] = float("nan")
    got, ws = run_ortho(G)
    assert U.device_error(ws) == (0, 0)
    assert not got[3].any() and got[7].isnan().all()
    for i in (0, 9):
        g = U.np64(G[i])
        ref = S.orthogonalize(g, 5)
        assert U.relf(U.np64(got[i]), ref) <= 1.25 * U.relf(S.orthogonalize_rounded(g, 5), ref) + 2.0 ** -12
    again, _ = run_ortho(G, ws=ws)
    assert torch.equal(got[:7], again[:7]) and torch.equal(got[8:], again[8:])


@pytest.mark.parametrize("mats,rows,cols,rank", [(1, 64, 2048, 5), (2, 300, 128, 9), (1, 500, 700, 20), (1, 700, 500, 100),
                                                 (9, 1300, 1400, 60)])
def test_orthogonalize_of_low_rank(mats, rows, cols, rank):
    """Gradients of an expert that saw few tokens: the steps raise what rounding leaves beside them 485-fold, so X carries
    the bits below fp16's too.  With fp16 alone these come out up to 4e-2 of their norm off."""
    G = (torch.randn(mats, rows, rank, generator=gen(1)) @ torch.randn(mats, rank, cols, generator=gen(2))) * 1e-4
    got, ws = run_ortho(G)
    for i in {0, mats - 1}:
        g = U.np64(G[i])
        ref = S.orthogonalize(g, 5)
        like = U.relf(S.orthogonalize_rounded(g, 5), ref)
        assert like <= 4e-3 and U.relf(U.np64(got[i]), ref) <= 1.25 * like + 2.0 ** -12
    assert U.device_error(ws) == (0, 0)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("mats,rows,cols", [(40, 2, 2), (40, 4, 4), (300, 8, 8), (40, 17, 16), (40, 32, 32), (3, 5, 700),
                                            (2, 2500, 32), (1000, 31, 64), (20, 30, 1500), (1, 16, 20000), (7, 48, 600), (200, 45, 47)])
def test_orthogonalize_small_sides_keep_two_values(mats, rows, cols, dt):
    """Sides up to 48, many of them with a singular value near 0: X, A and the polynomial have 22 bits and their sums 24
    (2^-21 together), so the result is off by little more than its own rounding: half a step of bf16 at most, 2^-8, and
    2^-8 / sqrt(3) where it is spread evenly."""
    G = (torch.randn(mats, rows, cols, generator=gen(8)) * 1e-3).to(dt)
    got, ws = run_ortho(G)
    assert U.device_error(ws) == (0, 0)
    errs = []
    for i in range(0, mats, max(1, mats // 40)):
        g = U.np64(G[i])
        errs.append(U.relf(U.np64(got[i]), S.orthogonalize(g, 5)))
        assert errs[-1] <= S.orthogonalize_spread(g, 5, unit=2.0 ** -21) + 2.0 ** -8
    assert np.median(errs) <= 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("rows,cols", [(6, 20), (33, 40), (700, 12), (1, 5)])
@pytest.mark.parametrize("steps", [1, 5])
def test_orthogonalize_small_sides_scales_zeros_and_bad_matrices(rows, cols, steps):
    base = torch.randn(rows, cols, generator=gen(4))
    scales = [1.0, 0.0, 1e-20, 1e15, 1e-9, 1e-4, 3e-17]
    G = torch.stack([base * s for s in scales] + [base.clone(), base.clone()])
    G[-2, 0, 3] = float("nan")
    G[-1, rows - 1, cols - 1] = -float("inf")
    got, ws = run_ortho(G, steps)
    for i, s in enumerate(scales):
        g = U.np64(G[i])
        if s == 0.0:
            assert not got[i].any()
        else:
            assert U.relf(U.np64(got[i]), S.orthogonalize(g, steps)) <= S.orthogonalize_spread(g, steps, unit=2.0 ** -21) + 2.0 ** -8, s
    assert got[-2:].isnan().all()
    again, _ = run_ortho(G[2:4], steps)  # other matrices, another workspace: the same bits
    assert torch.equal(got[2:4], again)
    g, out = put(G), torch.empty_like(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out, steps, ws)
    for _ in range(2):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[:-2], out[:-2]) and out[-2:].isnan().all()


def test_orthogonalize_offsets_past_32_bits():
    mats, m = 8300, 512
    assert mats * m * m > 2 ** 31
    G = torch.empty(mats, m, m, dtype=BF16, device=U.DEV)
    G.normal_(generator=torch.Generator(device=U.DEV).manual_seed(1))
    out = torch.empty_like(G)
    ws = moe.alloc_orthogonalize_workspace(mats, m, m)
    moe.moe_orthogonalize(G, out, 5, ws)
    for i in (0, 4096, 8191, 8192, mats - 1):
        g = U.np64(G[i])
        ref = S.orthogonalize(g, 5)
        assert U.relf(U.np64(out[i]), ref) <= 1.25 * U.relf(S.orthogonalize_rounded(g, 5), ref) + 2.0 ** -12
    assert moe.moe_get_device_error(ws) == (0, 0)


def shifted(shape, dt):
    """A tensor that begins 16 bytes past a 32-byte boundary."""
    n = 1
    for v in shape:
        n *= v
    k = 16 // torch.empty(0, dtype=dt).element_size()
    t = torch.empty(n + k, dtype=dt, device=U.DEV)[k:].view(shape)
    assert t.data_ptr() % 32 == 16
    return t


def test_outputs_between_32_byte_boundaries():
    T, V, d = 300, 1000, 192
    x, W, target = xent_inputs(T, V, d, 0.2)
    for dt in (BF16, F32):
        ref = run_xent(x, W, target, True, torch.ones(T), None, dt, dt)
        g = [t.to(U.DEV) for t in (x, W, target)]
        ws = moe.alloc_xent_workspace(T, V, d)
        dx, dW = shifted((T, d), dt), shifted((V, d), dt)
        moe.moe_xent_bwd(*g, ref[0], ref[1], torch.ones(T, device=U.DEV), None, dx, dW, ws)
        assert torch.equal(dx, ref[2]) and torch.equal(dW, ref[3])
    for mats, rows, cols in ((3, 300, 320), (2, 40, 64), (2, 300, 301)):
        G = torch.randn(mats, rows, cols, generator=gen(8))
        ref, ws = run_ortho(G)
        out, g = shifted((mats, rows, cols), BF16), shifted((mats, rows, cols), F32)
        g.copy_(G)
        moe.moe_orthogonalize(g, out, 5, ws)
        assert torch.equal(out, ref)


@pytest.mark.parametrize("T,V,d,dt", [(5000, 100, 64, F32), (5000, 100, 64, BF16), (64, 30000, 64, F32), (1, 20000, 512, F32),
                                      (129, 2, 64, F32), (700, 129, 1088, BF16)])
def test_xent_split_sums(T, V, d, dt):
    """Few tiles and long sums: the products' K is shared by several CTAs."""
    x, W, target = xent_inputs(T, V, d, 0.1, seed=3)
    dloss = torch.rand(T, generator=gen(9)) / T
    loss, lse, dx, dW, ws = run_xent(x, W, target, True, dloss, None, dt, dt)
    dz, rs = check_fwd(x, W, target, loss, lse)
    check_bwd(x, W, target, dloss, None, rs, dz, dx, dW, T, V)


def test_xent_offsets_past_32_bits():
    """Rows of D past 2^31 elements."""
    T, V, d = 270000, 8192, 64
    gd = torch.Generator(device=U.DEV).manual_seed(2)
    x = torch.empty(T, d, dtype=BF16, device=U.DEV).normal_(generator=gd)
    W = torch.empty(V, d, dtype=BF16, device=U.DEV).normal_(0, 0.1, generator=gd)
    target = torch.randint(V, (T,), generator=gd, device=U.DEV)
    loss, lse = (torch.empty(T, device=U.DEV) for _ in range(2))
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    w = torch.zeros(T, device=U.DEV)
    w[-1000:] = 1.0                          # what the last rows give is all there is of dW
    ws = moe.alloc_xent_workspace(T, V, d)
    moe.moe_xent_fwd(x, W, target, loss, lse, ws)
    moe.moe_xent_bwd(x, W, target, loss, lse, w, None, dx, dW, ws)
    assert moe.moe_get_device_error(ws) == (0, 0)
    xd, Wd, tg = x[-1000:].double(), W.double(), target[-1000:]
    z = xd @ Wd.t()
    D = torch.softmax(z, 1)
    assert (lse[-1000:].double() - torch.logsumexp(z, 1)).abs().max() < 1e-4
    D[torch.arange(1000, device=U.DEV), tg] -= 1.0
    assert not dx[:-1000].any()
    for got, ref in ((dx[-1000:], D @ Wd), (dW, D.t() @ xd)):
        assert ((got.double() - ref).norm() / ref.norm()).item() <= 1.5 * 2.0 ** -8


def test_two_calls_at_once_on_their_own_workspaces():
    T, V, d = 200, 5000, 256
    x, W, target = xent_inputs(T, V, d, 0.2)
    dloss = torch.ones(T) / T
    ref = run_xent(x, W, target, True, dloss, None, BF16, BF16)[:4]
    Gm = torch.randn(6, 700, 600, generator=gen(3))
    oref, _ = run_ortho(Gm)
    g, gd, gm = [t.to(U.DEV) for t in (x, W, target)], dloss.to(U.DEV), Gm.to(U.DEV)
    wx, wo = moe.alloc_xent_workspace(T, V, d), moe.alloc_orthogonalize_workspace(6, 700, 600)
    out, o = [torch.empty_like(t) for t in ref], torch.empty_like(oref)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        moe.moe_xent_fwd(*g, out[0], out[1], wx, stream=a)
        moe.moe_orthogonalize(gm, o, 5, wo, stream=b)
        moe.moe_xent_bwd(*g, out[0], out[1], gd, None, out[2], out[3], wx, stream=a)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(ref, out)) and torch.equal(o, oref)


def test_balance_graph_and_reuse_of_the_layers_workspace():
    """Between the layer's forward and backward, captured and replayed: the layer's results stay as they were."""
    from combine_fp32_softmax_gb300.configs import MoEConfig
    from combine_fp32_softmax_gb300.inputs import make_layer_inputs
    c = MoEConfig("b", 640, 128, 192, 8, 2, S=1)
    inp = make_layer_inputs(c, seed=0)
    g = U.to_dev(inp)
    plain, ws = U.run_layer(c, g)
    plain = {n: t.clone() for n, t in plain.items()}
    out = U.empty_outputs(c)
    counts, mean_p = U.guarded_empty((2, 8), I32), U.guarded_empty((2, 8), F32)
    loss, zloss = U.guarded_empty((2,), F32), U.guarded_empty((2,), F32)
    dl, total = torch.full((2,), 0.01, device=U.DEV), U.guarded_empty((c.T, c.E), F32)

    def step():
        moe.moe_layer_fwd(c, g["logits"], g["x"], g["W1"], g["W3"], g["W2"], out["y"], out["topk_idx"], out["topk_w"], ws)
        moe.moe_balance_fwd(c, g["logits"], out["topk_idx"], None, counts, mean_p, loss, zloss, ws)
        moe.moe_layer_bwd(c, g["dy"], g["logits"], g["x"], g["W1"], g["W3"], g["W2"], out["topk_idx"], out["topk_w"], ws,
                          out["dx"], out["dlogits"], out["dW1"], out["dW3"], out["dW2"])
        moe.moe_balance_bwd(c, g["logits"], counts, None, dl, dl, out["dlogits"], total, ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(plain[n], out[n]) for n in plain)
    ref = S.balance_bwd(inp.logits.numpy(), plain["topk_idx"].cpu().numpy(), 2, np.full(2, 0.01), np.full(2, 0.01),
                        plain["dlogits"].cpu().numpy())
    assert np.abs(U.np64(total) - ref).max() <= 2.0 ** -22 * np.abs(ref).max()
    assert U.device_error(ws) == (0, 0)


def test_balance_more_sequences_than_counters():
    z, idx, mask = balance_inputs(70 * 100, 32, 4, 70, "random")
    d = torch.ones(70)
    counts, mean_p, loss, *_ = run_balance(z, idx, mask, 70, d, d, None)
    rc, rp, rl, _ = S.balance_fwd(np.nan_to_num(z.numpy()), np.where(idx.numpy() < 32, idx.numpy(), 0), 70, mask.numpy())
    assert np.array_equal(counts.cpu().numpy(), rc) and np.allclose(U.np64(loss), rl, rtol=1e-5)


def test_balance_of_millions_of_tokens():
    """A block's sums stay short however many tokens there are."""
    T, E, k = 2_000_003, 8, 2
    z, idx, _ = balance_inputs(T, E, k, 1, None, scale=2.0)
    d = torch.ones(1)
    counts, mean_p, loss, zloss, out, ws = run_balance(z, idx, None, 1, d, d, None)
    rc, rp, rl, rz = S.balance_fwd(z.numpy(), idx.numpy(), 1)
    assert np.array_equal(counts.cpu().numpy(), rc)
    # p to 4e-6, at most 4096 / 16 / 32 of them on a lane and 16 warps added in fp32
    assert np.abs(U.np64(mean_p) - rp).max() <= (4e-6 + 24 * 2.0 ** -24) * rp.max()
    assert np.allclose(U.np64(loss), rl, rtol=1e-5) and np.allclose(U.np64(zloss), rz, rtol=1e-5)
    assert U.device_error(ws) == (0, 0)


FIRST_CALLS = """
import torch
from combine_fp32_softmax_gb300 import moe
dev, bf, f = "cuda", torch.bfloat16, torch.float32
T, V, d = 300, 700, 128
x, W = torch.randn(T, d, device=dev).to(bf), torch.randn(V, d, device=dev).to(bf)
t, g = torch.randint(V, (T,), device=dev), torch.ones(T, device=dev)
loss, lse = torch.zeros(T, device=dev), torch.zeros(T, device=dev)
dx, dW = torch.zeros(T, d, device=dev), torch.zeros(V, d, dtype=bf, device=dev)
G = [torch.randn(2, n, 200, device=dev) for n in (40, 300)]
O = [torch.zeros_like(m, dtype=bf) for m in G]
xws, ows = moe.alloc_xent_workspace(T, V, d), [moe.alloc_orthogonalize_workspace(*m.shape) for m in G]
def step():
    moe.moe_xent_fwd(x, W, t, loss, lse, xws)
    moe.moe_xent_bwd(x, W, t, loss, lse, g, None, dx, dW, xws)
    for m, o, w in zip(G, O, ows):
        moe.moe_orthogonalize(m, o, 5, w)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [v.clone() for v in (loss, lse, dx, dW, *O)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and a.isfinite().all() and a.any() for a, b in zip(got, (loss, lse, dx, dW, *O)))
print("same")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream: nothing is kept in a workspace from one call to the next."""
    cases = []
    ws = moe.alloc_xent_workspace(700, 3000, 256)
    for T, V, d in ((700, 3000, 256), (40, 2999, 128)):
        x, W, target = xent_inputs(T, V, d, 0.2, seed=T)
        dloss = torch.ones(T) / T
        ref = run_xent(x, W, target, True, dloss, None, BF16, F32)[:4]
        g, dl, out = [t.to(U.DEV) for t in (x, W, target)], dloss.to(U.DEV), [torch.empty_like(t) for t in ref]
        assert moe.moe_xent_workspace_bytes(T, V, d) <= ws.nbytes

        def step(g=g, dl=dl, out=out):
            moe.moe_xent_fwd(*g, out[0], out[1], ws)
            moe.moe_xent_bwd(*g, out[0], out[1], dl, None, out[2], out[3], ws)

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        cases.append((graph, ref, out, g, dl))  # a graph does not keep its inputs alive
    for _ in range(3):
        for graph, ref, out, *_ in cases:
            for t in out:
                t.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for _, ref, out, *_ in cases for a, b in zip(ref, out))
