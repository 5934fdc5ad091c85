"""The ends of a training step on the GPU, beside test_gpu_step_ends.py: the forms that only large products take, types that
differ, long sums, limits that a result may not depend on.

Tolerances are those of test_gpu_step_ends.py, or are derived at the test."""
import functools
import json
import os
import re
import tempfile

import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300 import moe
from oracle import step_oracle as S
from tests import gpu_util as U
from tests import test_gpu_step_ends as E

pytestmark = pytest.mark.gpu
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def profiled(fn):
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU, torch.profiler.ProfilerActivity.CUDA]) as p:
        fn()
        torch.cuda.synchronize()
    with tempfile.TemporaryDirectory() as d:
        path = os.path.join(d, "trace.json")
        p.export_chrome_trace(path)
        with open(path) as f:
            events = json.load(f)["traceEvents"]
    return [(e["name"], int(np.prod(e["args"]["grid"]))) for e in events if e.get("cat") == "kernel"]


@functools.cache
def profiler_works():
    """The first time it is used it may see nothing."""
    return any(profiled(lambda: torch.ones(4, device=U.DEV) + 1) for _ in range(3))


def launches(fn):
    """(name, CTAs) of the kernels that fn launches; None where they cannot be listed."""
    if profiler_works():
        return profiled(fn)
    fn()
    return None


def forms(seen, op):
    """How many CTAs share a tile in the launches of an operation of the dense products."""
    return [int(m.group(1)) for n, _ in seen if (m := re.search(rf"dense_kernel<.*{op}, ?(?:\(int\))?([12])>", n))]


def product(kind, number):
    return rf"{kind}<(?:\((?:bool|int)\))?{number}>"


DX, DW = product("ProdOp", "(?:true|1)"), product("ProdOp", "(?:false|0)")


# ----------------------------------------------------------- cross entropy
def check_xent(x, W, target, dloss, dlse, loss, lse, dx, dW):
    """The bounds of test_gpu_step_ends.check_fwd and check_bwd, in fp64 on the GPU."""
    xd, Wd, tg = x.to(U.DEV).double(), W.to(U.DEV).double(), target.to(U.DEV).long()
    T, V, d = len(xd), len(Wd), xd.shape[1]
    dz = (2.0 ** -18 + d * 2.0 ** -33) * (xd.abs() @ Wd.abs().t()).amax(1)
    z = xd @ Wd.t()
    rs = torch.logsumexp(z, 1)
    rows = (tg >= 0).nonzero()[:, 0]
    at = (rows, tg[rows])
    p = z.sub_(rs[:, None]).exp_()
    others = (p[rows].sum(1) - p[at]) if V * T < 2 ** 27 else 1 - p[at]
    rl = torch.zeros(T, dtype=torch.float64, device=U.DEV)
    rl[rows] = -torch.log(p[at])
    assert ((lse.double() - rs).abs() <= dz + 2.0 ** -20 + 2.0 ** -23 * rs.abs()).all()
    assert not loss[tg < 0].any()
    assert ((loss.double() - rl).abs()[rows] <= (2 * dz * rl.clamp(max=1) + 2.0 ** -20 * rl + 2.0 ** -22)[rows]).all()
    g = torch.where(tg >= 0, dloss.to(U.DEV).double(), 0.0)
    h = torch.zeros_like(g) if dlse is None else dlse.to(U.DEV).double()
    pt = p[at].clone()
    D = p.mul_((g + h)[:, None])
    D[at] = h[rows] * pt - g[rows] * others
    rel = 2 * dz + 2.0 ** -20 + 2.0 ** -23 * rs.abs()
    for name, got, K in (("dx", dx, V), ("dW", dW, T)):
        if got is None:
            continue
        half = got.dtype == BF16
        run = 2.0 ** -23 * (-(-K // 16)) if half else 2.0 ** -18 + 3 * K * 2.0 ** -33
        exact = D @ Wd if name == "dx" else D.t() @ xd
        B = D.abs().mul_((rel + (2.0 ** -8 if half else 2.0 ** -24) + run)[:, None])
        B[at] += 2.0 ** -22 * (g.abs() + h.abs())[rows]
        bound = (B @ Wd.abs() if name == "dx" else B.t() @ xd.abs()) + (2.0 ** -8 if half else 2.0 ** -24) * exact.abs()
        del B
        err = (got.double() - exact).abs()
        assert (err <= bound + 1e-30).all(), (name, float((err / (bound + 1e-30)).max()))


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)], ids=lambda t: "/".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("T,V,d", [(1300, 6000, 832), (2500, 9001, 1024)])
def test_xent_on_cta_pairs(T, V, d, types):
    """Logits in several runs of sums, uneven ones among them, and both products on pairs of CTAs, a ring that goes round
    many times, ends that are no whole tiles; dx of the smaller case with its K split."""
    x, W, target = E.xent_inputs(T, V, d, 0.2, seed=T)
    dloss, dlse = torch.rand(T, generator=E.gen(9)) / T, torch.randn(T, generator=E.gen(10)) * 1e-5
    out = []
    seen = launches(lambda: out.extend(E.run_xent(x, W, target, True, dloss, dlse, *types)))
    for op in ("StatsOp", "GradOp", DX, DW):
        assert seen is None or set(forms(seen, op)) == {2}, (op, seen)
    loss, lse, dx, dW, ws = out
    check_xent(x, W, target, dloss, dlse, loss, lse, dx, dW)
    assert U.device_error(ws) == (0, 0)


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (BF16, F32)], ids=lambda t: "/".join(str(x)[6:] for x in t))
def test_xent_pieces_on_cta_pairs(types):
    """More columns than a piece holds, each piece's products with a long K."""
    T, V, d = 33000, 8449, 832
    x, W, target = E.xent_inputs(T, V, d, 0.1)
    dloss = torch.rand(T, generator=E.gen(9)) / T
    out = []
    seen = launches(lambda: out.extend(E.run_xent(x, W, target, True, dloss, None, *types)))
    for op in ("GradOp", DX, DW):
        assert seen is None or len(forms(seen, op)) > 1, (op, seen)
        # four values of D make pieces of 2048 columns, of which dW's tiles are too few for pairs
        assert seen is None or 2 in forms(seen, op) or (op == DW and types == (BF16, F32)), (op, seen)
    loss, lse, dx, dW, ws = out
    check_xent(x, W, target, dloss, None, loss, lse, dx, dW)
    assert U.device_error(ws) == (0, 0)


@pytest.mark.parametrize("types", [(BF16, F32), (F32, BF16)], ids=lambda t: "/".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("weight", [1 + 2.0 ** -8 * 0.999, 1 / 900])
def test_xent_even_weights_with_types_that_differ(weight, types):
    """As with both gradients in bf16: the rounding of D to bf16 adds nothing that all tokens have in common.  The fp32
    gradient keeps its own precision: 2^-18 of its terms' magnitudes, which are the target's and, together, about as much
    again."""
    T, V, d = 900, 6000, 64
    x, W, target = E.xent_inputs(T, V, d, 0.1, sure=0.0)
    dloss = torch.full((T,), weight)
    loss, lse, dx, dW, ws = E.run_xent(x, W, target, True, dloss, None, *types)
    D = S.xent_grad(U.np64(x), U.np64(W), target.numpy().astype(np.int64), dloss.double().numpy(), None)
    for got, exact in ((dx, D @ U.np64(W)), (dW, D.T @ U.np64(x))):
        assert U.relf(U.np64(got), exact) <= (2.0 ** -8 / 3 ** 0.5 if got.dtype == BF16 else 2.0 ** -17)
    assert U.device_error(ws) == (0, 0)


def test_xent_long_sums_in_bf16():
    """2^22 tokens, all alike, so every term of a sum has one sign and what the tensor core's additions cut off adds up.
    What is left is the rounding of the result, half a step of bf16 at most and 2^-8 / sqrt(3) where it is spread evenly,
    at the target (whose entry in D is exact) and that of D's entry (2^-8 at most) elsewhere; and 2^-10 for the sums, which
    end after 131,072 terms."""
    T, V, d = 1 << 22, 8448, 64
    gd = torch.Generator(device=U.DEV).manual_seed(3)
    x = torch.empty(1, d, dtype=BF16, device=U.DEV).normal_(generator=gd).expand(T, d).contiguous()
    W = torch.empty(V, d, dtype=BF16, device=U.DEV).normal_(0, 0.05, generator=gd)
    target = torch.full((T,), 5, dtype=I32, device=U.DEV)
    dloss = torch.full((T,), 1.0, device=U.DEV)
    loss, lse = (torch.empty(T, device=U.DEV) for _ in range(2))
    dW = torch.empty_like(W)
    ws = moe.alloc_xent_workspace(T, V, d)
    moe.moe_xent_fwd(x, W, target, loss, lse, ws)
    moe.moe_xent_bwd(x, W, target, loss, lse, dloss, None, None, dW, ws)
    assert moe.moe_get_device_error(ws) == (0, 0)
    D = torch.softmax(x[0].double() @ W.double().t(), 0)
    D[5] -= 1.0
    ref = T * D[:, None] * x[:1].double()
    err = (dW.double() - ref).norm(dim=1) / ref.norm(dim=1)
    assert err[5].item() <= 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -10
    assert err.max().item() <= 2.0 ** -8 * (1 + 1 / 3 ** 0.5) + 2.0 ** -10


def test_xent_units_are_the_same_in_both_kernels():
    """A row of D is divided by its unit in one kernel and dx multiplied by it in another.  The unit comes of a rounding
    to bf16, so where the two differ in a last bit a whole row of dx is off by up to 2^-7; with a gradient of lse beside the
    loss's, over enough rows that some lie near the middle of two bf16 values.  Every row: its own rounding (half a step of
    bf16 at most) and D's, 2^-8 of each value against the row's sum of magnitudes."""
    T, V, d = 1 << 20, 256, 64
    gd = torch.Generator(device=U.DEV).manual_seed(4)
    x = torch.empty(T, d, dtype=BF16, device=U.DEV).normal_(generator=gd)
    W = torch.empty(V, d, dtype=BF16, device=U.DEV).normal_(0, 0.05, generator=gd)
    target = torch.randint(V, (T,), generator=gd, device=U.DEV)
    dloss = torch.rand(T, generator=gd, device=U.DEV) + 0.5
    dlse = torch.randn(T, generator=gd, device=U.DEV) * 0.3
    loss, lse = (torch.empty(T, device=U.DEV) for _ in range(2))
    dx = torch.empty_like(x)
    ws = moe.alloc_xent_workspace(T, V, d)
    moe.moe_xent_fwd(x, W, target, loss, lse, ws)
    moe.moe_xent_bwd(x, W, target, loss, lse, dloss, dlse, dx, None, ws)
    Wd = W.double()
    D = torch.softmax(x.double() @ Wd.t(), 1).mul_((dloss + dlse).double()[:, None])
    D[torch.arange(T, device=U.DEV), target] -= dloss.double()
    ref = D @ Wd
    # the target's entry in D is exact: its part of the row is off by the result's rounding alone
    D[torch.arange(T, device=U.DEV), target] = 0
    bound = 2.0 ** -8 * ref.norm(dim=1) + (2.0 ** -8 + 1e-4) * D.abs() @ Wd.norm(dim=1) + 1e-4 * ref.norm(dim=1)
    err = (dx.double() - ref).norm(dim=1)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("T,V,d", [(5, 300, 64), (300, 1000, 832)])
def test_xent_infinite_logits(T, V, d):
    """A logit of -Inf is a probability of 0; one of +Inf, a NaN, or nothing but -Inf gives NaN to its token alone."""
    x, W, target = E.xent_inputs(T, V, d, 0.0)
    x[:, 0] = x[:, 0].abs() + 0.5
    target[target == 7] = 8
    target[1] = 7
    W[7, 0] = -float("inf")
    loss, lse, ws = E.run_xent(x, W, target)
    z = U.np64(x)[:, 1:] @ U.np64(W)[:, 1:].T + U.np64(x)[:, :1] * U.np64(W)[:, 0]
    rs = S.logsumexp(z)
    rl = rs - z[np.arange(T), target.numpy()]
    Wf = U.np64(W)
    Wf[7] = 0
    dz = E.logit_error(U.np64(x), Wf)
    assert loss[1] == float("inf") and rl[1] == np.inf
    rest = np.arange(T) != 1
    assert np.all(np.abs(U.np64(lse) - rs) <= dz + 2.0 ** -20 + 2.0 ** -23 * np.abs(rs))
    assert np.all(np.abs(U.np64(loss)[rest] - rl[rest]) <= 2 * dz[rest] + 2.0 ** -20 * rl[rest] + 2.0 ** -22)
    assert U.device_error(ws) == (0, 0)
    x[2, 0] = -x[2, 0]                     # its logit is +Inf
    x[3, 5] = float("nan")
    loss, lse, ws = E.run_xent(x, W, target)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[2] = bad[3] = True
    assert torch.equal(loss.isnan().cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)
    W[:, 0] = -float("inf")
    x[2, 0] = 1.0
    loss, lse, ws = E.run_xent(x, W, target)
    assert loss.isnan().all() and (lse.isnan() | (lse == -float("inf"))).all()


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32), (BF16, F32)], ids=lambda t: "/".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("T,V,d", [(3, 1 << 22, 64), (5, 300, 65536), (300, 200, 65536)])
def test_xent_largest_sizes(T, V, d, types):
    gd = torch.Generator(device=U.DEV).manual_seed(5)
    W = torch.empty(V, d, dtype=BF16, device=U.DEV).normal_(0, d ** -0.5, generator=gd)
    x = torch.empty(T, d, dtype=BF16, device=U.DEV).normal_(generator=gd)
    target = torch.randint(V, (T,), generator=gd, device=U.DEV)
    target[0] = V - 1
    dloss = torch.rand(T, generator=gd, device=U.DEV)
    loss, lse, dx, dW, ws = E.run_xent(x, W, target, True, dloss, None, *types)
    check_xent(x, W, target, dloss, None, loss, lse, dx, dW)
    assert U.device_error(ws) == (0, 0)


# --------------------------------------------------------- orthogonalised
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("mats,rows,cols,pairs", [
    (22, 541, 1021, {"gram": 2, "square": 2, "update": 1}),   # halves on pairs, read by single CTAs
    (87, 623, 580, {"gram": 2, "square": 2, "update": 1}),    # the same where the products are tall
    (70, 1146, 636, {"gram": 2, "square": 1, "update": 2})])  # pairs store both halves for the square
def test_orthogonalize_forms_of_its_products(mats, rows, cols, pairs, dt):
    G = torch.empty(mats, rows, cols, device=U.DEV).normal_(0, 1e-3, generator=torch.Generator(device=U.DEV).manual_seed(1)).to(dt)
    G[1] = 0
    out = []
    seen = launches(lambda: out.extend(E.run_ortho(G)))
    tall = rows > cols
    for name, kind in (("gram", 1 if tall else 0), ("square", 2), ("update", 4 if tall else 3)):
        assert seen is None or set(forms(seen, product("OrthoOp", kind))) == {pairs[name]}, (name, seen)
    got, ws = out
    assert U.device_error(ws) == (0, 0) and not got[1].any()
    for i in (0, mats // 2, mats - 1):
        g = U.np64(G[i])
        ref = S.orthogonalize(g, 5)
        assert U.relf(U.np64(got[i]), ref) <= 1.25 * U.relf(S.orthogonalize_rounded(g, 5), ref) + 2.0 ** -12


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("mats,rows,cols", [(300, 60, 200), (300, 200, 60), (200, 100, 300), (150, 49, 50), (140, 130, 64), (1, 40, 32768),
                                            (3, 1, 32768), (1, 32768, 47)])
def test_orthogonalize_small_sides_of_many_or_long_matrices(mats, rows, cols, dt):
    """Too many of them for a cluster each, or too long for what is on chip: the products one by one, on tiles that are
    mostly not there."""
    G = torch.empty(mats, rows, cols, device=U.DEV).normal_(0, 1e-3, generator=torch.Generator(device=U.DEV).manual_seed(2)).to(dt)
    if mats > 2:
        G[1] = 0
        G[2, 0, 0] = float("nan")
    got, ws = E.run_ortho(G)
    assert U.device_error(ws) == (0, 0)
    assert mats <= 2 or (not got[1].any() and got[2].isnan().all())
    for i in sorted({0, mats // 2, mats - 1} - ({1, 2} if mats > 2 else set())):
        g = U.np64(G[i])
        assert U.relf(U.np64(got[i]), S.orthogonalize(g, 5)) <= S.orthogonalize_spread(g, 5) + 2.0 ** -8


@pytest.mark.parametrize("rows,cols", [(4, 4), (49, 51)])
def test_orthogonalize_most_matrices(rows, cols):
    """More than a grid has rows."""
    mats = 65536
    G = torch.empty(mats, rows, cols, device=U.DEV).normal_(generator=torch.Generator(device=U.DEV).manual_seed(3))
    got, ws = E.run_ortho(G)
    assert U.device_error(ws) == (0, 0)
    for i in (0, 40000, 65534, 65535):
        g = U.np64(G[i])
        assert U.relf(U.np64(got[i]), S.orthogonalize(g, 5)) <= S.orthogonalize_spread(g, 5) + 2.0 ** -8


@pytest.mark.parametrize("rows,cols", [(6, 2000), (96, 160), (300, 200), (700, 900)])
def test_orthogonalize_of_sums_of_squares_past_fp32(rows, cols):
    """Whether a matrix counts as finite does not depend on how its sum of squares is shared: alone and among others."""
    base = torch.randn(rows, cols, generator=E.gen(4))
    top = 3.4e38 / float(base.double().square().sum())
    over, under = base * (1.01 * top) ** 0.5, base * (0.98 * top) ** 0.5
    G = torch.stack([over, under] + [base] * 20 + [over, under])
    finite = {}
    for name, m in (("under", under), ("base", base)):
        g = U.np64(m)
        finite[name] = (S.orthogonalize(g, 5), S.orthogonalize_spread(g, 5) + 2.0 ** -8)
    for m in (G, G[:2], G[:1], G[1:2]):
        got, ws = E.run_ortho(m)
        for i in range(len(m)):
            if torch.equal(m[i], over):
                assert got[i].isnan().all()
            else:
                ref, bar = finite["under" if torch.equal(m[i], under) else "base"]
                assert U.relf(U.np64(got[i]), ref) <= bar
        assert U.device_error(ws) == (0, 0)


# ----------------------------------------------------------------- balance
@pytest.mark.parametrize("T,E_,k,B,masked", [(30000, 64, 6, 2, "random"), (5000, 33, 3, 1, None), (9000, 8, 2, 3, "tail"),
                                             (7000, 256, 8, 70, "random")])
def test_balance_keeps_to_a_grid_limit(T, E_, k, B, masked):
    """A block that takes several parts of one sequence, and of several, in turn: the same bits."""
    z, idx, mask = E.balance_inputs(T, E_, k, B, masked)
    d, add = torch.ones(B), torch.randn(T, E_, generator=E.gen(7))
    ref = E.run_balance(z, idx, mask, B, d, d, add)
    for limit in (1, 5):
        out = []
        moe.moe_set_grid_limit(limit)
        try:
            seen = launches(lambda: out.extend(E.run_balance(z, idx, mask, B, d, d, add)))
        finally:
            moe.moe_set_grid_limit(0)
        assert all(torch.equal(a, b) for a, b in zip(ref[:5], out[:5]))
        grids = [g for n, g in seen or () if "balance_" in n]
        assert seen is None or (len(grids) >= 2 and max(grids) <= limit)


def test_balance_counts_an_expert_picked_twice():
    z, idx, mask = E.balance_inputs(400, 12, 3, 2, "random")
    idx[mask, 2] = idx[mask, 0]
    d = torch.ones(2)
    counts, mean_p, loss, zloss, out, ws = E.run_balance(z, idx, mask, 2, d, d, None)
    zn, idn = np.nan_to_num(z.numpy()), np.where(idx.numpy() < 12, idx.numpy(), 0)
    rc, _, rl, _ = S.balance_fwd(zn, idn, 2, mask.numpy())
    assert np.array_equal(counts.cpu().numpy(), rc) and np.allclose(U.np64(loss), rl, rtol=1e-5)
    ref = S.balance_bwd(zn, idn, 2, np.ones(2), np.ones(2), None, mask.numpy())
    assert np.allclose(U.np64(out), ref, rtol=1e-4, atol=1e-5 * np.abs(ref).max())
    assert U.device_error(ws) == (0, 0)


def test_balance_two_calls_at_once_on_their_own_workspaces():
    cases = []
    for T, E_, B, seed in ((20000, 64, 2, 1), (30000, 33, 3, 2)):
        z, idx, mask = E.balance_inputs(T, E_, 4, B, "random", seed=seed)
        cfg = moe.moe_cfg(T, 64, 64, E_, 4, 0, 0)
        g = [t.to(U.DEV) for t in (z, idx, mask)]
        d = torch.ones(B, device=U.DEV)
        ref = E.run_balance(z, idx, mask, B, torch.ones(B), torch.ones(B), None)[:5]
        cases.append((cfg, g, d, ref, [torch.empty_like(t) for t in ref], moe.alloc_workspace(cfg), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for cfg, (z, idx, mask), d, _, (counts, mean_p, loss, zloss, out), ws, s in cases:
            moe.moe_balance_fwd(cfg, z, idx, mask, counts, mean_p, loss, zloss, ws, stream=s)
            moe.moe_balance_bwd(cfg, z, counts, mask, d, d, None, out, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for _, _, _, ref, got, _, _ in cases for a, b in zip(ref, got))


@pytest.mark.parametrize("E_", [3, 8, 33, 64, 129, 256])
@pytest.mark.parametrize("scale", [1.0, 8.0, 25.0])
def test_balance_probabilities(E_, scale):
    """Sequences of one token: mean_p is that token's p, to the bound that the header states."""
    T = 512
    z, idx, _ = E.balance_inputs(T, E_, 1, T, None, scale=scale)
    d = torch.ones(T)
    _, mean_p, *_, ws = E.run_balance(z, idx, None, T, d, d, None)
    assert U.device_error(ws) == (0, 0)
    zn = z.double().numpy()
    p = S.softmax(zn)
    below = zn.max(1, keepdims=True) - zn
    # results below 2^-126 are 0
    assert np.all(np.abs(U.np64(mean_p) - p) <= (2.0 ** -18 + below * 2.0 ** -22) * p + 2.0 ** -125)
