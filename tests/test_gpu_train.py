"""The training example: it runs, and its gradients are those of the whole model in fp64.

Between the fp64 model and the calls lie the layers' own bar (relative Frobenius 5e-3 each) and roundings to bf16 of the
normed streams, of the hidden states' gradient and of what goes into a layer's backward: at most 2^-8 of a value each,
four on the way to a gradient of a one-layer model."""
import numpy as np
import pytest
import torch

from combine_fp32_softmax_gb300.configs import MoEConfig
from examples import train
from oracle import moe_oracle as O
from oracle import step_oracle as S
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
BAR = 5e-3 + 4 * 2.0 ** -8


def norm(r):
    return r / np.sqrt((r ** 2).mean(-1, keepdims=True) + train.EPS)


def norm_bwd(r, dx):
    s = 1 / np.sqrt((r ** 2).mean(-1, keepdims=True) + train.EPS)
    return s * dx - r * s ** 3 * (dx * r).mean(-1, keepdims=True)


def test_gradients_of_a_step():
    cfg = MoEConfig("train", T=384, d=128, f=192, E=8, k=2, S=1)
    B, vocab = 3, 517
    model = train.Trainer(cfg, 1, vocab, B, seed=1, balance=0.5, zcoef=0.05)
    g = torch.Generator(device=U.DEV).manual_seed(2)
    tokens, target, mask = train.text(vocab, B, cfg.T // B, g)
    model.forward(tokens, target, mask)
    model.backward(target, mask)
    l = model.layers[0]

    r0 = U.np64(model.emb[tokens])
    x = norm(r0)
    logits = U.np64(l.logits)                          # the picks are those of the fp32 logits
    assert U.relf(logits, x @ U.np64(l.gate).T) <= 2.0 ** -8
    fw = O.layer_fwd(x, logits, *l.W, k=cfg.k, S=cfg.S)
    r1 = r0 + fw.y
    h = norm(r1)
    tn, mn = target.cpu().numpy(), mask.cpu().numpy()
    loss, lse = S.xent_fwd(h, U.np64(model.head), tn)
    assert U.relf(U.np64(model.loss), loss) <= BAR
    weight = (tn >= 0) / (tn >= 0).sum()
    D = S.xent_grad(h, U.np64(model.head), tn, weight)
    assert U.relf(U.np64(model.dhead), D.T @ h) <= BAR
    dr = norm_bwd(r1, D @ U.np64(model.head))
    bw = O.layer_bwd(fw, dr, x, *l.W)
    idx = fw.routing.sel
    assert np.array_equal(l.idx.cpu().numpy(), idx)
    dlogits = S.balance_bwd(logits, idx, B, np.full(B, 0.5 / B), np.full(B, 0.05 / B), bw.dlogits, mn)
    for name, ref in (("W1", bw.dW1), ("W3", bw.dW3), ("W2", bw.dW2), ("logits", dlogits), ("gate", dlogits.T @ x)):
        assert U.relf(U.np64(l.grads[name]), ref) <= BAR, name
    counts, _, bl, zl = S.balance_fwd(logits, idx, B, mn)
    assert np.array_equal(l.counts.cpu().numpy(), counts)
    assert np.allclose(U.np64(l.losses[0]), bl, rtol=1e-5) and np.allclose(U.np64(l.losses[1]), zl, rtol=1e-5)
    model.errors()


def test_update_is_the_orthogonalised_momentum():
    cfg = MoEConfig("train", T=128, d=64, f=128, E=4, k=2)
    model = train.Trainer(cfg, 1, 100, 2, seed=3)
    g = torch.Generator(device=U.DEV).manual_seed(4)
    tokens, target, mask = train.text(100, 2, 64, g)
    model.forward(tokens, target, mask)
    model.backward(target, mask)
    l = model.layers[0]
    before = [U.np64(w) for w in l.W]
    model.update(lr=0.5)
    for name, old, new in zip(("W1", "W3", "W2"), before, l.W):
        G = U.np64(l.grads[name])
        scale = 0.5 * max(1.0, G.shape[1] / G.shape[2]) ** 0.5
        for e in range(cfg.E):
            step = (old[e] - U.np64(new[e])) / scale
            ref = S.orthogonalize(G[e], 5)
            # the step's own error (its bar in the other tests), and the rounding of the new weights to bf16
            weights = 2.0 ** -8 * np.linalg.norm(U.np64(new[e])) / scale
            near = (1.25 * U.relf(S.orthogonalize_rounded(G[e], 5), ref) + 2.0 ** -12) * np.linalg.norm(ref)
            assert np.linalg.norm(step - ref) <= weights + near


def test_example_runs_and_repeats():
    cfg = MoEConfig("train", T=512, d=128, f=192, E=8, k=2, S=1)
    log, model = train.run(cfg, layers=2, vocab=300, sequences=4, steps=4)
    again, other = train.run(cfg, layers=2, vocab=300, sequences=4, steps=4)
    assert len(log) == 4 and all(np.isfinite(v) for step in log for v in step)
    for a, b in zip(model.layers, other.layers):
        assert all(torch.equal(p, q) for p, q in zip(a.W, b.W))
