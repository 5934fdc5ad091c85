"""Training steps of a small stack of MoE layers: loss, gradients and update through the library's calls.

    python examples/train.py [--steps 20] [--tokens 2048] [--layers 2] [--sequences 4]

Random weights and made-up text (each token's successor is fixed, with noise); no attention (the library has none), so a
token is predicted from the one before it.  It shows how the calls of a training step fit together:

  - forward: per layer the gate (``moe_linear_fwd``, fp32 logits), ``moe_layer_fwd`` and ``moe_balance_fwd`` (counts,
    balance and z losses of each sequence, its padding left out); at the end ``moe_xent_fwd`` against the next tokens;
  - backward: ``moe_xent_bwd`` gives the gradient of the hidden states and of the output projection, ``moe_layer_bwd``
    those of a layer, and ``moe_balance_bwd`` adds the balance losses' part to the logits' gradient;
  - update: momentum, then ``moe_orthogonalize`` on every expert's matrices and on the gates.

Norms, the residual stream and the gates' gradients are plain torch.
"""
import argparse
import math
import os
import sys
from dataclasses import dataclass, replace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_fp32_softmax_gb300 import moe  # noqa: E402
from combine_fp32_softmax_gb300.configs import MoEConfig  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-6


def norm(r):
    """Rows of the fp32 residual stream scaled to rms 1, in bf16."""
    return (r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)).to(BF16)


def norm_bwd(r, dx):
    """The gradient of r for that of norm(r)."""
    s = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    return s * dx - r * s.pow(3) * (dx * r).mean(-1, keepdim=True)


@dataclass
class Layer:
    gate: torch.Tensor    # [E, d] bf16
    W: list               # W1, W3, W2 bf16
    ws: torch.Tensor      # workspace: activations from forward to backward
    x: torch.Tensor       # [T, d] bf16, the layer's input
    logits: torch.Tensor
    y: torch.Tensor
    idx: torch.Tensor
    w: torch.Tensor
    counts: torch.Tensor  # [B, E]
    mean_p: torch.Tensor
    losses: list          # balance and z loss of each sequence [B]
    grads: dict
    momentum: dict


class Trainer:
    def __init__(self, cfg, layers, vocab, sequences, seed=0, balance=1e-2, zcoef=1e-3, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device=device) * std).to(BF16)

        def empty(*shape, dtype=F32):
            return torch.empty(*shape, dtype=dtype, device=device)

        self.cfg, self.vocab, self.B, self.device = cfg, vocab, sequences, device
        n, d, f, E, T = cfg.E + cfg.S, cfg.d, cfg.f, cfg.E, cfg.T
        self.emb, self.head = draw(vocab, d), draw(vocab, d, std=d ** -0.5)
        self.layers = []
        for _ in range(layers):
            W = [draw(n, f, d, std=d ** -0.5), draw(n, f, d, std=d ** -0.5), draw(n, d, f, std=f ** -0.5)]
            grads = {"W1": empty(n, f, d), "W3": empty(n, f, d), "W2": empty(n, d, f), "logits": empty(T, E), "x": empty(T, d)}
            self.layers.append(Layer(draw(E, d, std=d ** -0.5), W, moe.alloc_workspace(cfg, device), empty(T, d, dtype=BF16),
                                     empty(T, E), empty(T, d), empty(T, cfg.k, dtype=I32), empty(T, cfg.k),
                                     empty(sequences, E, dtype=I32), empty(sequences, E),
                                     [empty(sequences), empty(sequences)], grads,
                                     {"W1": 0.0, "W3": 0.0, "W2": 0.0, "gate": 0.0}))
        self.gate_ws = moe.alloc_linear_workspace(64, E, d, device)
        self.xent_ws = moe.alloc_xent_workspace(T, vocab, d, device=device)
        self.up_ws = {s: moe.alloc_orthogonalize_workspace(*s, device=device) for s in {(n, f, d), (n, d, f), (1, E, d)}}
        self.loss, self.lse = empty(T), empty(T)
        self.dh, self.dhead = empty(T, d, dtype=BF16), empty(vocab, d)
        self.dbalance = torch.full((sequences,), balance / sequences, device=device)
        self.dz = torch.full((sequences,), zcoef / sequences, device=device)

    def forward(self, tokens, target, mask):
        """Hidden states, and the losses of every token and sequence in self.loss and the layers' losses."""
        cfg = self.cfg
        r = self.emb[tokens].float()
        self.stream = [r]
        for l in self.layers:
            l.x.copy_(norm(r))
            for t in range(0, cfg.T, 64):
                moe.moe_linear_fwd(l.x[t:t + 64], l.gate, l.logits[t:t + 64], self.gate_ws)
            moe.moe_layer_fwd(cfg, l.logits, l.x, *l.W, l.y, l.idx, l.w, l.ws)
            moe.moe_balance_fwd(cfg, l.logits, l.idx, mask, l.counts, l.mean_p, *l.losses, l.ws)
            r = r + l.y
            self.stream.append(r)
        self.h = norm(r)
        moe.moe_xent_fwd(self.h, self.head, target, self.loss, self.lse, self.xent_ws)

    def backward(self, target, mask):
        """Gradients of the mean loss of the tokens with a target and of the layers' balance and z losses."""
        cfg = self.cfg
        weight = (target >= 0).float()
        weight /= weight.sum().clamp(min=1)
        moe.moe_xent_bwd(self.h, self.head, target, self.loss, self.lse, weight, None, self.dh, self.dhead, self.xent_ws)
        dr = norm_bwd(self.stream[-1], self.dh.float())
        for l, r in zip(reversed(self.layers), reversed(self.stream[:-1])):
            g = l.grads
            moe.moe_layer_bwd(cfg, dr.to(BF16), l.logits, l.x, *l.W, l.idx, l.w, l.ws, g["x"], g["logits"], g["W1"], g["W3"],
                              g["W2"])
            moe.moe_balance_bwd(cfg, l.logits, l.counts, mask, self.dbalance, self.dz, g["logits"], g["logits"], l.ws)
            g["gate"] = g["logits"].t() @ l.x.float()
            dr = dr + norm_bwd(r, g["x"] + g["logits"] @ l.gate.float())

    def update(self, lr=0.02):
        for l in self.layers:
            for name, W in zip(("W1", "W3", "W2", "gate"), (*l.W, l.gate)):
                l.momentum[name] = m = 0.9 * l.momentum[name] + l.grads[name]
                shape = m.shape if m.dim() == 3 else (1, *m.shape)
                step = torch.empty_like(W)
                moe.moe_orthogonalize(m, step, 5, self.up_ws[shape])
                scale = lr * math.sqrt(max(1.0, shape[1] / shape[2]))
                W.copy_(W.float() - scale * step.float())
        self.head.copy_(self.head.float() - 10 * lr * self.dhead)

    def errors(self):
        for ws in (self.gate_ws, self.xent_ws, *self.up_ws.values(), *(l.ws for l in self.layers)):
            code, info = moe.moe_get_device_error(ws)
            if code:
                raise RuntimeError(f"device error {code} ({info:#x})")


def text(vocab, sequences, length, generator, device="cuda"):
    """Tokens, their successors (none where a sequence is over) and which tokens are there, for sequences that end in padding."""
    follow = torch.randperm(vocab, generator=torch.Generator().manual_seed(0)).to(device)
    t = torch.empty(sequences, length + 1, dtype=torch.int64, device=device)
    t[:, 0] = torch.randint(vocab, (sequences,), generator=generator, device=device)
    noise = torch.rand(sequences, length, generator=generator, device=device) < 0.1
    other = torch.randint(vocab, (sequences, length), generator=generator, device=device)
    for i in range(length):
        t[:, i + 1] = torch.where(noise[:, i], other[:, i], follow[t[:, i]])
    kept = torch.randint(length // 2, length + 1, (sequences, 1), generator=generator, device=device)
    mask = torch.arange(length, device=device) < kept
    return t[:, :-1].reshape(-1), torch.where(mask, t[:, 1:], -100).reshape(-1), mask.reshape(-1)


def run(cfg, layers=2, vocab=1000, sequences=4, steps=20, seed=0):
    """Trains for some steps; (mean loss and balance loss of each step, the trainer)."""
    model = Trainer(cfg, layers, vocab, sequences, seed)
    g = torch.Generator(device=model.device).manual_seed(seed)
    log = []
    for _ in range(steps):
        tokens, target, mask = text(vocab, sequences, cfg.T // sequences, g, model.device)
        model.forward(tokens, target, mask)
        model.backward(target, mask)
        model.update()
        log.append((model.loss.sum() / (target >= 0).sum(), torch.stack([l.losses[0].mean() for l in model.layers]).mean()))
    model.errors()
    return [(a.item(), b.item()) for a, b in log], model


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--sequences", type=int, default=4)
    a = p.parse_args()
    cfg = replace(MoEConfig("train", T=0, d=256, f=512, E=8, k=2, S=1), T=a.tokens)
    log, _ = run(cfg, a.layers, 1000, a.sequences, a.steps)
    for i, (loss, balance) in enumerate(log):
        print(f"step {i:3d}  loss {loss:.3f}  balance loss {balance:.3f}")


if __name__ == "__main__":
    main()
