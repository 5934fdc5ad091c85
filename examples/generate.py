"""Generation with the layer for a few tokens: a small stack of MoE layers reads prompts and goes on, token by token.

    python examples/generate.py [--group 32|64|128|0] [--rows 4] [--prompt 48] [--steps 64]

Random weights; no attention (the library has none), so a token depends on the one before it only.  It shows how the
calls fit together:

  - the experts and the output projection go to 4 bits once (``moe_q4_quantize``); ``--group 0`` keeps bf16;
  - prompts run through ``moe_layer_fwd`` on the values that the 4-bit weights stand for (``moe_q4_dequantize``);
  - a step is, per layer, the gate (``moe_linear_fwd``, fp32 logits) and the whole MoE layer in one launch
    (``moe_decode_q4_fwd``, or ``moe_decode_fwd`` with bf16 weights), then the output projection
    (``moe_linear_q4_fwd`` or ``moe_linear_fwd``); the steps replay one CUDA graph;
  - workspaces are allocated once and looked at for device errors at the end.
"""
import argparse
import os
import sys
from dataclasses import dataclass, replace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_fp32_softmax_gb300 import moe  # noqa: E402
from combine_fp32_softmax_gb300.configs import MoEConfig  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def norm(x):
    """Rows of the fp32 residual stream scaled to rms 1, in bf16."""
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(BF16)


@dataclass
class Layer:
    gate: torch.Tensor        # [E, d] bf16
    W: list                   # W1, W3, W2 bf16: what prompts run on
    q: list                   # their codes and scales (empty with bf16 weights)


class Stack:
    def __init__(self, cfg, layers, vocab, group, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device=device) * std).to(BF16)

        self.cfg, self.group, self.vocab, self.device = cfg, group, vocab, device
        n, d, f = cfg.E + cfg.S, cfg.d, cfg.f
        self.emb = draw(vocab, d)
        self.layers = []
        for _ in range(layers):
            W = [draw(n, f, d, std=d ** -0.5), draw(n, f, d, std=d ** -0.5), draw(n, d, f, std=2 * f ** -0.5)]
            self.layers.append(Layer(draw(cfg.E, d, std=d ** -0.5), W, self.quantised(W)))
        self.head = [draw(vocab, d, std=d ** -0.5)]
        self.head_q = self.quantised(self.head)

    def quantised(self, mats):
        """Codes and scales of each tensor; the tensors then hold what those stand for."""
        if not self.group:
            return []
        out = []
        for W in mats:
            codes, scales = moe.q4_empty(W.shape[0] if W.dim() == 3 else 1, *W.shape[-2:], self.group, self.device)
            moe.moe_q4_quantize(W, codes, scales, self.group)
            moe.moe_q4_dequantize(codes, scales, W, self.group)
            out += [codes, scales]
        return out

    def logits(self, gate, x, out, ws):
        """Router logits of any number of rows, at most 64 at a time."""
        for t in range(0, x.shape[0], 64):
            moe.moe_linear_fwd(x[t:t + 64], gate, out[t:t + 64], ws)

    def read(self, tokens):
        """The residual stream of every prompt token [n, d], through the layer call for many tokens."""
        cfg, dev = replace(self.cfg, T=tokens.numel()), self.device
        r = self.emb[tokens.reshape(-1)].float()
        ws = moe.alloc_workspace(cfg, dev)
        gate_ws = moe.alloc_linear_workspace(64, cfg.E, cfg.d, dev)
        lg = torch.empty(cfg.T, cfg.E, dtype=F32, device=dev)
        y = torch.empty(cfg.T, cfg.d, dtype=F32, device=dev)
        idx = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=dev)
        w = torch.empty(cfg.T, cfg.k, dtype=F32, device=dev)
        for l in self.layers:
            x = norm(r)
            self.logits(l.gate, x, lg, gate_ws)
            moe.moe_layer_fwd(cfg, lg, x, *l.W, y, idx, w, ws)
            r = r + y
        self.errors(ws, gate_ws)
        return r

    def errors(self, *workspaces):
        for ws in workspaces:
            code, info = moe.moe_get_device_error(ws)
            if code:
                raise RuntimeError(f"device error {code} ({info:#x})")


class Steps:
    """One token for each of `rows` sequences, as a graph over fixed buffers."""

    def __init__(self, model, rows):
        self.m, cfg, dev = model, replace(model.cfg, T=rows), model.device
        self.cfg = cfg
        self.r = torch.empty(rows, cfg.d, dtype=F32, device=dev)          # residual stream after the layers
        self.token = torch.zeros(rows, dtype=torch.int64, device=dev)     # read by a step, then the next one
        self.lg = torch.empty(rows, cfg.E, dtype=F32, device=dev)
        self.y = torch.empty(rows, cfg.d, dtype=F32, device=dev)
        self.idx = torch.empty(rows, cfg.k, dtype=torch.int32, device=dev)
        self.w = torch.empty(rows, cfg.k, dtype=F32, device=dev)
        self.out = torch.empty(rows, model.vocab, dtype=F32, device=dev)
        self.ws = moe.alloc_decode_workspace(cfg, dev)
        self.gate_ws = moe.alloc_linear_workspace(rows, cfg.E, cfg.d, dev)
        self.head_ws = moe.alloc_linear_workspace(rows, model.vocab, cfg.d, dev)
        self.step()                                                       # warm-up, outside the capture
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.step()

    def project(self):
        """The next tokens from the residual stream."""
        m, x = self.m, norm(self.r)
        if m.group:
            moe.moe_linear_q4_fwd(x, *m.head_q, m.group, self.out, self.head_ws)
        else:
            moe.moe_linear_fwd(x, m.head[0], self.out, self.head_ws)
        self.token.copy_(self.out.argmax(-1))

    def step(self):
        m = self.m
        r = m.emb[self.token].float()
        for l in m.layers:
            x = norm(r)
            m.logits(l.gate, x, self.lg, self.gate_ws)
            if m.group:
                moe.moe_decode_q4_fwd(self.cfg, m.group, self.lg, x, *l.q, self.y, self.idx, self.w, self.ws)
            else:
                moe.moe_decode_fwd(self.cfg, self.lg, x, *l.W, self.y, self.idx, self.w, self.ws)
            r = r + self.y
        self.r.copy_(r)
        self.project()


def run(cfg, layers=2, vocab=1000, group=64, rows=4, prompt=48, steps=64, seed=0):
    """Reads `rows` prompts and generates `steps` tokens for each: (tokens [rows, steps], the relative difference of
    the two ways to the last prompt token's residual stream, microseconds a step)."""
    model = Stack(cfg, layers, vocab, group, seed)
    g = torch.Generator().manual_seed(seed)
    prompts = torch.randint(vocab, (rows, prompt), generator=g).to(model.device)
    last = model.read(prompts).view(rows, prompt, -1)[:, -1]
    gen = Steps(model, rows)
    gen.token.copy_(prompts[:, -1])
    gen.graph.replay()                        # the last prompt token the other way
    diff = ((gen.r - last).norm() / last.norm()).item()
    gen.r.copy_(last)
    gen.project()
    got = [gen.token.clone()]
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps - 1):
        gen.graph.replay()
        got.append(gen.token.clone())
    end.record()
    torch.cuda.synchronize()
    model.errors(gen.ws, gen.gate_ws, gen.head_ws)
    return torch.stack(got, 1), diff, begin.elapsed_time(end) * 1e3 / max(1, steps - 1)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--group", type=int, default=64, choices=(0, 32, 64, 128))
    p.add_argument("--rows", type=int, default=4)
    p.add_argument("--prompt", type=int, default=48)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--layers", type=int, default=4)
    a = p.parse_args()
    cfg = MoEConfig("generate", T=a.rows, d=2048, f=1408, E=64, k=6, S=2)
    tokens, diff, us = run(cfg, a.layers, 32000, a.group, a.rows, a.prompt, a.steps)
    print(f"{a.layers} layers of d={cfg.d} f={cfg.f} E={cfg.E} k={cfg.k} S={cfg.S}, "
          f"{'4-bit weights, groups of %d' % a.group if a.group else 'bf16 weights'}")
    print(f"prompt and step differ by {diff:.1e} (relative, last prompt token)")
    print(f"{us:.1f} us a step of {a.rows} tokens, {a.rows / us * 1e6:.0f} tokens/s")
    print("first row:", " ".join(map(str, tokens[0, :12].tolist())), "...")


if __name__ == "__main__":
    main()
