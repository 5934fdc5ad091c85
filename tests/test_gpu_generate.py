"""The generation example: the layer for many tokens and the one for a few give the same stream, and the tokens come
out the same on every run.

The two ways round h differently: one bf16 value of 8 bits in moe_layer_fwd (2^-9 of an element on average at most,
2^-8 at worst), three bf16 values here.  With 4 bits the prompt's weights are bf16(s (q - 8)), one more rounding of at
most 2^-8 in each of the two products.  A relative Frobenius norm sums such errors with random signs: below one worst
rounding of each, 3 * 2^-8, per layer, if no routing decision flips; the stream's own part, carried on unrounded, only
shrinks it.  Two layers: 6 * 2^-8."""
import pytest
import torch

from combine_fp32_softmax_gb300.configs import MoEConfig
from examples import generate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_prompt_and_steps_agree(group):
    cfg = MoEConfig("generate", T=5, d=256, f=384, E=8, k=2, S=1)
    tokens, diff, _ = generate.run(cfg, layers=2, vocab=500, group=group, rows=5, prompt=21, steps=16)
    assert tokens.shape == (5, 16) and int(tokens.min()) >= 0 and int(tokens.max()) < 500
    assert diff <= 6 * 2.0 ** -8, diff
    again, _, _ = generate.run(cfg, layers=2, vocab=500, group=group, rows=5, prompt=21, steps=16)
    assert torch.equal(tokens, again)
