"""One layer of examples/moe_layer.py over batches of different sizes."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def outputs(layer, x, mask):
    out = layer.forward(x, residual=x, token_mask=mask, stats=True)
    d_logits, d_y = layer.backward(torch.ones_like(out), torch.full((1,), 0.25, device="cuda"))
    torch.cuda.synchronize()
    return [t.clone() for t in (out, layer.counts, layer.loss, layer.loss_grad, d_logits, d_y)]


def test_a_layer_for_many_tokens_takes_fewer():
    # the buffers of a layer for 4200 tokens, where a token has fewer lanes than in batches up to 4096
    sizes = dict(H=256, I=64, experts=100, top_k=3)
    wide = moe_layer.synthetic_layer(max_tokens=4200, **sizes)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for M in (4200, 2000, 1, 4096):
        x = torch.randn(M, wide.H, device="cuda", generator=gen).bfloat16()
        mask = (torch.rand(M, device="cuda", generator=gen) > 0.1).to(torch.uint8)
        fitted = moe_layer.synthetic_layer(max_tokens=M, **sizes)
        assert all(torch.equal(a, b) for a, b in zip(outputs(wide, x, mask), outputs(fitted, x, mask))), M
