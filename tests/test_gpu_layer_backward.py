"""What the backward pass of examples/moe_layer.py may be asked for."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def inputs(layer, M):
    gen = torch.Generator(device="cuda").manual_seed(M)
    return torch.randn(M, layer.H, device="cuda", generator=gen).bfloat16(), torch.full((1,), 0.5, device="cuda")


def test_no_gradient_of_a_loss_that_this_forward_did_not_form():
    # loss_grad would be that of the batch before
    layer = moe_layer.synthetic_layer()
    x, d_loss = inputs(layer, 20)
    layer.forward(x, stats=True)
    layer.forward(x.flip(0).contiguous())
    with pytest.raises(ValueError, match="stats"):
        layer.backward(x, d_loss)


def test_backward_belongs_to_the_last_batch():
    layer = moe_layer.synthetic_layer()
    x, d_loss = inputs(layer, 20)
    with pytest.raises(ValueError, match="forward"):
        layer.backward(x, d_loss)
    layer.forward(x, stats=True)
    with pytest.raises(ValueError, match="20"):
        layer.backward(x[:19], d_loss)


def test_gradients_without_the_loss():
    layer = moe_layer.synthetic_layer()
    x, d_loss = inputs(layer, 20)
    layer.forward(x, stats=True)
    want = [t.clone() for t in layer.backward(x, torch.zeros_like(d_loss))]
    layer.forward(x)
    got = layer.backward(x)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
