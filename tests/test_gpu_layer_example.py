"""The layer of examples/moe_layer.py, step by step against the 64-bit forms, on an MI355X."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_reference as ref
from layer_gpu_helpers import check, host, replayed

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def step(layer, x, mask, d_out, d_loss):
    layer.forward(x, residual=x, token_mask=mask, stats=True)
    layer.backward(d_out, d_loss)


@pytest.mark.parametrize("M,kw", [(1, {}), (48, dict(score="sigmoid", scale=2.5))])
def test_layer(M, kw):
    layer = moe_layer.synthetic_layer(**kw)
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, layer.H, device="cuda", generator=gen).bfloat16()
    mask = torch.ones(M, dtype=torch.uint8, device="cuda")
    mask[5::7] = 0
    d_out = torch.randn(M, layer.H, device="cuda", generator=gen).bfloat16()
    d_loss = torch.full((1,), 0.5, device="cuda")
    step(layer, x, mask, d_out, d_loss)
    torch.cuda.synchronize()
    weights, scales, _ = layer.gate
    want, mag = ref.linear(host(weights), host(scales), None, layer.group, host(x), layer.E, layer.H)
    # the output's rounding, and a step of 2^-23 for each addition a term can pass through
    steps = 2 * layer.group + layer.H // layer.group + 32
    check(host(layer.logits[:M]), want, 2.0 ** -8 * np.abs(want) + steps * 2.0 ** -23 * mag, "logits")
    logits = host(layer.logits[:M])
    score, scale = layer.kw["score"], layer.kw["scale"]
    ids, w, counts, loss, grad = ref.route(logits, layer.K, score, True, scale, mask=host(mask))
    assert np.array_equal(host(layer.ids[:M]), ids) and np.array_equal(host(layer.counts), counts)
    # as the router's own tests: exp's argument at the spread of the logits, then sums over lanes
    rel = (64 + 2 * (np.abs(logits).max() * 2)) * 2.0 ** -24
    check(host(layer.weights[:M]), w, rel * w, "weights")
    check(host(layer.loss), [loss], (rel + (M / 4 + 64) * 2.0 ** -24) * loss, "loss")
    y, got_w = host(layer.y[:M]), host(layer.weights[:M])
    want, mag = ref.combine(y, got_w, ids, layer.E, host(x))
    check(host(layer.out[:M]), want, 2.0 ** -8 * np.abs(want) + (layer.K + 1) * 2.0 ** -24 * mag, "out")
    want_y, want_w, mag = ref.combine_backward(host(d_out), y, got_w, ids, layer.E)
    check(host(layer.d_y[:M]), want_y, (2.0 ** -8 + 2.0 ** -24) * np.abs(want_y), "d_y")
    check(host(layer.d_weights[:M]), want_w, (layer.H / 64 + 32) * 2.0 ** -24 * mag, "d_weights")
    want, mag = ref.route_backward(logits, ids, score, True, scale, host(layer.d_weights[:M]), 0.5, host(layer.loss_grad))
    rel = (128 + 4 * (np.abs(logits).max() * 2)) * 2.0 ** -24
    check(host(layer.d_logits[:M]), want, 2.0 ** -8 * np.abs(want) + rel * mag + 2.0 ** -120, "d_logits")


def test_layer_in_a_graph():
    layer = moe_layer.synthetic_layer(max_tokens=32)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(32, layer.H, device="cuda", generator=gen).bfloat16()
    mask = (torch.arange(32, device="cuda") % 5 != 2).to(torch.uint8)
    d_out, d_loss = torch.randn_like(x), torch.full((1,), 0.1, device="cuda")
    outs = [layer.out, layer.ids, layer.weights, layer.counts, layer.loss, layer.d_logits, layer.d_y]
    step(layer, x, mask, d_out, d_loss)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for got in replayed(lambda: step(layer, x, mask, d_out, d_loss), outs):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_example_runs():
    moe_layer.main()
