"""The balance loss of batches whose lanes add up many tokens each, against sums in 64 bits."""
import pytest
import torch

import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import TYPES, nan_like
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu


def route(logits, K, kind, **kw):
    """ids, counts, loss and loss_grad of one call."""
    M, E = logits.shape
    ids, weights = torch.full((M, K), 777, dtype=torch.int32, device="cuda"), nan_like((M, K))
    counts = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    loss, loss_grad = nan_like((1,)), nan_like((E,))
    n = q4.route_workspace_bytes(M, E)
    q4.route(logits, M, E, K, ids, weights, counts=counts, loss=loss, loss_grad=loss_grad,
             workspace=aligned_empty(n, 256), workspace_bytes=n, xdtype=kind, **kw)
    torch.cuda.synchronize()
    return ids, counts, loss, loss_grad


# (M, E): 512 to 2048 tokens a lane with 16 and with 64 lanes a token
@pytest.mark.parametrize("M,E", [(1 << 24, 7), (1 << 22, 60), (3000001, 100), (1 << 22, 300), (1 << 20, 1000)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_logits(M, E, score):
    # every probability is 1 / E, and its rounding always falls to the same
    # side; every token takes expert 0: loss = E * 1 * (1 / E) = 1
    ids, counts, loss, grad = route(torch.zeros((M, E), dtype=torch.bfloat16, device="cuda"), 1, "bf16", score=score)
    assert (ids == 0).all() and int(counts[0]) == M and int(counts.sum()) == M
    # 64 roundings for a probability (as in the other tests of the loss) and 64 for the sums, whatever M
    assert abs(loss.double().item() - 1.0) <= 128 * 2.0 ** -24
    assert abs(grad[0].double().item() * M / E - 1.0) <= 2.0 ** -22 and (grad[1:] == 0).all()


# past 8192 tokens a wave of four tokens makes a second trip
@pytest.mark.parametrize("M,E,K", [(8193, 256, 8), (20011, 96, 4), (300007, 64, 6), (70001, 250, 2), (40000, 384, 8)])
@pytest.mark.parametrize("kind,score", [("bf16", "softmax"), ("f32", "sigmoid")])
def test_random_logits(M, E, K, kind, score):
    gen = torch.Generator(device="cuda").manual_seed(M)
    l = (2 * torch.randn(M, E, device="cuda", generator=gen)).to(TYPES[kind])
    mask = (torch.rand(M, device="cuda", generator=gen) > 0.1).to(torch.uint8)
    ids, counts, loss, grad = route(l, K, kind, score=score, token_mask=mask)
    x, on = l.double(), mask.bool()
    best = x.sort(dim=1, descending=True, stable=True)[1][:, :K]
    assert torch.equal(ids[on].long(), best[on]) and (ids[~on] == -1).all()
    want = torch.bincount(best[on].flatten(), minlength=E)
    assert torch.equal(counts.long(), want)
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    T = int(on.sum())
    g = E * want.double() / (K * T * T)
    exact = (g * (s / s.sum(1, keepdim=True))[on].sum(0)).sum().item()
    assert ((grad.double() - g).abs() <= 2.0 ** -22 * g).all()
    spread = float(x.max() - x.min()) + float(x.abs().max())
    # a probability within (64 + 2 spread) roundings, its sums within 64, whatever M
    assert abs(loss.double().item() - exact) <= (128 + 2 * spread) * 2.0 ** -24 * exact
