"""The router's gradient where ids name no expert: what stands at such a place never reaches a result."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import check, dev, host, i32, nan_like
from test_gpu_route import logits_of

pytestmark = pytest.mark.gpu


# widths of 16, 32, 64, 256 and 512 experts that the rows do not fill, and full ones
@pytest.mark.parametrize("E,width", [(12, 16), (16, 16), (17, 32), (40, 64), (167, 256), (256, 256), (300, 512)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unwritten_gradients_of_foreign_ids(E, width, renormalize, score, bad):
    foreign = [E, width - 1, width, -1, -2 ** 31, 2 ** 31 - 1]
    M, K = len(foreign), 4
    rng = np.random.default_rng(E)
    l = dev(logits_of(E, M, E))
    ids = np.stack([rng.permutation(E)[:K] for _ in range(M)])
    for t, e in enumerate(foreign):
        if e < 0 or e >= E:
            ids[t, 2] = e
    dw = rng.normal(size=(M, K)).astype(np.float32)
    grad = rng.uniform(0, 0.1, size=E).astype(np.float32)
    given = np.where((ids >= 0) & (ids < E), dw, np.float32(bad))
    out = nan_like((M, E))
    q4.route_backward(l, M, E, K, i32(ids), out, d_weights=dev(given), d_loss=dev([0.25]), loss_grad=dev(grad), score=score,
                      renormalize=renormalize, scale=1.5, xdtype="f32")
    torch.cuda.synchronize()
    lh = host(l)
    want, mag = ref.route_backward(lh, ids, score, renormalize, 1.5, dw.astype(np.float64), 0.25, grad.astype(np.float64))
    # scores within (32 + spread) 2^-24, twice, plus sums over lanes and products
    rel = (128 + 4 * (np.abs(lh).max() * 2)) * 2.0 ** -24
    check(host(out), want, 2.0 ** -24 * np.abs(want) + rel * mag + 2.0 ** -120, "d_logits")


def test_a_first_id_past_the_experts_keeps_its_token():
    # only a negative first id takes the token out
    M, E, K = 3, 20, 3
    l = dev(logits_of(5, M, E))
    ids = np.array([[20, 3, 4], [31, 5, 6], [-1, 7, 8]])
    dw = np.random.default_rng(6).normal(size=(M, K)).astype(np.float32)
    given = dw.copy()
    given[:, 0] = np.nan
    out = nan_like((M, E))
    q4.route_backward(l, M, E, K, i32(ids), out, d_weights=dev(given), xdtype="f32")
    torch.cuda.synchronize()
    want, mag = ref.route_backward(host(l), ids, "softmax", False, 1.0, dw.astype(np.float64), 0.0, np.zeros(E))
    check(host(out), want, 2.0 ** -16 * mag + 2.0 ** -120, "d_logits")
    assert (host(out)[2] == 0).all()
