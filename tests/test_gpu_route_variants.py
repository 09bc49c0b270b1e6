"""The router's variants by tokens and experts, and choices that only double precision settles."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from layer_gpu_helpers import check, host
from test_gpu_route import Call, backward_case, logits_of

pytestmark = pytest.mark.gpu


# 16 and 64 lanes a token, one to sixteen experts a lane, last waves that are not full
@pytest.mark.parametrize("M", [1, 3, 4099])
@pytest.mark.parametrize("E,K", [(5, 5), (16, 2), (17, 17), (31, 3), (63, 20), (64, 64), (66, 4), (129, 33), (250, 8), (257, 5)])
def test_every_width(M, E, K):
    if M > 1000 and K > 10:
        K = 10
    rng = np.random.default_rng(M + E)
    mask = None if M == 1 else rng.random(M) > 0.2
    Call(logits_of(M + E, M, E), K, "bf16", mask=mask, renormalize=True, scale=0.5).check()
    Call(logits_of(M + E, M, E), K, "f32", bias=rng.normal(size=E) * 0.1, score="sigmoid", mask=mask).check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E", [(3, 60), (9, 200), (4101, 200), (2, 700)])
def test_choices_below_float_precision(M, E, score):
    # scores that F32 cannot tell apart, in one of every four tokens: the order of the doubles counts
    rng = np.random.default_rng(E)
    l = logits_of(E + 1, M, E)
    l[::4] = l[::4, :1] + 3e-7 * rng.permuted(np.tile(np.arange(E), (len(l[::4]), 1)), axis=1)
    Call(l, 6, "f32", bias=1e-8 * rng.permutation(E), score=score).check()


def test_a_token_without_any_expert_counts_nowhere():
    # every expert is taken out by the bias or the logit: as for a masked token
    l = logits_of(3, 7, 20)
    l[2, :10] = -np.inf
    l[5, :10] = -np.inf
    bias = np.zeros(20)
    bias[10:] = -np.inf
    c = Call(l, 3, "f32", bias=bias)
    c.run()
    keep = Call(l[[0, 1, 3, 4, 6]], 3, "f32", bias=bias)
    keep.run()
    torch.cuda.synchronize()
    assert (c.ids[[2, 5]] == -1).all() and (c.weights[[2, 5]] == 0).all()
    for name in ("counts", "loss_grad"):
        assert torch.equal(c.stats[name], keep.stats[name])
    check(host(c.stats["loss"]), host(keep.stats["loss"]), 2.0 ** -20, "loss")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,K", [(1, 16, 16), (5, 17, 3), (4101, 130, 4), (4097, 64, 20), (6, 300, 40)])
def test_gradient_of_every_width(M, E, K, score):
    for kind, renormalize in (("bf16", True), ("f32", False)):
        lh, got, args = backward_case(M, E, K, kind, score, renormalize, 1.5, seed=4)
        want, mag = ref.route_backward(lh, *args)
        # as in the other gradient tests: scores within (32 + spread) 2^-24, twice, sums over lanes and products
        rel = (128 + 4 * (np.abs(lh).max() * 2)) * 2.0 ** -24
        check(got, want, ref.HALF_STEP[kind] * np.abs(want) + rel * mag + 2.0 ** -120, "d_logits")
