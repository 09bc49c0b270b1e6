"""The router over groups where a group's two best experts carry biases of opposite sign, so that their
sum is small beside its parts, against the 64-bit form on an MI355X."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_q4_amd as q4
import tuning_reference as tune
from layer_gpu_helpers import dev, host, nan_like

pytestmark = pytest.mark.gpu


def check_ids(logits, bias, K, groups, top, score):
    M, E = logits.shape
    l, b = dev(logits), dev(bias)
    ids = torch.full((M, K), 777, dtype=torch.int32, device="cuda")
    q4.route_groups(l, M, E, K, groups, top, ids, nan_like((M, K)), score=score, select_bias=b, xdtype="f32")
    torch.cuda.synchronize()
    want, *_ = tune.route_groups(host(l), K, groups, top, 2, score, bias=host(b))
    wrong = np.flatnonzero((host(ids) != want).any(1))
    assert wrong.size == 0, f"{wrong.size} of {M} tokens, the first {wrong[0]}: {host(ids)[wrong[0]]} for {want[wrong[0]]}"


def near(seed, M, E, score):
    """Logits whose scores lie within a few 1e-4 of each other."""
    return np.random.default_rng(seed).normal(size=(M, E)) * (1e-3 if score == "sigmoid" else 2.5e-4 * E)


def opposite(E, groups, bias):
    """+b and -b for the first two experts of a group, b from bias to twice that: the experts' own order is plain,
    while the groups are ranked by sums of two scores, which keys of 24 bits hold to 2^-24 of b only."""
    b = np.full(E, -np.inf)
    size = E // groups
    up = bias * (1 + np.random.default_rng(E).permutation(groups) / groups)
    b[0::size], b[1::size] = up, -up
    return b


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [64.0, 256.0, 1000.0, 1e4])
@pytest.mark.parametrize("E,groups,top", [(64, 32, 4), (256, 64, 5), (512, 64, 3)])
def test_opposite_biases_cancel(E, groups, top, bias, score):
    check_ids(near(E + int(bias), 400, E, score), opposite(E, groups, bias), top, groups, top, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("odd", [0, 1])
def test_one_group_cancels_and_its_neighbour_does_not(odd, score):
    # every other group has the biases: the last kept or the first left out may be the only one whose rank is rounded
    E, groups = 64, 32
    b = opposite(E, groups, 512.0)
    b[2 * odd::4], b[2 * odd + 1::4] = 0.0, 0.0
    check_ids(near(odd, 400, E, score), b, 1, groups, 4, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_of_the_lowest_value_beside_a_positive_one(score):
    # masks by the type's lowest value and by a large finite one, in some groups of every token
    rng = np.random.default_rng(9)
    E, groups, M = 64, 16, 200
    b = 0.1 * rng.normal(size=E)
    b[1:16] = np.finfo(np.float32).min
    b[17:24], b[16] = -1e9, 1e9
    check_ids(rng.normal(size=(M, E)), b, 6, groups, 5, score)
