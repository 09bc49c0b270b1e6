"""The router over groups at its limits (64 groups, 1024 experts, 64 chosen) and in every width of its kernels,
on an MI355X."""
import numpy as np
import pytest

from test_gpu_route_groups import Call, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,K,groups,top", [
    (70, 1024, 64, 64, 7), (3, 1024, 1, 64, 63), (2, 960, 64, 64, 5),            # 16 experts a lane
    (70, 512, 8, 64, 1), (5, 448, 9, 64, 33),
    (4100, 32, 2, 16, 3), (4100, 64, 8, 64, 11), (4100, 128, 4, 64, 9), (4100, 256, 5, 64, 40), (4100, 16, 3, 4, 2)])
def test_limits(M, E, K, groups, top, score, kind):
    rng = np.random.default_rng(M + E + groups)
    ways = [(1, None, None), (2, None, rng.random(M) > 0.1), (2, rng.normal(size=E), None)]
    for group_top, bias, mask in ways if M < 1000 else ways[1:2] if kind == "bf16" else ways[2:]:
        Call(logits_of(E + K, M, E), K, groups, top, group_top, kind, bias=bias, mask=mask, score=score, renormalize=True,
             scale=2.5).check()


@pytest.mark.parametrize("E,groups", [(1024, 64), (64, 64), (256, 8)])
def test_every_token_in_doubt(E, groups):
    # all logits alike: ties in every comparison, decided by the lowest index
    for M in (9, 4100 if E <= 256 else 300):
        Call(np.full((M, E), 0.25), 6, groups, max(2, groups // 4), 2 if E > groups else 1, "f32", bias=np.zeros(E),
             score="sigmoid").check()
