"""Refusals of the router over groups, the adapters and the linear's gradient on the host (nothing is enqueued, no GPU)."""
import pytest

import quantized_moe_expert_q4_amd as q4

W, S, B, X, OUT, IDS, WS = (1 << 20, 1 << 22, 1 << 23, 1 << 24, 1 << 26, 1 << 27, 1 << 28)   # fake device addresses
INVALID, ALIGN, UNSUPPORTED, WORKSPACE = (q4.Q4_ERR_INVALID_ARGUMENT, q4.Q4_ERR_ALIGNMENT, q4.Q4_ERR_UNSUPPORTED,
                                          q4.Q4_ERR_WORKSPACE)


def _groups(**kw):
    a = dict(logits=X, M=4, E=64, K=8, groups=8, top_groups=4, ids=IDS, weights=OUT)
    a.update(kw)
    return q4.validate_route_groups(**a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(groups=64, top_groups=8), dict(groups=1, top_groups=1), dict(top_groups=8, K=64),
                                dict(top_groups=1), dict(group_top=1), dict(E=1, K=1, groups=1, top_groups=1),
                                dict(E=1024, groups=64), dict(xdtype="f32"), dict(score="sigmoid", select_bias=B),
                                dict(counts=S, workspace=WS, workspace_bytes=1 << 20)])
def test_route_groups_accepts(kw):
    assert _groups(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), INVALID), (dict(groups=-8), INVALID), (dict(groups=7), INVALID), (dict(groups=128), INVALID),
    (dict(E=128, groups=128), UNSUPPORTED), (dict(top_groups=0), INVALID), (dict(top_groups=9), INVALID),
    (dict(top_groups=-1), INVALID), (dict(group_top=0), INVALID), (dict(group_top=3), INVALID),
    (dict(top_groups=1, K=9), INVALID), (dict(groups=64, top_groups=7), INVALID), (dict(M=0), INVALID), (dict(E=0), INVALID),
    (dict(K=0), INVALID), (dict(E=1032), UNSUPPORTED), (dict(logits=None), INVALID), (dict(logits=X + 1), ALIGN),
    (dict(logits=X + 2, xdtype="f32"), ALIGN), (dict(counts=S), WORKSPACE),
    (dict(counts=S, workspace=WS, workspace_bytes=16), WORKSPACE)])
def test_route_groups_refuses(kw, status):
    got, message = _groups(**kw)
    assert got == status and message
