"""The router's validators answer as its calls do for the type they are asked about (host only)."""
import pytest

import quantized_moe_expert_q4_amd as q4

X, IDS, W, D = 1 << 24, 1 << 26, 1 << 27, 1 << 28     # fake device addresses: every call below is refused before a launch


@pytest.mark.parametrize("off,xdtype,status", [(1, "bf16", q4.Q4_ERR_ALIGNMENT), (2, "bf16", q4.Q4_OK),
                                               (1, "f32", q4.Q4_ERR_ALIGNMENT), (2, "f32", q4.Q4_ERR_ALIGNMENT),
                                               (4, "f32", q4.Q4_OK)])
def test_alignment_of_the_logits(off, xdtype, status):
    assert q4.validate_route(X + off, 4, 64, 8, IDS, W, xdtype=xdtype) == status
    for a, b in ((X + off, D), (X, D + off)):
        assert q4.validate_route_backward(a, 4, 64, 8, IDS, b, d_weights=W, xdtype=xdtype) == status
    if status == q4.Q4_OK:
        return
    with pytest.raises(q4.Q4Error) as e:
        q4.route(X + off, 4, 64, 8, IDS, W, xdtype=xdtype, stream=0)
    assert e.value.status == status
    for a, b in ((X + off, D), (X, D + off)):
        with pytest.raises(q4.Q4Error) as e:
            q4.route_backward(a, 4, 64, 8, IDS, b, d_weights=W, xdtype=xdtype, stream=0)
        assert e.value.status == status


def test_types_that_do_not_exist():
    with pytest.raises(ValueError):
        q4.validate_route(X, 4, 64, 8, IDS, W, xdtype="f16")
    with pytest.raises(ValueError):
        q4.validate_route_backward(X, 4, 64, 8, IDS, D, d_weights=W, xdtype="f16")
