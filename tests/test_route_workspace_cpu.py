"""The router's workspace: what is allocated for the largest batch serves every smaller one (host only)."""
import pytest

import quantized_moe_expert_q4_amd as q4

# around every change of lanes, widths and work-groups
TOKENS = sorted({m + d for m in (1, 8, 32, 256, 512, 1024, 2048, 4096, 6000, 8192, 16384, 1 << 20, 1 << 24) for d in (-1, 0, 1)
                 if 1 <= m + d <= 1 << 24})
EXPERTS = [1, 2, 15, 16, 17, 63, 64, 65, 128, 255, 256, 257, 511, 512, 513, 1023, 1024]


@pytest.mark.parametrize("E", EXPERTS)
def test_more_tokens_need_no_less(E):
    sizes = [q4.route_workspace_bytes(M, E) for M in TOKENS]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("M", TOKENS)
def test_more_experts_need_no_less(M):
    sizes = [q4.route_workspace_bytes(M, E) for E in EXPERTS]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("E", [64, 65, 128, 256, 257])
@pytest.mark.parametrize("most", [4097, 6000, 1 << 20])
def test_a_workspace_of_the_largest_batch_is_accepted(E, most):
    n = q4.route_workspace_bytes(most, E)
    for M in (1, 1500, 4095, 4096, 4097, most):
        if M <= most:
            status = q4.validate_route(1 << 24, M, E, 8, 1 << 26, 1 << 27, counts=1 << 28, workspace=1 << 29, workspace_bytes=n)
            assert status == q4.Q4_OK, (M, q4.last_error())
