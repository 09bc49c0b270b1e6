"""The linear's variants by rows, tokens and lengths: exact sums, and one result for a token whichever runs it."""
import pytest
import torch

import layer_reference as ref
from layer_gpu_helpers import TYPES, check, host
from test_gpu_linear import make, run, tolerance

pytestmark = pytest.mark.gpu


# one to many waves along K, one and two row tiles, 4 to 64 tokens of a work-group, odd row ends
SHAPES = [(1, 33000, 264), (2, 16391, 520), (4, 40003, 72), (3, 1001, 2056), (7, 6011, 520), (8, 12291, 264), (16, 6011, 776),
          (13, 12007, 136), (20, 2577, 520), (32, 12019, 264), (40, 9619, 520), (64, 14341, 264), (65, 2600, 136),
          (130, 9601, 72)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K, kind):
    # |x| <= 3, w < 40, K <= 2056: every partial sum is a multiple of 2^-2 below 2^20
    for group, affine, scales in ((32, True, "bf16"), (64, False, "f32"), (128, True, "f32"), (128, False, "bf16")):
        w, s, b, x, wh = make(M + N + K + group, M, N, K, group, affine, kind, scales, exact=True)
        got = run(w, s, b, x, M, N, K, group, kind)
        want, _ = ref.linear(wh, host(s), None if b is None else host(b), group, host(x), N, K)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(TYPES[kind])), (group, affine, scales)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,group", [(1, 40, 65536, 32), (1, 3, 20008, 64), (3, 70, 33000, 128), (6, 50, 20008, 32),
                                         (16, 20, 65536, 128), (33, 17, 33000, 64)])
def test_long_rows(M, N, K, group, kind):
    # the scales of such rows pass through LDS in several parts
    w, s, b, x, wh = make(K + M, M, N, K, group, True, kind, "f32")
    got = run(w, s, b, x, M, N, K, group, kind)
    want, mag = ref.linear(wh, host(s), host(b), group, host(x), N, K)
    check(host(got), want, tolerance(want, mag, K, group, kind), "linear")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2600, 6011, 12007])
def test_a_token_has_one_result(N, kind):
    K, group = 1288, 64
    w, s, b, x, _ = make(N, 66, N, K, group, True, kind, "bf16")
    whole = run(w, s, b, x, 66, N, K, group, kind)
    for M in (1, 3, 4, 7, 8, 15, 16, 27, 32, 50, 64):
        assert torch.equal(run(w, s, b, x[:M].contiguous(), M, N, K, group, kind), whole[:M]), M


@pytest.mark.parametrize("M", [1, 6, 20])
@pytest.mark.parametrize("K,group", [(520, 32), (264, 128), (8, 64)])
def test_ends_of_buffers(M, K, group):
    # odd numbers of groups (their scales at odd addresses), and inputs that end where their buffers do
    N = 37
    w, s, b, x, wh = make(M + K, M, N, K, group, True, "bf16", "bf16")
    s_raw, b_raw = (torch.full((s.numel() + 1,), float("nan"), dtype=s.dtype, device="cuda") for _ in range(2))
    s_raw[1:], b_raw[1:] = s.flatten(), b.flatten()
    got = run(w, s_raw[1:], b_raw[1:], x, M, N, K, group, "bf16")
    want, mag = ref.linear(wh, host(s), host(b), group, host(x), N, K)
    check(host(got), want, tolerance(want, mag, K, group, "bf16"), "linear")
