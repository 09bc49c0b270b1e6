"""The linear on both sides of the sizes where its variants change: exact sums, and one result for a token whichever runs it."""
import pytest
import torch

import layer_reference as ref
from layer_gpu_helpers import TYPES, host
from test_gpu_linear import make, run

pytestmark = pytest.mark.gpu


def exact_and_alone(M, N, K, group, affine, scales, kind):
    # |x| <= 3, w < 40, K <= 2056: every partial sum is a multiple of 2^-2 below 2^20
    w, s, b, x, wh = make(M + N + K + group, M, N, K, group, affine, kind, scales, exact=True)
    got = run(w, s, b, x, M, N, K, group, kind)
    want, _ = ref.linear(wh, host(s), None if b is None else host(b), group, host(x), N, K)
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(TYPES[kind]))
    # real values: the last token of the batch has the bits that it has alone
    w, s, b, x, _ = make(M + N, M, N, K, group, affine, kind, scales)
    last = run(w, s, b, x[M - 1:].contiguous(), 1, N, K, group, kind)
    assert torch.equal(run(w, s, b, x, M, N, K, group, kind)[M - 1:], last)


@pytest.mark.parametrize("group,affine", [(32, True), (128, False)])
@pytest.mark.parametrize("M,N,K", [(8, 4096, 2056), (8, 4097, 2056), (16, 4089, 1032), (16, 4112, 1032), (11, 5990, 520), (16, 6011, 264)])
def test_waves_along_the_row(M, N, K, group, affine):
    exact_and_alone(M, N, K, group, affine, "bf16", "bf16")


# (M, N): one and two row tiles of a wave for up to 8, 16, 32 and 64 tokens of a work-group
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(5, 16384), (5, 16411), (8, 28817), (7, 65555), (9, 8209), (16, 16411), (12, 65555), (29, 8209),
                                 (40, 4001), (70, 8209)])
def test_row_tiles(M, N, group, affine, kind):
    exact_and_alone(M, N, 392, group, affine, "bf16" if group == 64 else "f32", kind)
