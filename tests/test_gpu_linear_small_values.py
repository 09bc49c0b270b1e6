"""The linear with float tokens near the lower end of the range."""
import numpy as np
import pytest
import torch

from layer_gpu_helpers import dev, host
from test_gpu_linear import run
from test_gpu_linear_float import full_digits

pytestmark = pytest.mark.gpu


def test_the_smallest_tokens():
    # tokens are taken to a multiple of 2^-133 towards zero: all digits from 2^-110 up
    N, K, low = 16, 32, range(-133, -95)
    rng = np.random.default_rng(5)
    w = torch.full((N, K // 2), 0x99, dtype=torch.uint8, device="cuda")     # q - 8 = 1
    for e in low:
        for M in (1, 4, 20):
            x = np.zeros((M, K))
            x[np.arange(M), rng.integers(0, K, size=M)] = full_digits(rng, M, e, e + 1)
            xt = dev(x)
            got = run(w, torch.ones(N, 1, device="cuda"), None, xt, M, N, K, 32, "f32")
            kept = np.ldexp(np.trunc(np.ldexp(host(xt), 133)), -133).sum(1)
            assert np.array_equal(host(got), np.repeat(kept[:, None], N, 1)), (e, M)
