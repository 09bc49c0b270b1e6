"""The precision of the linear with float tokens: every digit of a token counts."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from layer_gpu_helpers import dev, host
from test_gpu_linear import make, run

pytestmark = pytest.mark.gpu

# (M, N, K): every number of tokens a work-group takes, one and two row tiles of a wave, long rows
SHAPES = [(1, 33, 520), (4, 70, 1032), (6, 97, 4104), (16, 48, 264), (40, 200, 2056), (7, 12007, 264), (16, 9001, 136),
          (33, 9619, 264), (2, 24, 33000)]


def full_digits(rng, shape, low, high):
    """Floats of 24 significant bits, the last one set, 2^low up to 2^high in size."""
    m = rng.integers(1 << 22, 1 << 23, size=shape) * 2 + 1
    return np.ldexp(m.astype(np.float64), rng.integers(low, high, size=shape) - 23) * rng.choice([-1.0, 1.0], size=shape)


def pack(q):
    return torch.from_numpy((q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)).cuda()


@pytest.mark.parametrize("scales", ["bf16", "f32"])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_every_digit_arrives(M, N, K, group, affine, scales):
    # one value of 24 bits a token, weights that are powers of two: the result
    # is one product, exact, and so is every sum on the way to it
    rng = np.random.default_rng(M * N + K + group)
    G = -(-K // group)
    at = rng.integers(0, K, size=M)
    x = np.zeros((M, K))
    x[np.arange(M), at] = full_digits(rng, M, -60, 60)
    s = 2.0 ** rng.integers(-3, 4, size=(N, G))
    off = rng.choice([-8, -4, -2, -1, 1, 2, 4], size=(N, G))       # q - 8 of the whole group
    q = np.repeat(off + 8, group, axis=1)[:, :K]
    weight = rng.choice([-4, -2, -1, 1, 2, 4], size=(N, G)) if affine else off
    b = dev(s * (weight - (off + 8)), scales) if affine else None
    got = run(pack(q), dev(s, scales), b, dev(x), M, N, K, group, "f32")
    want = x[np.arange(M), at][:, None] * (s * weight)[:, at // group].T
    assert np.array_equal(host(got), want)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weights_of_zero_give_zero(M, N, K, affine):
    # q = 8 without biases, or with a bias of -8 s: nothing of the tokens may be left over
    rng = np.random.default_rng(K)
    s = dev(rng.uniform(0.005, 0.02, size=(N, -(-K // 64))), "bf16")
    w = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    got = run(w, s, -8 * s if affine else None, dev(rng.normal(size=(M, K)) + 3.0), M, N, K, 64, "f32")
    assert (got == 0).all()


def rms(a):
    return float(np.sqrt(np.mean(np.square(a))))


@pytest.mark.parametrize("scales", ["bf16", "f32"])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("M,N,K,group", [(1, 1536, 4096, 64), (4, 300, 7168, 128), (6, 97, 4104, 32), (16, 512, 6144, 128),
                                         (40, 200, 4096, 64), (64, 96, 7168, 32), (6, 40, 65536, 32), (3, 70, 33000, 128)])
def test_error_over_all_results(M, N, K, group, affine, scales):
    # terms of random sign: sums of n of them are about sqrt(n) of one.  A
    # rounding of 2^-23 (the matrix unit may truncate) for each of the three
    # parts' products, spread over a group's partial sums, comes to sqrt(group /
    # 2) steps of 2^-23 of the result's rms, the group sums on the way to the
    # total to at most sqrt(K / group), the result's own rounding to half of one.
    # (x without its lowest eight bits would be 2^-16 / 1.44 = 90 such steps off.)
    w, s, b, x, wh = make(M + N + K + group, M, N, K, group, affine, "f32", scales)
    got = run(w, s, b, x, M, N, K, group, "f32")
    want, _ = ref.linear(wh, host(s), None if b is None else host(b), group, host(x), N, K)
    steps = (group / 2) ** 0.5 + (K / group) ** 0.5 + 0.5
    assert rms(host(got) - want) <= steps * 2.0 ** -23 * rms(want)
