"""The group-scaled 4-bit linear against its 64-bit form on an MI355X."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import TYPES, check, dev, host, nan_like, replayed

pytestmark = pytest.mark.gpu


def make(seed, M, N, K, group, affine, x, scales, exact=False):
    """Host weights, scales, biases and x as the types hold them.  With
    `exact`, small whole numbers and powers of two: every sum is exact in F32."""
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    G = -(-K // group)
    if exact:
        s = 2.0 ** rng.integers(-2, 2, size=(N, G))
        b = rng.integers(-4, 5, size=(N, G)).astype(np.float64) if affine else None
        xv = rng.integers(-3, 4, size=(M, K)).astype(np.float64)
    else:
        s = rng.uniform(0.005, 0.02, size=(N, G))
        b = -7.5 * s + 0.01 * rng.normal(size=(N, G)) if affine else None
        xv = rng.normal(size=(M, K)) * np.where(rng.random((1, K)) < 0.01, 16, 1)
    cast = lambda a, kind: None if a is None else dev(a, kind)
    return torch.from_numpy(w).cuda(), cast(s, scales), cast(b, scales), cast(xv, x), w


def run(w, s, b, x, M, N, K, group, kind, out=None):
    out = nan_like((M, N), kind) if out is None else out
    q4.linear(w, s, x, M, N, K, group, out, biases=b, xdtype=kind)
    torch.cuda.synchronize()
    return out


def tolerance(want, mag, K, group, kind):
    # rounding of the output, plus one F32 step (2^-23: the matrix unit may
    # truncate) of the magnitude for each addition a term can pass through:
    # at most 2 per weight of its group, one per group and 32 to join waves
    steps = 2 * group + -(-K // group) + 32
    return ref.HALF_STEP[kind] * np.abs(want) + steps * 2.0 ** -23 * mag


SHAPES = [  # M, N, K: one token and one row; short and odd ends of rows, groups, tiles and units
    (1, 1, 8), (1, 16, 32), (2, 17, 40), (3, 33, 128), (4, 15, 136), (5, 64, 256), (7, 31, 264), (8, 100, 512),
    (16, 48, 1000), (17, 65, 768), (31, 130, 1288), (33, 70, 520), (64, 257, 2056), (65, 19, 392), (130, 40, 256)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K, group, kind):
    # |x| <= 3, w < 40, K <= 2056: every partial sum is a multiple of 2^-2 below 2^20
    for affine, scales in ((False, "bf16"), (True, "f32")):
        w, s, b, x, wh = make(M * 1000 + K + group, M, N, K, group, affine, kind, scales, exact=True)
        got = run(w, s, b, x, M, N, K, group, kind)
        want, _ = ref.linear(wh, host(s), None if b is None else host(b), group, host(x), N, K)
        want = torch.from_numpy(want).to(TYPES[kind])
        assert torch.equal(got.cpu(), want), (affine, scales)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("scales", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,group", [(1, 1536, 4096, 64), (1, 4099, 1032, 32), (4, 300, 7168, 128), (6, 97, 4104, 32),
                                         (16, 512, 6144, 128), (40, 200, 4096, 64), (64, 96, 7168, 32)])
def test_real_values(M, N, K, group, kind, scales, affine):
    w, s, b, x, wh = make(M + N + K, M, N, K, group, affine, kind, scales)
    got = run(w, s, b, x, M, N, K, group, kind)
    want, mag = ref.linear(wh, host(s), None if b is None else host(b), group, host(x), N, K)
    check(host(got), want, tolerance(want, mag, K, group, kind), "linear")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_tokens_do_not_depend_on_the_batch(kind):
    N, K, group = 131, 4104, 64
    w, s, b, x, _ = make(3, 70, N, K, group, True, kind, "bf16")
    whole = run(w, s, b, x, 70, N, K, group, kind)
    for M in (1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 64):
        part = run(w, s, b, x[:M].contiguous(), M, N, K, group, kind)
        assert torch.equal(part, whole[:M]), M


def test_nan_and_infinity_stay_in_their_token():
    N, K = 64, 512
    w, s, b, x, wh = make(9, 6, N, K, 128, False, "bf16", "bf16")
    x[1, 100] = float("nan")
    x[4, 7] = float("inf")
    got = host(run(w, s, b, x, 6, N, K, 128, "bf16"))
    assert np.isnan(got[1]).all() and not np.isfinite(got[4]).any()
    keep = [0, 2, 3, 5]
    want, mag = ref.linear(wh, host(s), None, 128, host(x)[keep], N, K)
    check(got[keep], want, tolerance(want, mag, K, 128, "bf16"), "rows")


def test_large_and_tiny_values():
    # products up to 2^100 and down to 2^-100: F32 range, no overflow of the sums
    N, K = 40, 256
    for e in (100, -100):
        w, s, b, x, wh = make(11, 3, N, K, 64, False, "f32", "f32")
        x = x * 2.0 ** e
        got = run(w, s, b, x, 3, N, K, 64, "f32")
        want, mag = ref.linear(wh, host(s), None, 64, host(x), N, K)
        check(host(got), want, tolerance(want, mag, K, 64, "f32"), f"2^{e}")


def test_zero_scale_rows_and_unaligned_ends():
    # output rows that start at any 2-byte address, and scales at odd multiples of their size
    M, N, K = 3, 21, 136
    w, s, b, x, wh = make(12, M, N, K, 64, False, "bf16", "bf16")
    s[5] = 0
    raw = torch.empty(s.numel() + 1, dtype=s.dtype, device="cuda")
    raw[1:] = s.flatten()
    out = torch.full((M * N + 3,), 99.0, dtype=torch.bfloat16, device="cuda")
    q4.linear(w, raw[1:], x, M, N, K, 64, out[1:1 + M * N])
    torch.cuda.synchronize()
    want, mag = ref.linear(wh, host(s), None, 64, host(x), N, K)
    got = host(out)
    check(got[1:1 + M * N].reshape(M, N), want, tolerance(want, mag, K, 64, "bf16"), "linear")
    assert got[0] == 99 and (got[1 + M * N:] == 99).all()
    assert (got[1:1 + M * N].reshape(M, N)[:, 5] == 0).all()


def test_runs_in_a_graph_and_on_another_stream():
    M, N, K, group = 5, 300, 1032, 32
    w, s, b, x, _ = make(13, M, N, K, group, True, "bf16", "f32")
    want = run(w, s, b, x, M, N, K, group, "bf16")
    out = nan_like((M, N), "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q4.linear(w, s, x, M, N, K, group, out, biases=b, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    for got, in replayed(lambda: q4.linear(w, s, x, M, N, K, group, out, biases=b), [out]):
        assert torch.equal(got, want)


def test_refusals_enqueue_nothing():
    w, s, b, x, _ = make(14, 1, 16, 64, 64, False, "bf16", "bf16")
    out = nan_like((1, 16), "bf16")
    with pytest.raises(q4.Q4Error):
        q4.linear(w, s, x, 1, 16, 64, 48, out)
    with pytest.raises(ValueError):
        q4.linear(w, s, x, 1, 17, 64, 64, out)
    torch.cuda.synchronize()
    assert torch.isnan(out.float()).all()
