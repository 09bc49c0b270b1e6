"""The gradient of the 4-bit linear's input against its 64-bit form on an MI355X."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
import tuning_reference as tune
from layer_gpu_helpers import TYPES, check, dev, host, nan_like, replayed
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu


def make(seed, M, N, K, group, affine, kind, scales, exact=False):
    """Host weights and device scales, biases and d_out.  With `exact`, small
    whole numbers and powers of two: every weight is exact in bf16, every sum in F32."""
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    G = -(-K // group)
    if exact:
        s = 2.0 ** rng.integers(-2, 2, size=(N, G))
        b = rng.integers(-4, 5, size=(N, G)).astype(np.float64) if affine else None
        d = rng.integers(-3, 4, size=(M, N)).astype(np.float64)
    else:
        s = rng.uniform(0.005, 0.02, size=(N, G))
        b = -7.5 * s + 0.01 * rng.normal(size=(N, G)) if affine else None
        d = rng.normal(size=(M, N))
    cast = lambda a, kind: None if a is None else dev(a, kind)
    return torch.from_numpy(w).cuda(), cast(s, scales), cast(b, scales), cast(d, kind), w


def workspace(M, N, K):
    n = q4.linear_backward_workspace_bytes(M, N, K)
    ws = aligned_empty(n, 256)
    ws.fill_(0xFF)                       # NaNs
    return ws, n


def run(w, s, b, d, M, N, K, group, kind):
    d_x = nan_like((M, K), kind)
    q4.linear_backward(w, s, d, M, N, K, group, d_x, *workspace(M, N, K), biases=b, xdtype=kind)
    torch.cuda.synchronize()
    return d_x


def tolerance(want, mag, N, kind):
    # the output's rounding, each weight's rounding to the products' type, and a
    # step (2^-23: the matrix unit may truncate) of the magnitude for each
    # addition a term can pass: N of them at most, and 16 parts
    return ref.HALF_STEP[kind] * np.abs(want) + (ref.HALF_STEP[kind] + (N + 16) * 2.0 ** -23) * mag


SHAPES = [  # M, N, K: one token and one row; odd rows; ends inside tiles of tokens, columns and steps
    (1, 1, 8), (1, 17, 40), (2, 64, 128), (3, 33, 136), (15, 65, 256), (16, 128, 264), (17, 31, 520), (31, 130, 96),
    (33, 257, 1000), (64, 40, 392), (65, 300, 168), (100, 129, 136), (128, 64, 128), (130, 19, 2056), (260, 515, 72)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K, group, kind):
    # weights are multiples of 1/4 up to 34, |d| <= 3, N <= 515: sums below 2^24 quarters
    for affine, scales in ((False, "bf16"), (True, "f32")):
        w, s, b, d, wh = make(M * 1000 + K + group, M, N, K, group, affine, kind, scales, exact=True)
        got = run(w, s, b, d, M, N, K, group, kind)
        want, _ = tune.linear_backward(wh, host(s), None if b is None else host(b), group, host(d), N, K)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(TYPES[kind])), (affine, scales)


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("scales", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,group", [(1, 4096, 1536, 64), (5, 6147, 520, 32), (40, 2049, 1032, 128), (70, 1536, 776, 64),
                                         (300, 1000, 1544, 32)])
def test_real_values(M, N, K, group, kind, scales, affine):
    w, s, b, d, wh = make(M + N + K, M, N, K, group, affine, kind, scales)
    got = run(w, s, b, d, M, N, K, group, kind)
    want, mag = tune.linear_backward(wh, host(s), None if b is None else host(b), group, host(d), N, K)
    check(host(got), want, tolerance(want, mag, N, kind), "d_x")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_is_the_adjoint_of_the_linear(kind):
    # <d_out, linear(x)> = <d_x, x>, exactly: whole numbers whose results the types hold
    M, N, K, group = 6, 40, 64, 32
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)).cuda()
    s = torch.ones(N, K // group, device="cuda")
    x = torch.zeros(M, K, dtype=TYPES[kind], device="cuda")
    d = torch.zeros(M, N, dtype=TYPES[kind], device="cuda")
    for m in range(M):                   # a few entries a row: results stay below 2^8
        x[m, rng.integers(0, K, 3)] = 2.0
        d[m, rng.integers(0, N, 3)] = -3.0
    out, d_x = nan_like((M, N), kind), run(w, s, None, d, M, N, K, group, kind)
    q4.linear(w, s, x, M, N, K, group, out, xdtype=kind)
    torch.cuda.synchronize()
    assert float((out.double() * d.double()).sum()) == float((d_x.double() * x.double()).sum())


def test_against_differences():
    # the objective sum(d_out * linear(x)) is linear in x: differences of any step are its gradient
    M, N, K, group = 3, 70, 72, 32
    w, s, b, d, wh = make(5, M, N, K, group, True, "f32", "f32")
    got = host(run(w, s, b, d, M, N, K, group, "f32"))
    W = tune.dense_weights(wh, host(s), host(b), group, N, K)
    rng = np.random.default_rng(1)
    x, dh = rng.normal(size=(M, K)), host(d)
    f = lambda x: float((dh * (x @ W.T)).sum())
    for m, k in ((0, 0), (1, 71), (2, 33)):
        e = np.zeros((M, K))
        e[m, k] = 0.5
        assert abs(f(x + e) - f(x - e) - got[m, k]) <= 1e-4 * (1 + abs(got[m, k]))


def test_nan_and_infinity_stay_in_their_token():
    M, N, K = 70, 200, 136
    w, s, b, d, wh = make(9, M, N, K, 64, False, "bf16", "bf16")
    d[1, 100] = float("nan")
    d[69, 7] = float("inf")
    got = host(run(w, s, b, d, M, N, K, 64, "bf16"))
    assert np.isnan(got[1]).all() and not np.isfinite(got[69]).any()
    keep = [i for i in range(M) if i not in (1, 69)]
    want, mag = tune.linear_backward(wh, host(s), None, 64, host(d)[keep], N, K)
    check(got[keep], want, tolerance(want, mag, N, "bf16"), "rows")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_at_any_element_and_nothing_beside_the_result(kind):
    M, N, K, group = 21, 71, 136, 64
    w, s, b, d, wh = make(12, M, N, K, group, True, kind, "bf16")
    raw = torch.empty(d.numel() + 1, dtype=d.dtype, device="cuda")
    raw[1:] = d.flatten()
    sraw, braw = (torch.empty(a.numel() + 1, dtype=a.dtype, device="cuda") for a in (s, b))
    sraw[1:], braw[1:] = s.flatten(), b.flatten()
    d_x = torch.full((M * K + 64,), 99.0, dtype=d.dtype, device="cuda")
    q4.linear_backward(w, sraw[1:], raw[1:], M, N, K, group, d_x[:M * K], *workspace(M, N, K), biases=braw[1:], xdtype=kind)
    torch.cuda.synchronize()
    want, mag = tune.linear_backward(wh, host(s), host(b), group, host(d), N, K)
    got = host(d_x)
    check(got[:M * K].reshape(M, K), want, tolerance(want, mag, N, kind), "d_x")
    assert (got[M * K:] == 99).all()


def test_a_workspace_for_the_largest_batch_serves_smaller_ones():
    N, K = 520, 264
    big = [q4.linear_backward_workspace_bytes(M, N, K) for M in (1, 16, 17, 64, 65, 128, 1000, 5000, 65535)]
    assert big == sorted(big)
    assert q4.linear_backward_workspace_bytes(100, N, K) >= q4.linear_backward_workspace_bytes(100, 8, K)


@pytest.mark.parametrize("M", [5, 300])
def test_runs_in_a_graph_and_on_another_stream(M):
    N, K, group = 1000, 264, 32
    w, s, b, d, _ = make(13, M, N, K, group, True, "bf16", "f32")
    want = run(w, s, b, d, M, N, K, group, "bf16")
    d_x, ws = nan_like((M, K), "bf16"), workspace(M, N, K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q4.linear_backward(w, s, d, M, N, K, group, d_x, *ws, biases=b, stream=side)
    side.synchronize()
    assert torch.equal(d_x, want)
    for got, in replayed(lambda: q4.linear_backward(w, s, d, M, N, K, group, d_x, *ws, biases=b), [d_x]):
        assert torch.equal(got, want)


def test_refusals_enqueue_nothing():
    w, s, b, d, _ = make(14, 1, 16, 64, 64, False, "bf16", "bf16")
    d_x, (ws, n) = nan_like((1, 64), "bf16"), workspace(1, 16, 64)
    with pytest.raises(q4.Q4Error):
        q4.linear_backward(w, s, d, 1, 16, 64, 48, d_x, ws, n)
    with pytest.raises(q4.Q4Error):
        q4.linear_backward(w, s, d, 1, 16, 64, 64, d_x, ws, n - 256)
    with pytest.raises(ValueError):
        q4.linear_backward(w, s, d, 1, 17, 64, 64, d_x, ws, n)
    torch.cuda.synchronize()
    assert torch.isnan(d_x.float()).all()
