"""Every variant of the adapters' kernels (tiles of 16 or 64 rows, one launch or two, parts of the long sum,
slices of the results, ranks, types and directions) and the calls' limits, with exact sums, on an MI355X."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import TYPES, host, i32, replayed
from test_gpu_adapter import Case

pytestmark = pytest.mark.gpu

RANKS = (8, 24, 56, 72)                  # one of each kernel: up to 16, 32, 64 ranks in a pass, and more than a pass of 64


def exact(c, forward=True, backward=True):
    """Both calls against the 64-bit forms, to the bit: every sum is below 2^24 of its smallest unit (a quarter),
    and the values between the products have 16 bits, which the reference shows for these inputs."""
    def low(*arrays):
        assert all(np.abs(4 * a).max() < 2 ** 24 and np.array_equal(4 * a, np.rint(4 * a)) for a in arrays)
    kind = c.kind
    if forward:
        out, hidden = c.outputs()
        c.forward(out, hidden)
        want, mag, h, hm = c.want_forward()
        low(mag, hm)
        assert np.abs(h).max() * 4 < 2 ** 15
        torch.cuda.synchronize()
        assert torch.equal(hidden.cpu().double(), torch.from_numpy(h))
        assert torch.equal(out.cpu(), torch.from_numpy(want).float().to(TYPES[kind]))
    if backward:
        grads = c.gradients()
        c.backward(*grads)
        (d_x, d_a, d_b), mags = c.want_backward()
        low(*mags)
        d, b, s, n = host(c.d_out), host(c.b), c.host_scales(), c.sizes[4]
        assert all(np.abs(s[i] * (d[t] @ b[i])).max() * 4 < 2 ** 15 for t, i in enumerate(c.host_ids()) if 0 <= i < n)
        torch.cuda.synchronize()
        assert torch.equal(grads[0].cpu(), torch.from_numpy(d_x).float().to(TYPES[kind]))
        assert torch.equal(grads[1].cpu().double(), torch.from_numpy(d_a))
        assert torch.equal(grads[2].cpu().double(), torch.from_numpy(d_b))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("ids", ["mixed", "sorted", None])
@pytest.mark.parametrize("R", (8, 16, 24, 40, 64, 72, 200))
def test_tiles_of_64_rows_with_parts_and_slices(R, ids, kind):
    # 17 tiles: three parts of the sum either way, three slices of the results; N and the rows end inside a tile
    exact(Case(R, 1030, 1099, 1096, R, 3, kind, ids=ids, exact=True))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("R", RANKS)
def test_tiles_of_64_rows_in_one_part(R, kind):
    exact(Case(R, 1100, 71, 136, R, 5, kind, exact=True))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("M", [40, 70])
@pytest.mark.parametrize("R", RANKS)
def test_two_launches_of_tiles_of_16_rows(R, M, backward, kind):
    # the first product's matrix is above 256 KB, so that its sum is shared by work-groups
    size = 2 if kind == "bf16" else 4
    long = ((1 << 18) // (R * size) // 8 + 1) * 8 + 512
    N, K = (long + 3, 64) if backward else (67, long)
    exact(Case(R + M, M, N, K, R, 3, kind, exact=True), not backward, backward)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M", [300, 1100, 2600])
def test_mixed_rows_of_many_adapters(M, kind):
    # every window of 256 rows holds most of the adapters
    exact(Case(M, M, 70, 72, 16, 200, kind, exact=True))


@pytest.mark.parametrize("M,N,K,R,n", [
    (65535, 8, 8, 8, 3), (5, 1 << 20, 8, 8, 2), (3, 9, 65536, 8, 2), (70, 8, 8, 8, 65535), (1100, 33, 40, 8, 65535),
    (40, 16, 16, 256, 4096)])
def test_limits(M, N, K, R, n):
    exact(Case(M + n, M, N, K, R, n, "bf16", exact=True))


def test_adapters_no_row_names():
    # one adapter of 65535 has all rows: the others' gradients are zeros
    c = Case(4, 600, 24, 16, 8, 65535, "bf16", exact=True)
    c.ids = i32(np.full(600, 65534))
    exact(c)
    d_b = c.gradients()[2]
    q4.adapter_backward(c.d_out, c.a, c.b, *c.sizes, c.ws, c.need, hidden=c.h, d_b=d_b, adapter_ids=c.ids, scales=c.scales)
    torch.cuda.synchronize()
    _, _, want = c.want_backward()[0]
    assert torch.equal(d_b.cpu().double(), torch.from_numpy(want))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,R", [(1030, 1099, 1096, 24), (1030, 1099, 1096, 72), (70, 2503, 2504, 64), (70, 300, 264, 40)])
def test_infinities_and_nan_stay_where_they_are(M, N, K, R, kind):
    # the calls again with one adapter, a row of x, of base and of d_out made infinite or NaN: all else keeps its bits
    n, bad = 5, 2
    c = Case(M + R, M, N, K, R, n, kind)

    def run():
        o = [*c.outputs(), *c.gradients()]
        c.forward(*o[:2])
        c.backward(*o[2:])
        torch.cuda.synchronize()
        return o
    clean = run()
    ids = host(c.ids)
    free = [int(np.flatnonzero(ids == i)[1]) for i in (0, 1)]           # rows of the adapters 0 and 1
    none = int(np.flatnonzero((ids < 0) | (ids >= n))[0])
    c.a[bad, R - 1, K - 1], c.b[bad, 0, 0] = float("nan"), float("inf")
    c.x[free[0], 3], c.d_out[free[1], N - 1] = float("inf"), float("nan")
    c.x[none], c.d_out[none] = float("nan"), float("inf")               # a row without an adapter
    out, hidden, d_x, d_a, d_b = run()
    torch.cuda.synchronize()
    row = np.arange(M)
    same = torch.from_numpy((ids != bad) & (row != free[0])).cuda()
    assert torch.equal(out[same], clean[0][same]) and torch.equal(hidden[same], clean[1][same])
    assert not torch.isfinite(hidden[free[0]]).any()
    same = torch.from_numpy((ids != bad) & (row != free[1])).cuda()
    assert torch.equal(d_x[same], clean[2][same])
    assert not torch.isfinite(d_x[free[1]].float()).any()
    for i in (3, 4):                     # the adapters without any such row
        assert torch.equal(d_a[i], clean[3][i]) and torch.equal(d_b[i], clean[4][i])
    assert torch.equal(d_b[0], clean[4][0])                             # x has no part in it
    assert not torch.isfinite(d_a[0, :, 3]).any() and not torch.isfinite(d_b[1, N - 1]).any()


@pytest.mark.parametrize("M,N,K,R", [(1030, 1099, 1096, 24), (70, 2503, 2504, 64)])
def test_two_launches_in_a_graph(M, N, K, R):
    c = Case(M, M, N, K, R, 3, "bf16")
    outs = [*c.outputs(), *c.gradients()]

    def both():
        c.forward(*outs[:2])
        c.backward(*outs[2:])
    both()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for got in replayed(both, outs):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
