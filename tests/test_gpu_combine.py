"""Combination of expert outputs and its gradients against their 64-bit forms on an MI355X."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import check, dev, host, i32, nan_like, replayed

pytestmark = pytest.mark.gpu
SLOTS = 9


def make(M, K, H, kind, ids=True, base=True):
    rng = np.random.default_rng(M * 31 + K * 7 + H)
    y, w = dev(rng.normal(size=(M, K, H)), kind), dev(rng.normal(size=(M, K)))
    i = rng.integers(-1, SLOTS + 1, size=(M, K)) if ids else None
    if ids:
        i[M // 2] = -1                                        # a token with nothing
        y[torch.from_numpy((i < 0) | (i >= SLOTS)).cuda()] = float("nan")   # left-out rows are never read
    b = dev(rng.normal(size=(M, H)), kind) if base else None
    return y, w, i, b


def tol(want, mag, steps, kind):
    return ref.HALF_STEP[kind] * np.abs(want) + steps * 2.0 ** -24 * mag


SHAPES = [(1, 1, 8), (1, 8, 4096), (2, 3, 16), (3, 8, 264), (5, 6, 1032), (7, 2, 520), (33, 4, 2056), (64, 10, 128),
          (3, 64, 72), (300, 8, 136), (2, 1, 65536), (1, 5, 8192)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("ids", [False, True])
@pytest.mark.parametrize("M,K,H", SHAPES)
def test_combine(M, K, H, ids, kind):
    for with_base in (False, True):
        y, w, i, b = make(M, K, H, kind, ids, with_base)
        out = nan_like((M, H), kind)
        q4.combine(y, w, M, K, H, out, slot_ids=i32(i) if ids else None, num_slots=SLOTS, base=b, xdtype=kind)
        torch.cuda.synchronize()
        want, mag = ref.combine(np.nan_to_num(host(y)), host(w), i, SLOTS, None if b is None else host(b))
        check(host(out), want, tol(want, mag, K + 1, kind), "combine")      # one rounding a term


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("ids", [False, True])
@pytest.mark.parametrize("M,K,H", SHAPES)
def test_combine_backward(M, K, H, ids, kind):
    y, w, i, _ = make(M, K, H, kind, ids)
    d = dev(np.random.default_rng(1).normal(size=(M, H)), kind)
    kw = dict(slot_ids=i32(i) if ids else None, num_slots=SLOTS, xdtype=kind)
    d_y, d_w = nan_like((M, K, H), kind), nan_like((M, K))
    q4.combine_backward(d, y, w, M, K, H, d_y=d_y, d_weights=d_w, **kw)
    torch.cuda.synchronize()
    want_y, want_w, mag = ref.combine_backward(host(d), np.nan_to_num(host(y)), host(w), i, SLOTS)
    check(host(d_y), want_y, tol(want_y, np.abs(want_y), 1, kind), "d_y")   # the F32 product, then its type
    # a lane adds at most H / 64 products (or all eight of a short row), then 6 + 16 joins
    check(host(d_w), want_w, (H / 64 + 32) * 2.0 ** -24 * mag + 0 * want_w, "d_weights")
    only_w, only_y = nan_like((M, K)), nan_like((M, K, H), kind)
    q4.combine_backward(d, y, w, M, K, H, d_weights=only_w, **kw)
    q4.combine_backward(d, None, w, M, K, H, d_y=only_y, **kw)
    torch.cuda.synchronize()
    assert torch.equal(only_w, d_w) and torch.equal(only_y, d_y)


def test_base_may_be_the_output():
    y, w, i, b = make(6, 4, 264, "bf16")
    out = nan_like((6, 264), "bf16")
    q4.combine(y, w, 6, 4, 264, out, slot_ids=i32(i), num_slots=SLOTS, base=b)
    q4.combine(y, w, 6, 4, 264, b, slot_ids=i32(i), num_slots=SLOTS, base=b)
    torch.cuda.synchronize()
    assert torch.equal(out, b)


def test_nan_and_infinity_of_live_rows_come_through():
    y, w = dev(np.ones((2, 2, 16))), dev(np.ones((2, 2)))
    y[0, 1, 3] = float("nan")
    y[1, 0, 5] = float("inf")
    out = nan_like((2, 16))
    q4.combine(y, w, 2, 2, 16, out, xdtype="f32")
    torch.cuda.synchronize()
    got = host(out)
    assert np.isnan(got[0, 3]) and np.isinf(got[1, 5]) and np.isfinite(got).sum() == 30


def test_rows_past_two_to_the_31_elements():
    # 2.2e9 bf16 elements of y: offsets beyond 32 bits
    M, K, H = 66, 512, 65536
    y = torch.zeros((M, K, H), dtype=torch.bfloat16, device="cuda")
    y[M - 1] = 1.0
    w = torch.full((M, K), 1 / 512, device="cuda")
    out = nan_like((M, H), "bf16")
    q4.combine(y, w, M, K, H, out)
    d, d_w = torch.ones((M, H), dtype=torch.bfloat16, device="cuda"), nan_like((M, K))
    q4.combine_backward(d, y, w, M, K, H, d_weights=d_w)
    torch.cuda.synchronize()
    assert (out[M - 1] == 1).all() and (out[:M - 1] == 0).all()
    assert (d_w[M - 1] == H).all() and (d_w[:M - 1] == 0).all()


def test_runs_in_a_graph_and_on_another_stream():
    y, w, i, b = make(20, 8, 1032, "bf16")
    idt, out, d_y, d_w = i32(i), nan_like((20, 1032), "bf16"), nan_like((20, 8, 1032), "bf16"), nan_like((20, 8))

    def call(stream=None):
        q4.combine(y, w, 20, 8, 1032, out, slot_ids=idt, num_slots=SLOTS, base=b, stream=stream)
        q4.combine_backward(b, y, w, 20, 8, 1032, d_y=d_y, d_weights=d_w, slot_ids=idt, num_slots=SLOTS, stream=stream)

    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, d_y, d_w)]
    for got in replayed(call, [out, d_y, d_w]):
        assert all(torch.equal(a, b_) for a, b_ in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, b_) for a, b_ in zip((out, d_y, d_w), want))


def test_refusals_enqueue_nothing():
    y, w, i, b = make(2, 2, 16, "f32", ids=False)
    out = nan_like((2, 16))
    with pytest.raises(q4.Q4Error):
        q4.combine(y, w, 2, 2, 12, out, xdtype="f32")
    with pytest.raises(ValueError):
        q4.combine(y, w, 2, 3, 16, out, xdtype="f32")
    torch.cuda.synchronize()
    assert torch.isnan(out).all()
