"""The values between the adapters' two products (hidden and g), which bf16 calls take into the second product
with 16 bits, seen alone: what their leading 16 bits give is taken off again.  On an MI355X."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import check, dev, host, nan_like
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu


def bf16(v):
    return host(dev(v, "bf16"))


def values(M, largest=False):
    """M floats of 24 bits and their three bf16 parts, whose sums in any order are exact."""
    rng = np.random.default_rng(M)
    v = rng.integers(1 << 23, 1 << 24, M) * 2.0 ** rng.integers(-43, -3, M) * rng.choice([-1, 1], M)
    near = rng.integers(1 << 23, (1 << 23) + (1 << 18), M) * 2.0 ** -23   # above a power of two, where a cut counts most
    v = np.where(rng.random(M) < 0.5, near, v)
    v[0] = 1 + 2.0 ** -8 + 2.0 ** -15 - 2.0 ** -23
    if largest:                          # up to the largest float, which bf16 would round to infinity
        v[1:] = (2.0 ** 24 - rng.integers(1, 1 << 14, M - 1)) * 2.0 ** 104
    cut = (v.astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
    rest = bf16(v - cut)
    parts = np.stack([cut, rest, v - cut - rest], 1)
    assert np.array_equal(bf16(parts), parts) and np.array_equal(parts.sum(1), v)
    return v, parts


@pytest.mark.parametrize("largest", [False, True])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("M", [3, 70, 1100])
def test_middle_values_keep_16_bits(M, backward, largest):
    # hidden (or g) of rank 0 is v; rank 1 takes off its leading bf16 number and base the next one.  What is left
    # of v is at most 2^-16 of it and exact in F32, so that its error is that of the middle value, 2^-16, beside
    # which the output's rounding counts little
    v, parts = values(M, largest)
    wide, R = 8, 8                       # three columns carry the parts
    rows = np.zeros((M, wide))
    rows[:, :3] = parts
    first = np.zeros((R, wide))          # ranks from columns: rank 0 their sum, rank 1 the leading one
    first[0, :3], first[1, 0] = 1, 1
    second = np.zeros((wide, R))         # columns from ranks
    second[:, 0], second[:, 1] = 1, -1
    a, b = (second.T, first.T) if backward else (first, second)
    a, b, x = dev(a[None], "bf16"), dev(b[None], "bf16"), dev(rows, "bf16")
    base = dev(np.repeat(-parts[:, 1:2], wide, 1), "bf16")
    sizes = (M, wide, wide, R, 1)
    need = q4.adapter_workspace_bytes(*sizes)
    ws, out = aligned_empty(need, 256), nan_like((M, wide), "bf16")
    if backward:
        q4.adapter_backward(x, a, b, *sizes, ws, need, d_x=out, base=base)
    else:
        hidden = nan_like((M, R))
        q4.adapter(a, b, x, *sizes, out, ws, need, base=base, hidden=hidden)
    torch.cuda.synchronize()
    if not backward:
        assert np.array_equal(host(hidden)[:, 0], v)
    want = np.repeat(parts[:, 2:], wide, 1)
    check(host(out), want, 2.0 ** -16 * np.abs(v)[:, None] + 2.0 ** -8 * np.abs(want), "rest")
