"""The linear's gradient at its limits (row and element numbers that 32 bits or the large tile's offsets do not
hold) on an MI355X.  The gradients are sparse, so that a few rows of the weights give the result."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import TYPES, host, nan_like
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,kind,scales", [
    (130, 1 << 22, 8, "bf16", "bf16"),               # above 128 tokens, rows too long for the large tile
    (600, 1 << 22, 8, "bf16", "f32"),                # the same with more than 2^31 elements of d_out
    (520, 1 << 22, 8, "f32", "bf16"),
    (1100, (1 << 21) + 3, 8, "bf16", "bf16"),        # the large tile with more than 2^31, rows at any element
    (300, (1 << 22) - 1, 8, "bf16", "bf16"),         # the longest rows of the large tile
    (2, ((1 << 31) - 16) // 4, 8, "bf16", "f32"),    # the largest matrices, tall and wide
    (2, ((1 << 31) - 16) // 4, 8, "f32", "bf16"),
    (2, 65535, 65536, "bf16", "bf16"), (3, 65535, 65536, "f32", "f32")])
def test_limits(M, N, K, kind, scales):
    # weights are (q - 8) / 2, /1 or *2, gradients -3 .. 3, a hundred of them a token at most: exact in F32
    group, G = 128, -(-K // 128)
    gen = torch.Generator(device="cuda").manual_seed(N)
    rng = np.random.default_rng(M)
    w = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    w.random_(0, 256, generator=gen)
    s = torch.empty(N, G, dtype=TYPES[scales], device="cuda")
    s.random_(0, 3, generator=gen)
    s.sub_(1).exp2_()
    d = torch.zeros(M, N, dtype=TYPES[kind], device="cuda")
    m = np.concatenate([np.arange(M), np.arange(M), rng.integers(0, M, 40 * M if M < 200 else M)])
    n = np.concatenate([np.full(M, N - 1), N - 1 - rng.integers(1, 200, M), rng.integers(0, N, m.size - 2 * M)])
    v = rng.integers(-3, 4, m.size)
    at = torch.from_numpy(m).cuda(), torch.from_numpy(n).cuda()
    d[at] = torch.from_numpy(v).to(d)                # a place named twice holds one of its values
    v = host(d[at])
    need = q4.linear_backward_workspace_bytes(M, N, K)
    d_x = nan_like((M, K), kind)
    q4.linear_backward(w, s, d, M, N, K, group, d_x, aligned_empty(need, 256), need, xdtype=kind)
    torch.cuda.synchronize()
    rows, first = np.unique(n, return_inverse=True)
    picked = torch.from_numpy(rows).cuda()
    W = (ref.unpack_q4(host(w[picked]), rows.size, K) - 8.0) * np.repeat(host(s[picked]), group, axis=1)[:, :K]
    want = np.zeros((M, K))
    for (i, j), value in {(a, b): c for a, b, c in zip(m, first, v)}.items():
        want[i] += value * W[j]
    assert torch.equal(d_x.cpu(), torch.from_numpy(want).to(TYPES[kind]))
