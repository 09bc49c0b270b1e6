"""Adapters on tensors of more than 2^31 elements, rows at both ends checked, on an MI355X."""
import numpy as np
import pytest
import torch

import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import TYPES
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu


def small(shape, gen, kind):
    """-1, 0 and 1."""
    t = torch.empty(shape, dtype=torch.int8, device="cuda")
    return t.random_(-1, 2, generator=gen).to(TYPES[kind])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(2100, (1 << 20) - 1, 8), (40000, 24, 65536)])
def test_more_than_2_to_the_31_elements(M, N, K, kind):
    # the output's side is that large, or the input's; whole numbers: sums are exact (|hidden| <= K and |g| <= 24
    # by the few non-zero gradients), checked at rows of both ends and of the middle
    R, n = 8, 2
    gen = torch.Generator(device="cuda").manual_seed(M)
    a, b, x = small((n, R, K), gen, kind), small((n, N, R), gen, kind), small((M, K), gen, kind)
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    if K > 8:                            # few terms, so that bf16 holds the result
        a[:, :, 16:-16] = 0
    ids = (torch.arange(M, device="cuda") % (n + 1) - 1).to(torch.int32)
    sizes = (M, N, K, R, n)
    need = q4.adapter_workspace_bytes(*sizes)
    ws, hidden = aligned_empty(need, 256), torch.empty(M, R, device="cuda")
    out = torch.empty(M, N, dtype=TYPES[kind], device="cuda")
    q4.adapter(a, b, x, *sizes, out, ws, need, adapter_ids=ids, hidden=hidden, xdtype=kind)
    torch.cuda.synchronize()
    for t in rows.tolist():
        i = int(ids[t])
        h = a[i].double() @ x[t].double() if i >= 0 else torch.zeros(R, dtype=torch.float64, device="cuda")
        assert torch.equal(hidden[t].double(), h), t
        want = b[max(i, 0)].double() @ h
        assert torch.equal(out[t], want.to(TYPES[kind])), t
    # gradients at a few columns of those rows, the last one among them
    d = out.zero_()
    columns = torch.tensor([0, N // 2, N - 1], device="cuda")
    for t in rows.tolist():
        d[t, columns] = 1.0
    d_x = torch.empty(M, K, dtype=TYPES[kind], device="cuda")
    d_a, d_b = torch.empty(n, R, K, device="cuda"), torch.empty(n, N, R, device="cuda")
    q4.adapter_backward(d, a, b, *sizes, ws, need, x=x, hidden=hidden, d_x=d_x, d_a=d_a, d_b=d_b, adapter_ids=ids,
                        xdtype=kind)
    torch.cuda.synchronize()
    want_a, want_b = torch.zeros(n, R, K, dtype=torch.float64, device="cuda"), torch.zeros(n, N, R, dtype=torch.float64, device="cuda")
    for t in rows.tolist():
        i = int(ids[t])
        if i < 0:
            assert not d_x[t].any()
            continue
        g = b[i, columns].double().sum(0)
        assert torch.equal(d_x[t], (g @ a[i].double()).to(TYPES[kind])), t
        want_a[i] += g[:, None] * x[t].double()
        want_b[i, columns] += hidden[t].double()
    assert torch.equal(d_a.double(), want_a) and torch.equal(d_b.double(), want_b)
    others = torch.ones(M, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert not d_x[others].any()
