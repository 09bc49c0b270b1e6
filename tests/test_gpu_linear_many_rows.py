"""The linear at the most rows its matrix limit allows (more work-groups than one launch takes)."""
import pytest
import torch

import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import TYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,kind", [(1, "bf16"), (5, "bf16"), (9, "f32"), (33, "bf16")])
def test_most_rows_of_eight_weights(M, kind):
    N, K = ((1 << 31) - 16) // 4, 8
    gen = torch.Generator(device="cuda").manual_seed(M)
    w = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((N, 1), dtype=torch.bfloat16, device="cuda")
    step = 1 << 24
    for at in range(0, N, step):
        part = w[at:at + step]
        part.copy_(torch.randint(0, 256, part.shape, device="cuda", generator=gen, dtype=torch.uint8))
        s[at:at + step] = torch.randint(1, 4, (part.shape[0], 1), device="cuda", generator=gen).bfloat16()
    x = torch.randint(-3, 4, (M, K), device="cuda", generator=gen).to(TYPES[kind])
    out = torch.full((M, N), 7.0e9, dtype=TYPES[kind], device="cuda")
    q4.linear(w, s, x, M, N, K, 64, out, xdtype=kind)
    torch.cuda.synchronize()
    for at in range(0, N, step):
        part = w[at:at + step]
        q = torch.stack((part & 15, part >> 4), 2).view(-1, K).float() - 8
        # whole numbers of at most 8 * 3 * 8 * 3: exact in F32
        want = sum(x[:, k, None].float() * (q[:, k] * s[at:at + step, 0].float()) for k in range(K))
        assert torch.equal(out[:, at:at + step], want.to(TYPES[kind])), at
