"""Tuning the router of a mixture-of-experts layer with low-rank adapters.

``AdapterLinear`` is a frozen 4-bit projection with adapters beside it: a batch
holds rows of several adapters (many requests served at once, or several
variants tuned side by side).  ``TunedRouter`` feeds its output to the router over
groups of experts and takes the gradients of the routing weights and of the
balance loss back to the adapters and to the hidden states.  Nothing
synchronises and nothing is allocated after the constructors, so a step can be
captured into a graph.

    python examples/adapter_tuning.py        # a few steps of a small router on the GPU
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_moe_expert_q4_amd as q4  # noqa: E402
from quantized_moe_expert_q4_amd.device import aligned_empty  # noqa: E402


def _new(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


class AdapterLinear:
    """``weights``, ``scales`` and ``biases`` (or None) as of q4.linear, ``a``
    [n, R, K], ``b`` [n, N, R] and ``adapter_scales`` [n] as of q4.adapter, in bf16."""

    def __init__(self, weights, scales, biases, group, a, b, adapter_scales, max_tokens):
        self.weights, self.scales, self.biases, self.group = weights, scales, biases, group
        self.a, self.b, self.adapter_scales = a, b, adapter_scales
        self.n, self.R, self.K = a.shape
        self.N = b.shape[1]
        M = max_tokens
        self.out, self.d_x = _new(M, self.N), _new(M, self.K)
        self.hidden = _new(M, self.R, dtype=torch.float32)
        self.d_a, self.d_b = (torch.empty_like(t, dtype=torch.float32) for t in (a, b))
        self.adapter_bytes = q4.adapter_workspace_bytes(M, self.N, self.K, self.R, self.n)
        self.linear_bytes = q4.linear_backward_workspace_bytes(M, self.N, self.K)
        self.adapter_ws, self.linear_ws = aligned_empty(self.adapter_bytes, 256), aligned_empty(self.linear_bytes, 256)
        self.x = self.ids = None                # of the last forward

    def forward(self, x, ids):
        """The projection of the bf16 rows ``x`` plus each row's adapter (int32 ``ids``, -1 for none)."""
        M = x.shape[0]
        q4.linear(self.weights, self.scales, x, M, self.N, self.K, self.group, self.out, biases=self.biases)
        q4.adapter(self.a, self.b, x, M, self.N, self.K, self.R, self.n, self.out, self.adapter_ws, self.adapter_bytes,
                   adapter_ids=ids, scales=self.adapter_scales, base=self.out, hidden=self.hidden)
        self.x, self.ids = x, ids
        return self.out[:M]

    def backward(self, d_out):
        """The gradient of the last forward's ``x``; those of the adapters are in ``d_a`` and ``d_b``."""
        M = d_out.shape[0]
        if self.x is None or M != self.x.shape[0]:
            raise ValueError("the gradient belongs to the last forward's rows")
        q4.linear_backward(self.weights, self.scales, d_out, M, self.N, self.K, self.group, self.d_x, self.linear_ws,
                           self.linear_bytes, biases=self.biases)
        q4.adapter_backward(d_out, self.a, self.b, M, self.N, self.K, self.R, self.n, self.adapter_ws, self.adapter_bytes,
                            x=self.x, hidden=self.hidden, d_x=self.d_x, d_a=self.d_a, d_b=self.d_b,
                            adapter_ids=self.ids, scales=self.adapter_scales, base=self.d_x)
        return self.d_x[:M]


class TunedRouter:
    """The router over groups of experts behind ``gate``, an AdapterLinear from hidden states to logits."""

    def __init__(self, gate, groups, top_groups, top_k, max_tokens, select_bias=None, score="sigmoid", scale=1.0):
        self.gate, self.groups, self.top_groups, self.top_k = gate, groups, top_groups, top_k
        self.select_bias = select_bias
        self.kw = dict(score=score, renormalize=True, scale=scale)
        M, E = max_tokens, gate.N
        self.ids, self.weights = _new(M, top_k, dtype=torch.int32), _new(M, top_k, dtype=torch.float32)
        self.counts, self.loss = _new(E, dtype=torch.int32), _new(1, dtype=torch.float32)
        self.loss_grad, self.d_logits = _new(E, dtype=torch.float32), _new(M, E)
        self.ws_bytes = q4.route_workspace_bytes(M, E)
        self.ws = aligned_empty(self.ws_bytes, 256)

    def forward(self, x, adapter_ids, token_mask=None):
        """(ids, weights) of the rows' experts; ``counts``, ``loss`` and ``loss_grad`` are kept."""
        logits = self.gate.forward(x, adapter_ids)
        M = x.shape[0]
        q4.route_groups(logits, M, self.gate.N, self.top_k, self.groups, self.top_groups, self.ids, self.weights,
                        select_bias=self.select_bias, token_mask=token_mask, counts=self.counts, loss=self.loss,
                        loss_grad=self.loss_grad, workspace=self.ws, workspace_bytes=self.ws_bytes, **self.kw)
        return self.ids[:M], self.weights[:M]

    def backward(self, d_weights, d_loss):
        """The gradient of ``x`` from those of the weights and of the balance loss (F32, on the device)."""
        M = d_weights.shape[0]
        q4.route_backward(self.gate.out, M, self.gate.N, self.top_k, self.ids, self.d_logits, d_weights=d_weights,
                          d_loss=d_loss, loss_grad=self.loss_grad, **self.kw)
        return self.gate.backward(self.d_logits[:M])


def synthetic_router(seed=7, K=512, experts=64, rank=16, adapters=3, groups=8, top_groups=3, top_k=6, max_tokens=64,
                     group=64, **kw):
    """A router with random weights of those sizes."""
    rng = np.random.default_rng(seed)
    bf16 = lambda v: torch.from_numpy(np.asarray(v, np.float32)).bfloat16().cuda()
    weights = torch.from_numpy(rng.integers(0, 256, (experts, K // 2), dtype=np.uint8)).cuda()
    scales = bf16(rng.uniform(0.002, 0.01, (experts, -(-K // group))))
    a, b = bf16(rng.normal(size=(adapters, rank, K)) * K ** -0.5), bf16(rng.normal(size=(adapters, experts, rank)) * 0.05)
    gate = AdapterLinear(weights, scales, None, group, a, b, torch.full((adapters,), 2.0, device="cuda"), max_tokens)
    return TunedRouter(gate, groups, top_groups, top_k, max_tokens, **kw)


def main():
    M = 48
    router = synthetic_router(max_tokens=M)
    gate = router.gate
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, gate.K, device="cuda", generator=gen).bfloat16()
    ids = (torch.arange(M, device="cuda") % 4 - 1).to(torch.int32)        # a quarter of the rows without an adapter
    d_weights, d_loss = torch.zeros(M, router.top_k, device="cuda"), torch.ones(1, device="cuda")
    master = [t.float() for t in (gate.a, gate.b)]
    for step in range(5):                                                 # gradient descent on the balance loss
        router.forward(x, ids)
        router.backward(d_weights, d_loss)
        for m, t, d in zip(master, (gate.a, gate.b), (gate.d_a, gate.d_b)):
            m -= 20.0 * d
            t.copy_(m)
        print("step %d: balance loss %.4f, largest gradient of an adapter %.3g" % (
            step, router.loss.item(), max(gate.d_a.abs().max().item(), gate.d_b.abs().max().item())))


if __name__ == "__main__":
    main()
