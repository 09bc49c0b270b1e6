"""A mixture-of-experts layer out of the library's calls.

``MoeLayer`` keeps the weights and the buffers that a program would keep and
enqueues, for a batch of tokens, the router's linear (4-bit weights with group
scales), the choice of experts with the balance loss, the routed 4-bit experts
and the weighted sum of their outputs onto the residual; ``backward`` enqueues
the gradients of the router's logits and of the expert outputs.  Nothing
synchronises and nothing is allocated after the constructor, so a step can be
captured into a graph.

    python examples/moe_layer.py        # a small layer on the GPU
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


class MoeLayer:
    """``slots`` holds one expert in each slot (``layout``); ``gate`` the
    router's packed weights, scales and biases (or None) for groups of ``group``."""

    def __init__(self, slots, layout, slot_stride, num_experts, gate, group, H, I, top_k, max_tokens,
                 score="softmax", renormalize=True, scale=1.0, select_bias=None):
        self.slots, self.layout, self.slot_stride, self.E = slots, layout, slot_stride, num_experts
        self.gate, self.group, self.H, self.I, self.K = gate, group, H, I, top_k
        self.kw = dict(score=score, renormalize=renormalize, scale=scale)
        self.select_bias = select_bias
        new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="cuda")
        M, K, E = max_tokens, top_k, num_experts
        self.logits, self.d_logits = new(M, E), new(M, E)
        self.ids, self.weights = new(M, K, dtype=torch.int32), new(M, K, dtype=torch.float32)
        self.d_weights = new(M, K, dtype=torch.float32)
        self.mid, self.y, self.d_y = new(M, K, I), new(M, K, H), new(M, K, H)
        self.out = new(M, H)
        self.counts, self.loss = new(E, dtype=torch.int32), new(1, dtype=torch.float32)
        self.loss_grad = new(E, dtype=torch.float32)
        self.expert_bytes = q4.grouped_workspace_bytes(M, K, E)
        self.expert_ws = aligned_empty(self.expert_bytes, 256)
        self.route_bytes = q4.route_workspace_bytes(M, E)
        self.route_ws = aligned_empty(self.route_bytes, 256)
        self.tokens, self.stats = 0, False      # of the last forward

    def forward(self, x, residual=None, token_mask=None, stats=False):
        """The layer's output for the bf16 rows ``x``; with ``stats`` also ``counts``, ``loss`` and ``loss_grad``."""
        M = x.shape[0]
        self.tokens, self.stats = 0, False
        weights, scales, biases = self.gate
        q4.linear(weights, scales, x, M, self.E, self.H, self.group, self.logits, biases=biases)
        stat = dict(counts=self.counts, loss=self.loss, loss_grad=self.loss_grad, workspace=self.route_ws,
                    workspace_bytes=self.route_bytes) if stats else {}
        q4.route(self.logits, M, self.E, self.K, self.ids, self.weights, select_bias=self.select_bias,
                 token_mask=token_mask, **self.kw, **stat)
        q4.expert_forward_grouped(self.slots, self.slot_stride, self.E, self.layout, x, M, self.ids, self.K, self.H,
                                  self.I, self.mid, self.y, self.expert_ws, self.expert_bytes)
        q4.combine(self.y, self.weights, M, self.K, self.H, self.out, slot_ids=self.ids, num_slots=self.E,
                   base=residual)
        self.tokens, self.stats = M, stats
        return self.out[:M]

    def backward(self, d_out, d_loss=None):
        """Gradients of the router's logits (through the weights and, with ``d_loss``, ``d_loss``
        times the balance loss) and of the expert outputs, of the last forward; ``d_loss``
        needs its ``stats``."""
        M = d_out.shape[0]
        if M != self.tokens:
            raise ValueError(f"the last forward had {self.tokens} tokens, not {M}")
        if d_loss is not None and not self.stats:
            raise ValueError("the gradient of the balance loss needs a forward with stats")
        q4.combine_backward(d_out, self.y, self.weights, M, self.K, self.H, d_y=self.d_y, d_weights=self.d_weights,
                            slot_ids=self.ids, num_slots=self.E)
        q4.route_backward(self.logits, M, self.E, self.K, self.ids, self.d_logits, d_weights=self.d_weights,
                          d_loss=d_loss, loss_grad=None if d_loss is None else self.loss_grad, **self.kw)
        return self.d_logits[:M], self.d_y[:M]


def synthetic_layer(seed=7, H=512, I=128, experts=16, top_k=4, max_tokens=64, group=64, **kw):
    """A layer with random weights of those sizes."""
    import synth
    from quantized_moe_expert_q4_amd.device import upload_slots
    rng = np.random.default_rng(seed)
    layout = synth.expert_layout(H, I)
    host = np.zeros((experts, layout.slot_bytes), np.uint8)
    for e in range(experts):
        synth.fill_slot(rng, H, I, layout, out=host[e])
    groups = -(-H // group)
    weights = torch.from_numpy(rng.integers(0, 256, (experts, H // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.uniform(0.002, 0.01, (experts, groups)).astype(np.float32)).to(torch.bfloat16).cuda()
    return MoeLayer(upload_slots(host), layout, layout.slot_bytes, experts, (weights, scales, None), group, H, I,
                    top_k, max_tokens, **kw)


def main():
    layer = synthetic_layer()
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(48, layer.H, device="cuda", generator=gen).bfloat16()
    mask = (torch.arange(48, device="cuda") % 8 != 7).to(torch.uint8)     # padding
    out = layer.forward(x, residual=x, token_mask=mask, stats=True)
    d_logits, d_y = layer.backward(torch.ones_like(out), torch.full((1,), 0.01, device="cuda"))
    torch.cuda.synchronize()
    print("tokens per expert", layer.counts.tolist())
    print("balance loss %.4f (1 when even)" % layer.loss.item())
    print("largest gradient of a logit %.3g" % d_logits.float().abs().max().item())
    assert (out[7] == x[7]).all() and (d_logits[7] == 0).all() and (d_y[7] == 0).all(), "padding keeps its residual"


if __name__ == "__main__":
    main()
