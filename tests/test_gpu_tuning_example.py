"""The tuned router of examples/adapter_tuning.py (linear, adapters, router over groups, and their
gradients in one run), step by step against the 64-bit forms, on an MI355X."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_reference as ref
import tuning_reference as tune
from layer_gpu_helpers import check, host, replayed

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import adapter_tuning  # noqa: E402

pytestmark = pytest.mark.gpu


def inputs(router, M, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, router.gate.K, device="cuda", generator=gen).bfloat16()
    ids = torch.randint(-1, router.gate.n, (M,), device="cuda", generator=gen).to(torch.int32)
    mask = torch.ones(M, dtype=torch.uint8, device="cuda")
    mask[5::7] = 0
    d_weights = torch.randn(M, router.top_k, device="cuda", generator=gen)
    return x, ids, mask, d_weights, torch.full((1,), 0.5, device="cuda")


def step(router, x, ids, mask, d_weights, d_loss):
    router.forward(x, ids, token_mask=mask)
    router.backward(d_weights, d_loss)


@pytest.mark.parametrize("M,kw", [(1, {}), (48, dict(score="softmax", scale=2.5)), (300, dict(rank=24, adapters=5)),
                                  (1100, dict(experts=160, groups=10, K=264))])
def test_router(M, kw):
    router = adapter_tuning.synthetic_router(max_tokens=M, **kw)
    gate = router.gate
    x, ids, mask, d_weights, d_loss = inputs(router, M, M)
    step(router, x, ids, mask, d_weights, d_loss)
    torch.cuda.synchronize()
    N, K, R, n = gate.N, gate.K, gate.R, gate.n
    hx, hi, s = host(x), host(ids), host(gate.adapter_scales)
    a, b = host(gate.a), host(gate.b)
    # the linear's output is rounded to bf16 once, the adapters' onto it once more
    base, mag = ref.linear(host(gate.weights), host(gate.scales), None, gate.group, hx, N, K)
    base_tol = 2.0 ** -8 * np.abs(base) + (2 * gate.group + K // gate.group + 33) * 2.0 ** -23 * mag
    want, amag, hidden, hmag = tune.adapter(a, b, hx, hi, s, base)
    tol = base_tol + 2.0 ** -8 * (np.abs(want) + base_tol) + ((K + R + 64) * 2.0 ** -23 + 2.0 ** -16) * amag
    check(host(gate.out), want, tol, "logits")
    check(host(gate.hidden), hidden, (K + 64) * 2.0 ** -23 * hmag, "hidden")
    logits = host(gate.out)
    score, scale = router.kw["score"], router.kw["scale"]
    eids, w, counts, loss, grad = tune.route_groups(logits, router.top_k, router.groups, router.top_groups, 2, score, True,
                                                    scale, mask=host(mask))
    assert np.array_equal(host(router.ids), eids) and np.array_equal(host(router.counts), counts)
    # as the router's own tests: exp's argument at the spread of the logits, then sums over lanes
    rel = (64 + 4 * np.abs(logits).max()) * 2.0 ** -24
    check(host(router.weights), w, rel * w, "weights")
    check(host(router.loss), [loss], (rel + 128 * 2.0 ** -24) * loss, "loss")
    want, mag = ref.route_backward(logits, eids, score, True, scale, host(d_weights), 0.5, host(router.loss_grad))
    rel = (128 + 8 * np.abs(logits).max()) * 2.0 ** -24
    check(host(router.d_logits), want, 2.0 ** -8 * np.abs(want) + rel * mag + 2.0 ** -120, "d_logits")
    d = host(router.d_logits)
    base, mag = tune.linear_backward(host(gate.weights), host(gate.scales), None, gate.group, d, N, K)
    base_tol = 2.0 ** -8 * np.abs(base) + (2.0 ** -8 + (N + 16) * 2.0 ** -23) * mag
    (d_x, d_a, d_b), (mx, ma, mb) = tune.adapter_backward(d, a, b, hx, host(gate.hidden), hi, s, base)
    tol = base_tol + 2.0 ** -8 * (np.abs(d_x) + base_tol) + ((N + R + 64) * 2.0 ** -23 + 2.0 ** -16) * mx
    check(host(gate.d_x), d_x, tol, "d_x")
    check(host(gate.d_a), d_a, (M + N + 64) * 2.0 ** -23 * ma, "d_a")
    check(host(gate.d_b), d_b, (M + 64) * 2.0 ** -23 * mb, "d_b")


@pytest.mark.parametrize("M", [30, 600])
def test_router_in_a_graph(M):
    router = adapter_tuning.synthetic_router(max_tokens=M)
    gate, args = router.gate, inputs(router, M, 3)
    step(router, *args)
    torch.cuda.synchronize()
    outs = [router.ids, router.weights, router.counts, router.loss, router.d_logits, gate.out, gate.hidden, gate.d_x, gate.d_a,
            gate.d_b]
    want = [o.clone() for o in outs]
    for got in replayed(lambda: step(router, *args), outs):
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_two_layers_on_two_streams():
    # calls with workspaces of their own may overlap
    routers = [adapter_tuning.synthetic_router(seed=s, max_tokens=300) for s in (1, 2)]
    args = [inputs(r, 300, s) for r, s in zip(routers, (4, 5))]
    for r, a in zip(routers, args):
        step(r, *a)
    torch.cuda.synchronize()
    want = [[o.clone() for o in (r.weights, r.gate.d_x, r.gate.d_a, r.gate.d_b)] for r in routers]
    streams = [torch.cuda.Stream() for _ in routers]
    for _ in range(3):
        for r, a, s in zip(routers, args, streams):
            with torch.cuda.stream(s):
                step(r, *a)
    torch.cuda.synchronize()
    for r, w in zip(routers, want):
        assert all(torch.equal(o, v) for o, v in zip((r.weights, r.gate.d_x, r.gate.d_a, r.gate.d_b), w))


def test_backward_belongs_to_the_last_forward():
    router = adapter_tuning.synthetic_router(max_tokens=8)
    x, ids, mask, d_weights, d_loss = inputs(router, 8, 1)
    router.forward(x, ids)
    with pytest.raises(ValueError):
        router.gate.backward(router.d_logits[:7])


def test_the_example_runs(capsys):
    adapter_tuning.main()
    assert capsys.readouterr().out.count("balance loss") == 5
