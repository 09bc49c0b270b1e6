"""Refusals of the layer operators on the host (nothing is enqueued, no GPU)."""
import pytest
import torch

import quantized_moe_expert_q4_amd as q4

W, S, B, X, OUT, IDS, WS = (1 << 20, 1 << 22, 1 << 23, 1 << 24, 1 << 26, 1 << 27, 1 << 28)   # fake device addresses
INVALID, ALIGN, UNSUPPORTED, WORKSPACE = (q4.Q4_ERR_INVALID_ARGUMENT, q4.Q4_ERR_ALIGNMENT, q4.Q4_ERR_UNSUPPORTED,
                                          q4.Q4_ERR_WORKSPACE)


def _linear(xdtype="bf16", **kw):
    a = dict(weights=W, scales=S, x=X, M=1, N=4096, K=4096, group=64, out=OUT, biases=None, scale_dtype="bfloat16")
    a.update(kw)
    return q4.validate_linear(xdtype=xdtype, **a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(biases=B), dict(M=65535), dict(K=8), dict(K=65536), dict(N=1), dict(group=32),
                                dict(group=128, K=4104), dict(xdtype="f32"), dict(scale_dtype="float32")])
def test_linear_accepts(kw):
    assert _linear(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=4), INVALID),
    (dict(K=4100), INVALID), (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED), (dict(group=256), UNSUPPORTED),
    (dict(M=65536), UNSUPPORTED), (dict(K=65544), UNSUPPORTED), (dict(N=1 << 20, K=4096), UNSUPPORTED),
    (dict(N=1 << 62), UNSUPPORTED), (dict(weights=None), INVALID), (dict(scales=None), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(weights=W + 8), ALIGN), (dict(x=X + 8), ALIGN), (dict(scales=S + 1), ALIGN),
    (dict(scales=S + 2, scale_dtype="float32"), ALIGN), (dict(biases=B + 1), ALIGN), (dict(out=OUT + 1), ALIGN),
    (dict(out=OUT + 2, xdtype="f32"), ALIGN)])
def test_linear_refuses(kw, status):
    got, message = _linear(**kw)
    assert got == status and message


def _route(**kw):
    a = dict(logits=X, M=4, E=64, K=8, ids=IDS, weights=OUT)
    a.update(kw)
    return q4.validate_route(**a), q4.last_error()


def test_route_workspace():
    for M, E in ((1, 1), (1003, 167), (1 << 24, 1024)):
        n = q4.route_workspace_bytes(M, E)
        assert n >= 8 * E and n % 256 == 0
    for M, E in ((0, 8), (8, 0), (-1, 8), ((1 << 24) + 1, 8), (8, 1025)):
        assert q4.route_workspace_bytes(M, E) == 0


@pytest.mark.parametrize("kw", [{}, dict(K=64), dict(E=1, K=1), dict(E=1024), dict(M=1 << 24), dict(token_mask=W + 1),
                                dict(counts=S, workspace=WS, workspace_bytes=1 << 20), dict(score="sigmoid", select_bias=B)])
def test_route_accepts(kw):
    assert _route(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(K=65), INVALID), (dict(E=7, K=8), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(E=128, K=65), UNSUPPORTED), (dict(M=(1 << 24) + 1), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(logits=X + 1), ALIGN),
    (dict(ids=IDS + 2), ALIGN), (dict(weights=OUT + 2), ALIGN), (dict(select_bias=B + 2), ALIGN),
    (dict(counts=S), WORKSPACE), (dict(loss=S), WORKSPACE), (dict(loss_grad=S), WORKSPACE),
    (dict(counts=S, workspace=WS, workspace_bytes=16), WORKSPACE),
    (dict(counts=S + 1, workspace=WS, workspace_bytes=1 << 20), ALIGN),
    (dict(counts=S, workspace=WS + 128, workspace_bytes=1 << 20), ALIGN)])
def test_route_refuses(kw, status):
    got, message = _route(**kw)
    assert got == status and message


def _back(**kw):
    a = dict(logits=X, M=4, E=64, K=8, ids=IDS, d_logits=OUT, d_weights=S)
    a.update(kw)
    return q4.validate_route_backward(**a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(d_loss=B, loss_grad=W), dict(d_weights=None, d_loss=B, loss_grad=W)])
def test_route_backward_accepts(kw):
    assert _back(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(E=0), INVALID), (dict(K=0), INVALID), (dict(E=1025), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(d_logits=None), INVALID), (dict(d_weights=None), INVALID),
    (dict(d_loss=B), INVALID), (dict(loss_grad=B), INVALID), (dict(ids=IDS + 1), ALIGN), (dict(d_logits=OUT + 1), ALIGN),
    (dict(d_weights=S + 2), ALIGN)])
def test_route_backward_refuses(kw, status):
    got, message = _back(**kw)
    assert got == status and message


def _combine(**kw):
    a = dict(y=X, weights=S, M=4, K=8, H=4096, out=OUT)
    a.update(kw)
    return q4.validate_combine(**a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(slot_ids=IDS, num_slots=64), dict(base=OUT), dict(H=8), dict(H=65536), dict(M=1, K=1)])
def test_combine_accepts(kw):
    assert _combine(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(K=0), INVALID), (dict(H=0), INVALID), (dict(H=12), INVALID), (dict(H=65544), UNSUPPORTED),
    (dict(M=1 << 30, K=2), UNSUPPORTED), (dict(M=1 << 40), UNSUPPORTED), (dict(slot_ids=IDS), INVALID),
    (dict(y=None), INVALID), (dict(weights=None), INVALID), (dict(out=None), INVALID), (dict(y=X + 8), ALIGN),
    (dict(base=W + 8), ALIGN), (dict(out=OUT + 2), ALIGN), (dict(weights=S + 2), ALIGN),
    (dict(slot_ids=IDS + 2, num_slots=4), ALIGN)])
def test_combine_refuses(kw, status):
    got, message = _combine(**kw)
    assert got == status and message


def _combine_back(**kw):
    a = dict(d_out=W, y=X, weights=S, M=4, K=8, H=4096, d_y=OUT, d_weights=B)
    a.update(kw)
    return q4.validate_combine_backward(**a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(d_y=None), dict(d_weights=None), dict(d_weights=None, y=None)])
def test_combine_backward_accepts(kw):
    assert _combine_back(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(K=0), INVALID), (dict(H=4), INVALID), (dict(d_out=None), INVALID),
    (dict(weights=None), INVALID), (dict(y=None), INVALID), (dict(d_y=None, d_weights=None), INVALID),
    (dict(d_out=W + 8), ALIGN), (dict(d_y=OUT + 4), ALIGN), (dict(d_weights=B + 2), ALIGN),
    (dict(slot_ids=IDS, num_slots=0), INVALID)])
def test_combine_backward_refuses(kw, status):
    got, message = _combine_back(**kw)
    assert got == status and message


def test_binding_rejects_tensors_the_kernels_would_misread():
    M, N, K = 2, 16, 64
    good = dict(weights=torch.zeros(N, K // 2, dtype=torch.uint8), scales=torch.ones(N, 1, dtype=torch.bfloat16),
                x=torch.zeros(M, K, dtype=torch.bfloat16), out=torch.zeros(M, N, dtype=torch.bfloat16))

    def call(**kw):
        a = dict(good)
        a.update(kw)
        q4.linear(a["weights"], a["scales"], a["x"], M, N, K, 64, a["out"], biases=a.get("biases"))

    for kw, text in [(dict(weights=good["weights"].int()), "uint8"), (dict(x=good["x"].float()), "bfloat16"),
                     (dict(x=torch.zeros(K, M, dtype=torch.bfloat16).t()), "contiguous"),
                     (dict(out=torch.zeros(M, N - 1, dtype=torch.bfloat16)), "elements"),
                     (dict(scales=torch.ones(N, 1, dtype=torch.float16)), "scales"),
                     (dict(biases=torch.ones(N, 1)), "bfloat16"), ({}, "device")]:
        with pytest.raises(ValueError, match=text):
            call(**kw)
    logits, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in (dict(score="relu"), dict(token_mask=torch.ones(4, dtype=torch.bool)), dict(select_bias=torch.zeros(7)),
                dict(counts=torch.zeros(8, dtype=torch.int64)), {}):
        with pytest.raises(ValueError):
            q4.route(logits, 4, 8, 2, ids, w, xdtype="f32", **bad)
    with pytest.raises(ValueError):
        q4.route_backward(logits, 4, 8, 2, ids.long(), logits, d_weights=w, xdtype="f32")
    with pytest.raises(ValueError):
        q4.combine(torch.zeros(4, 2, 16), w.double(), 4, 2, 16, torch.zeros(4, 16), xdtype="f32")
    with pytest.raises(ValueError):
        q4.combine_backward(torch.zeros(4, 8), torch.zeros(4, 2, 16), w, 4, 2, 16, d_weights=w, xdtype="f32")
