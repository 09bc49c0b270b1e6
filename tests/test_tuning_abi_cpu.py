"""Refusals of the router over groups, the adapters and the linear's gradient on the host (nothing is enqueued, no GPU)."""
import pytest

import quantized_moe_expert_q4_amd as q4

W, S, B, X, OUT, IDS, WS = (1 << 20, 1 << 22, 1 << 23, 1 << 24, 1 << 26, 1 << 27, 1 << 28)   # fake device addresses
INVALID, ALIGN, UNSUPPORTED, WORKSPACE = (q4.Q4_ERR_INVALID_ARGUMENT, q4.Q4_ERR_ALIGNMENT, q4.Q4_ERR_UNSUPPORTED,
                                          q4.Q4_ERR_WORKSPACE)


def _groups(**kw):
    a = dict(logits=X, M=4, E=64, K=8, groups=8, top_groups=4, ids=IDS, weights=OUT)
    a.update(kw)
    return q4.validate_route_groups(**a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(groups=64, top_groups=8), dict(groups=1, top_groups=1), dict(top_groups=8, K=64),
                                dict(top_groups=1), dict(group_top=1), dict(E=1, K=1, groups=1, top_groups=1),
                                dict(E=1024, groups=64), dict(xdtype="f32"), dict(score="sigmoid", select_bias=B),
                                dict(counts=S, workspace=WS, workspace_bytes=1 << 20)])
def test_route_groups_accepts(kw):
    assert _groups(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), INVALID), (dict(groups=-8), INVALID), (dict(groups=7), INVALID), (dict(groups=128), INVALID),
    (dict(E=128, groups=128), UNSUPPORTED), (dict(top_groups=0), INVALID), (dict(top_groups=9), INVALID),
    (dict(top_groups=-1), INVALID), (dict(group_top=0), INVALID), (dict(group_top=3), INVALID),
    (dict(top_groups=1, K=9), INVALID), (dict(groups=64, top_groups=7), INVALID), (dict(M=0), INVALID), (dict(E=0), INVALID),
    (dict(K=0), INVALID), (dict(E=1032), UNSUPPORTED), (dict(logits=None), INVALID), (dict(logits=X + 1), ALIGN),
    (dict(logits=X + 2, xdtype="f32"), ALIGN), (dict(counts=S), WORKSPACE),
    (dict(counts=S, workspace=WS, workspace_bytes=16), WORKSPACE)])
def test_route_groups_refuses(kw, status):
    got, message = _groups(**kw)
    assert got == status and message


def _back(xdtype="bf16", **kw):
    a = dict(weights=W, scales=S, d_out=X, M=1, N=4096, K=4096, group=64, d_x=OUT, workspace=WS, workspace_bytes=1 << 28,
             biases=None, scale_dtype="bfloat16")
    a.update(kw)
    return q4.validate_linear_backward(xdtype=xdtype, **a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(biases=B), dict(M=65535), dict(K=8), dict(K=65536), dict(N=1), dict(group=32),
                                dict(group=128, K=4104), dict(xdtype="f32"), dict(scale_dtype="float32"),
                                dict(d_out=X + 2), dict(d_out=X + 4, xdtype="f32")])
def test_linear_backward_accepts(kw):
    assert _back(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=4100), INVALID), (dict(group=16), UNSUPPORTED),
    (dict(M=65536), UNSUPPORTED), (dict(K=65544), UNSUPPORTED), (dict(N=1 << 20, K=4096), UNSUPPORTED),
    (dict(N=1 << 62), UNSUPPORTED), (dict(weights=None), INVALID), (dict(scales=None), INVALID), (dict(d_out=None), INVALID),
    (dict(d_x=None), INVALID), (dict(weights=W + 8), ALIGN), (dict(d_x=OUT + 8), ALIGN), (dict(d_out=X + 1), ALIGN),
    (dict(d_out=X + 2, xdtype="f32"), ALIGN), (dict(scales=S + 1), ALIGN), (dict(biases=B + 1), ALIGN),
    (dict(workspace=None), WORKSPACE), (dict(workspace=WS + 128), ALIGN), (dict(workspace_bytes=0), WORKSPACE)])
def test_linear_backward_refuses(kw, status):
    got, message = _back(**kw)
    assert got == status and message


def test_linear_backward_workspace():
    assert q4.linear_backward_workspace_bytes(1, 1, 8) % 256 == 0
    for M, N, K in ((0, 8, 8), (1, 0, 8), (1, 8, 0), (1, 8, 12), (65536, 8, 8), (1, 1 << 40, 4096), (1, 8, 65544)):
        assert q4.linear_backward_workspace_bytes(M, N, K) == 0


def _adapter(xdtype="bf16", **kw):
    a = dict(a=W, b=B, x=X, M=4, N=4096, K=4096, R=16, num_adapters=3, out=OUT, workspace=WS, workspace_bytes=1 << 26)
    a.update(kw)
    return q4.validate_adapter(xdtype=xdtype, **a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(M=65535, workspace_bytes=1 << 32), dict(N=1), dict(N=1 << 20), dict(K=8), dict(K=65536),
                                dict(R=8), dict(R=256), dict(num_adapters=65535), dict(adapter_ids=IDS, scales=S, hidden=S),
                                dict(base=OUT), dict(base=S + 2, out=OUT + 2), dict(xdtype="f32", base=S + 4, out=OUT + 4)])
def test_adapter_accepts(kw):
    assert _adapter(**kw) == (0, "")


SIZE_FAULTS = [(dict(M=0), INVALID), (dict(M=-3), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=12), INVALID),
               (dict(R=0), INVALID), (dict(R=4), INVALID), (dict(R=-8), INVALID), (dict(num_adapters=0), INVALID),
               (dict(M=65536), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=65544), UNSUPPORTED),
               (dict(R=264), UNSUPPORTED), (dict(num_adapters=65536), UNSUPPORTED), (dict(workspace=None), WORKSPACE),
               (dict(workspace=WS + 16), ALIGN), (dict(workspace_bytes=0), WORKSPACE), (dict(a=None), INVALID),
               (dict(b=None), INVALID), (dict(a=W + 8), ALIGN), (dict(b=B + 8), ALIGN), (dict(x=X + 8), ALIGN),
               (dict(adapter_ids=IDS + 2), ALIGN), (dict(scales=S + 2), ALIGN), (dict(hidden=S + 8), ALIGN)]


@pytest.mark.parametrize("kw,status", SIZE_FAULTS + [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(out=OUT + 1), ALIGN), (dict(base=S + 1), ALIGN),
    (dict(out=OUT + 2, xdtype="f32"), ALIGN), (dict(base=S + 2, xdtype="f32"), ALIGN)])
def test_adapter_refuses(kw, status):
    got, message = _adapter(**kw)
    assert got == status and message


def _adapter_back(xdtype="bf16", **kw):
    a = dict(d_out=X, a=W, b=B, M=4, N=4096, K=4096, R=16, num_adapters=3, workspace=WS, workspace_bytes=1 << 26, x=X,
             hidden=S, d_x=OUT, d_a=OUT, d_b=OUT)
    a.update(kw)
    return q4.validate_adapter_backward(xdtype=xdtype, **a), q4.last_error()


@pytest.mark.parametrize("kw", [{}, dict(d_x=None), dict(d_a=None, x=None), dict(d_b=None, hidden=None), dict(base=OUT),
                                dict(d_out=X + 2), dict(d_x=None, d_a=None, x=None), dict(xdtype="f32", d_out=X + 4)])
def test_adapter_backward_accepts(kw):
    assert _adapter_back(**kw) == (0, "")


@pytest.mark.parametrize("kw,status", SIZE_FAULTS + [
    (dict(d_out=None), INVALID), (dict(d_x=None, d_a=None, d_b=None), INVALID), (dict(x=None), INVALID),
    (dict(hidden=None), INVALID), (dict(d_x=None, base=OUT), INVALID), (dict(d_out=X + 1), ALIGN), (dict(d_x=OUT + 8), ALIGN),
    (dict(d_a=OUT + 8), ALIGN), (dict(d_b=OUT + 8), ALIGN), (dict(base=OUT + 8), ALIGN),
    (dict(d_out=X + 2, xdtype="f32"), ALIGN)])
def test_adapter_backward_refuses(kw, status):
    got, message = _adapter_back(**kw)
    assert got == status and message


def test_adapter_workspace():
    assert q4.adapter_workspace_bytes(1, 1, 8, 8, 1) % 256 == 0
    for sizes in ((0, 1, 8, 8, 1), (1, 0, 8, 8, 1), (1, 1, 4, 8, 1), (1, 1, 8, 12, 1), (1, 1, 8, 8, 0), (65536, 1, 8, 8, 1)):
        assert q4.adapter_workspace_bytes(*sizes) == 0
