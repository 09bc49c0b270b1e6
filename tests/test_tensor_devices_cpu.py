"""Tensors of another device than the current one are refused before anything is enqueued (stand-ins for device
tensors, no GPU)."""
import types

import pytest
import torch

import quantized_moe_expert_q4_amd as q4
from quantized_moe_expert_q4_amd import _lib


class Tensor:
    """What the checks ask of a tensor, at an address that nothing may read."""

    def __init__(self, dtype, numel, index):
        self.dtype, self.size, self.index = dtype, numel, index
        self.device = types.SimpleNamespace(type="cuda", index=index)
        self.is_cuda = True

    def numel(self):
        return self.size

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("the call was not refused")


M, N, K, R = 2, 16, 64, 8
BF, F, U = torch.bfloat16, torch.float32, torch.uint8


def tensors(index, **other):
    sizes = dict(a=(BF, R * K), b=(BF, N * R), x=(BF, M * K), out=(BF, M * N), workspace=(U, 4096), logits=(BF, M * N),
                 ids=(torch.int32, M), weights=(F, M), scales=(BF, N), w=(U, N * K // 2))
    return {k: Tensor(*v, other.get(k, index)) for k, v in sizes.items()}


def calls(t):
    return [lambda: q4.adapter(t["a"], t["b"], t["x"], M, N, K, R, 1, t["out"], t["workspace"], 4096),
            lambda: q4.adapter_backward(t["out"], t["a"], t["b"], M, N, K, R, 1, t["workspace"], 4096, d_x=t["x"]),
            lambda: q4.linear_backward(t["w"], t["scales"], t["out"], M, N, K, 64, t["x"], t["workspace"], 4096),
            lambda: q4.linear(t["w"], t["scales"], t["x"], M, N, K, 64, t["out"]),
            lambda: q4.route_groups(t["logits"], M, N, 1, 4, 2, t["ids"], t["weights"]),
            lambda: q4.route(t["logits"], M, N, 1, t["ids"], t["weights"])]


@pytest.mark.parametrize("call", range(6))
def test_all_on_another_device(monkeypatch, call):
    monkeypatch.setattr(_lib, "_raw_device", lambda: 0)
    with pytest.raises(ValueError, match="is on cuda:1, but the current device is cuda:0"):
        calls(tensors(1))[call]()


@pytest.mark.parametrize("call,name", [(0, "a"), (0, "workspace"), (1, "x"), (2, "scales"), (3, "out"), (4, "weights"), (5, "ids")])
def test_one_on_another_device(monkeypatch, call, name):
    monkeypatch.setattr(_lib, "_raw_device", lambda: 1)
    with pytest.raises(ValueError, match="is on cuda:0, but the current device is cuda:1"):
        calls(tensors(1, **{name: 0}))[call]()


def test_those_of_the_current_device_pass(monkeypatch):
    monkeypatch.setattr(_lib, "_raw_device", lambda: 1)
    _lib._args(*((n, t, str(t.dtype).replace("torch.", ""), t.size) for n, t in tensors(1).items()))
    _lib._args(("a", 4096, "uint8", 1), ("b", None, "uint8", 1))
