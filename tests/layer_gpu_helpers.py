"""Shared helpers of the layer operators' GPU tests."""
import numpy as np
import torch

import quantized_moe_expert_q4_amd as q4
from quantized_moe_expert_q4_amd.device import aligned_empty

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, kind="f32"):
    """numpy array -> device tensor of the activation type."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(TYPES[kind]).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def nan_like(shape, kind="f32"):
    return torch.full(shape, float("nan"), dtype=TYPES[kind], device="cuda")


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def check(got, want, tol, label):
    """Equal where both are infinite or both NaN, else within tol (element-wise)."""
    got, want, tol = (np.asarray(a, np.float64) for a in (got, want, tol))
    assert got.shape == want.shape, label
    with np.errstate(invalid="ignore"):
        ok = (np.abs(got - want) <= tol) | (got == want) | (np.isnan(got) & np.isnan(want))
    if not ok.all():
        i = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{label}: {int((~ok).sum())} of {ok.size} off, first at {i}: {got[i]!r} for {want[i]!r}")


def replayed(enqueue, outs, work=None, times=3):
    """Capture enqueue() into a graph and return the outputs of every replay;
    outputs are overwritten and other eager work runs between the replays."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        enqueue()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        enqueue()
    got = []
    for _ in range(times):
        for o in outs:
            o.fill_(-7)
        torch.ones(1 << 16, device="cuda").mul_(2.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got.append([o.clone() for o in outs])
    return got
