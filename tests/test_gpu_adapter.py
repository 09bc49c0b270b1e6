"""Low-rank adapters and their gradients against their 64-bit forms on an MI355X."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
import tuning_reference as tune
from layer_gpu_helpers import TYPES, check, dev, host, i32, nan_like, replayed
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu

NO_ADAPTER = (-1, -2 ** 31, 2 ** 31 - 1)      # and num_adapters


class Case:
    """Inputs on the device, and the same values in 64 bits.  With `exact`, small
    whole numbers and powers of two: every sum is exact in F32, hidden values in 16 bits."""

    def __init__(self, seed, M, N, K, R, n, kind, ids="mixed", exact=False, scales=True, base=True):
        rng = np.random.default_rng(seed)
        self.sizes, self.kind = (M, N, K, R, n), kind
        if exact:
            sparse = lambda shape, p: rng.integers(-1, 2, size=shape) * (rng.random(shape) < p)
            a, b, x, d = sparse((n, R, K), 0.4), sparse((n, N, R), 0.4), sparse((M, K), 0.4), sparse((M, N), 0.4)
            s = 2.0 ** rng.integers(-1, 2, size=n)
            o, c, h = rng.integers(-9, 10, size=(M, N)), rng.integers(-9, 10, size=(M, K)), rng.integers(-20, 21, size=(M, R))
        else:
            a, b = rng.normal(size=(n, R, K)) * K ** -0.5, rng.normal(size=(n, N, R)) * 0.1
            x, d = rng.normal(size=(M, K)), rng.normal(size=(M, N)) * 0.1
            s = rng.uniform(-2, 2, size=n)
            o, c, h = rng.normal(size=(M, N)), rng.normal(size=(M, K)), rng.normal(size=(M, R))
        for name, v in (("a", a), ("b", b), ("x", x), ("d_out", d), ("o_base", o), ("x_base", c)):
            setattr(self, name, dev(v, kind))
        self.h = dev(h)
        self.scales = dev(s) if scales else None
        if not base:
            self.o_base = self.x_base = None
        self.ids = None
        if ids is not None:
            i = rng.integers(0, n, M)
            none = np.array(NO_ADAPTER + (n,))[rng.integers(0, 4, M)]
            i = np.where(rng.random(M) < 0.15, none, i)
            self.ids = i32(np.sort(i) if ids == "sorted" else i)
        self.need = q4.adapter_workspace_bytes(*self.sizes)
        self.ws = aligned_empty(self.need, 256)
        self.ws.fill_(0xFF)               # NaNs

    def host_ids(self):
        return np.zeros(self.sizes[0], int) if self.ids is None else host(self.ids)

    def host_scales(self):
        return np.ones(self.sizes[4]) if self.scales is None else host(self.scales)

    def forward(self, out, hidden=None, base="own", stream=None):
        q4.adapter(self.a, self.b, self.x, *self.sizes, out, self.ws, self.need, adapter_ids=self.ids, scales=self.scales,
                   base=self.o_base if isinstance(base, str) else base, hidden=hidden, xdtype=self.kind, stream=stream)

    def backward(self, d_x=None, d_a=None, d_b=None, base="own", stream=None):
        base = self.x_base if isinstance(base, str) else base
        q4.adapter_backward(self.d_out, self.a, self.b, *self.sizes, self.ws, self.need, x=self.x, hidden=self.h, d_x=d_x,
                            d_a=d_a, d_b=d_b, adapter_ids=self.ids, scales=self.scales, base=base if d_x is not None else None,
                            xdtype=self.kind, stream=stream)

    def outputs(self):
        M, N, K, R, n = self.sizes
        return nan_like((M, N), self.kind), nan_like((M, R))

    def gradients(self):
        M, N, K, R, n = self.sizes
        return nan_like((M, K), self.kind), nan_like((n, R, K)), nan_like((n, N, R))

    def want_forward(self):
        M, N, K, R, n = self.sizes
        base = np.zeros((M, N)) if self.o_base is None else host(self.o_base)
        return tune.adapter(host(self.a), host(self.b), host(self.x), self.host_ids(), self.host_scales(), base)

    def want_backward(self):
        M, N, K, R, n = self.sizes
        base = np.zeros((M, K)) if self.x_base is None else host(self.x_base)
        return tune.adapter_backward(host(self.d_out), host(self.a), host(self.b), host(self.x), host(self.h),
                                     self.host_ids(), self.host_scales(), base)

    # Rounding of the output; a step (2^-23: the matrix unit may truncate) of the
    # magnitude for each addition a term can pass, 64 to join parts; and for bf16
    # rows the values between the two products with 16 bits.
    def row_tolerance(self, want, mag, adds):
        return ref.HALF_STEP[self.kind] * np.abs(want) + ((adds + 64) * 2.0 ** -23 + (2.0 ** -16 if self.kind == "bf16" else 0)) * mag

    def check_forward(self):
        M, N, K, R, n = self.sizes
        out, hidden = self.outputs()
        self.forward(out, hidden)
        torch.cuda.synchronize()
        want, mag, h, hm = self.want_forward()
        check(host(hidden), h, (K + 64) * 2.0 ** -23 * hm, "hidden")
        check(host(out), want, self.row_tolerance(want, mag, K + R), "out")

    def check_backward(self):
        M, N, K, R, n = self.sizes
        grads = self.gradients()
        self.backward(*grads)
        torch.cuda.synchronize()
        (d_x, d_a, d_b), (mx, ma, mb) = self.want_backward()
        check(host(grads[0]), d_x, self.row_tolerance(d_x, mx, N + R), "d_x")
        check(host(grads[1]), d_a, (M + N + 64) * 2.0 ** -23 * ma, "d_a")
        check(host(grads[2]), d_b, (M + 64) * 2.0 ** -23 * mb, "d_b")


SHAPES = [  # M, N, K, R, adapters: one row and column; odd columns; ends inside tiles; more adapters than rows
    (1, 1, 8, 8, 1), (1, 40, 64, 16, 3), (2, 17, 72, 24, 2), (5, 100, 136, 32, 70), (16, 64, 256, 16, 1), (17, 256, 96, 8, 2),
    (33, 257, 264, 40, 4), (64, 300, 520, 64, 5), (100, 65, 1000, 128, 3), (257, 129, 392, 8, 300), (300, 31, 72, 256, 2),
    (600, 515, 136, 16, 7), (70, 1100, 2056, 72, 2)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("ids", ["mixed", "sorted", None])
@pytest.mark.parametrize("shape", SHAPES)
def test_exact_sums(shape, ids, kind):
    # |hidden|, |g| <= 2056: times 256 ranks and a scale of 2, or 600 rows, below 2^23
    c = Case(sum(shape), *shape, kind, ids=ids, exact=True)
    out, hidden = c.outputs()
    c.forward(out, hidden)
    grads = c.gradients()
    c.backward(*grads)
    torch.cuda.synchronize()
    want, _, h, _ = c.want_forward()
    assert torch.equal(hidden.cpu().double(), torch.from_numpy(h))
    assert torch.equal(out.cpu(), torch.from_numpy(want).float().to(TYPES[kind]))
    (d_x, d_a, d_b), _ = c.want_backward()
    assert torch.equal(grads[0].cpu(), torch.from_numpy(d_x).float().to(TYPES[kind]))
    assert torch.equal(grads[1].cpu().double(), torch.from_numpy(d_a))
    assert torch.equal(grads[2].cpu().double(), torch.from_numpy(d_b))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,R,n,ids,scales,base", [
    (1, 4096, 4096, 16, 4, "mixed", True, True), (48, 1536, 1544, 32, 9, "mixed", True, True),
    (333, 515, 2056, 24, 3, "sorted", True, False), (520, 1000, 776, 64, 2, "mixed", False, True),
    (1100, 130, 264, 128, 4, "sorted", True, True), (700, 264, 1000, 16, 1, None, False, False)])
def test_real_values(M, N, K, R, n, ids, scales, base, kind):
    c = Case(M + N, M, N, K, R, n, kind, ids=ids, scales=scales, base=base)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_nothing_passes_between_rows_or_adapters(kind):
    # infinities and NaN in one adapter, one row, one base and one gradient stay there
    M, N, K, R, n = 300, 70, 136, 24, 5
    c = Case(3, M, N, K, R, n, kind)
    ids = host(c.ids)
    nan, inf = float("nan"), float("inf")
    c.a[2, 3, 5], c.b[2, 10, 0], c.b[2, 11, 1] = nan, inf, nan
    c.x[7], c.o_base[9, 4], c.d_out[11, 3], c.x_base[13, 2], c.h[15, 1], c.x[17, 0] = nan, inf, nan, nan, inf, -inf
    out, hidden = c.outputs()
    c.forward(out, hidden)
    grads = c.gradients()
    c.backward(*grads)
    torch.cuda.synchronize()
    own = (ids >= 0) & (ids < n)
    bad = (ids == 2) | ((own) & np.isin(np.arange(M), (7, 17)))
    rows = [t for t in range(M) if not bad[t] and t != 9]
    want, mag, h, hm = c.want_forward()
    check(host(out)[rows], want[rows], c.row_tolerance(want, mag, K + R)[rows], "out")
    check(host(hidden)[rows], h[rows], ((K + 64) * 2.0 ** -23 * hm)[rows], "hidden")
    assert np.isinf(host(out)[9, 4]) or bad[9]
    # d_out of a row without an adapter reaches nothing
    rows = [t for t in range(M) if not (ids[t] == 2 or t == 13 or (t == 11 and own[t]))]
    (d_x, d_a, d_b), (mx, ma, mb) = c.want_backward()
    check(host(grads[0])[rows], d_x[rows], c.row_tolerance(d_x, mx, N + R)[rows], "d_x")
    for i in range(n):
        if i != 2 and i not in (ids[7], ids[11], ids[17]):
            check(host(grads[1])[i], d_a[i], (M + N + 64) * 2.0 ** -23 * ma[i], "d_a")
        if i not in (ids[11], ids[15]):
            check(host(grads[2])[i], d_b[i], (M + 64) * 2.0 ** -23 * mb[i], "d_b")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_without_adapters(kind):
    M, N, K, R, n = 40, 33, 64, 16, 3
    c = Case(4, M, N, K, R, n, kind)
    c.ids = i32(np.array(NO_ADAPTER + (n,))[np.arange(M) % 4])
    c.x.fill_(float("nan"))
    c.d_out.fill_(float("nan"))
    out, hidden = c.outputs()
    c.forward(out, hidden)
    grads = c.gradients()
    c.backward(*grads)
    torch.cuda.synchronize()
    assert torch.equal(out, c.o_base) and (hidden == 0).all()
    assert torch.equal(grads[0], c.x_base) and (grads[1] == 0).all() and (grads[2] == 0).all()
    out.fill_(float("nan"))
    c.forward(out, base=None)
    torch.cuda.synchronize()
    assert (out == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_base_in_place_and_each_gradient_alone(kind):
    c = Case(5, 90, 71, 136, 24, 4, kind)
    out, hidden = c.outputs()
    c.forward(out, hidden)
    again = c.o_base.clone()
    c.forward(again, base=again)
    grads = c.gradients()
    c.backward(*grads)
    d_x = c.x_base.clone()
    c.backward(d_x=d_x, base=d_x)
    alone = c.gradients()
    c.backward(d_a=alone[1])
    c.backward(d_b=alone[2])
    torch.cuda.synchronize()
    assert torch.equal(again, out) and torch.equal(d_x, grads[0])
    assert torch.equal(alone[1], grads[1]) and torch.equal(alone[2], grads[2])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_at_any_element_and_nothing_beside_the_result(kind):
    M, N, K, R, n = 21, 71, 72, 8, 2
    c = Case(6, M, N, K, R, n, kind)

    def shifted(t):
        raw = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        raw[1:] = t.flatten()
        return raw[1:].view(t.shape)
    c.o_base, c.d_out = shifted(c.o_base), shifted(c.d_out)
    raw = torch.full((M * N + 40,), 99.0, dtype=TYPES[kind], device="cuda")
    c.forward(raw[1:1 + M * N].view(M, N))
    tails = [torch.full((size + 64,), 99.0, dtype=t, device="cuda") for size, t in
             ((M * K, TYPES[kind]), (n * R * K, torch.float32), (n * N * R, torch.float32))]
    c.backward(*(t[:-64] for t in tails))
    torch.cuda.synchronize()
    want, mag, _, _ = c.want_forward()
    got = host(raw)
    check(got[1:1 + M * N].reshape(M, N), want, c.row_tolerance(want, mag, K + R), "out")
    assert got[0] == 99 and (got[1 + M * N:] == 99).all()
    wants, mags = c.want_backward()
    check(host(tails[0])[:-64].reshape(M, K), wants[0], c.row_tolerance(wants[0], mags[0], N + R), "d_x")
    check(host(tails[1])[:-64].reshape(n, R, K), wants[1], (M + N + 64) * 2.0 ** -23 * mags[1], "d_a")
    check(host(tails[2])[:-64].reshape(n, N, R), wants[2], (M + 64) * 2.0 ** -23 * mags[2], "d_b")
    assert all((t[-64:] == 99).all() for t in tails)


def test_against_differences():
    # the objective sum(d_out * out) is linear in each of a, b and x: differences of any step are its gradient
    M, N, K, R, n = 6, 20, 24, 8, 2
    c = Case(7, M, N, K, R, n, "f32", base=False)
    out, hidden = c.outputs()
    c.forward(out, hidden)
    c.h = hidden
    grads = c.gradients()
    c.backward(*grads)
    torch.cuda.synchronize()
    at = dict(a=host(c.a), b=host(c.b), x=host(c.x))
    d = host(c.d_out)

    def f(**kw):
        v = {**at, **kw}
        return float((d * tune.adapter(v["a"], v["b"], v["x"], c.host_ids(), c.host_scales(), np.zeros((M, N)))[0]).sum())
    rng = np.random.default_rng(1)
    for name, grad in zip(("x", "a", "b"), grads):
        for _ in range(6):
            i = tuple(rng.integers(0, k) for k in at[name].shape)
            e = np.zeros(at[name].shape)
            e[i] = 0.5
            diff = f(**{name: at[name] + e}) - f(**{name: at[name] - e})
            assert abs(diff - host(grad)[i]) <= 1e-4 * (1 + abs(diff)), (name, i)


@pytest.mark.parametrize("M", [3, 700])
def test_runs_in_a_graph_and_on_another_stream(M):
    c = Case(8, M, 300, 264, 16, 3, "bf16")
    want = (*c.outputs(), *c.gradients())
    got = (*c.outputs(), *c.gradients())

    def both(o, stream=None):
        c.forward(*o[:2], stream=stream)
        c.backward(*o[2:], stream=stream)
    both(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(got, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for outs in replayed(lambda: both(got), got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_a_workspace_for_the_largest_batch_serves_smaller_ones():
    size = q4.adapter_workspace_bytes
    for N, K, R, n in ((64, 64, 8, 1), (4096, 4096, 64, 9)):
        sizes = [size(M, N, K, R, n) for M in (1, 15, 16, 17, 255, 257, 511, 513, 1000, 8191, 8193, 65535)]
        assert sizes == sorted(sizes)
    assert size(100, 64, 64, 8, 1) <= min(size(100, 65, 64, 8, 1), size(100, 64, 72, 8, 1), size(100, 64, 64, 16, 1),
                                          size(100, 64, 64, 8, 2))


def test_refusals_enqueue_nothing():
    c = Case(9, 2, 16, 64, 8, 1, "bf16")
    out, hidden = c.outputs()
    c.need -= 256
    with pytest.raises(q4.Q4Error):
        c.forward(out, hidden)
    c.need += 256
    c.sizes = (2, 17, 64, 8, 1)
    with pytest.raises(ValueError):
        c.forward(out, hidden)
    c.sizes = (2, 16, 64, 12, 1)
    with pytest.raises((q4.Q4Error, ValueError)):
        c.forward(out, hidden)
    c.sizes = (2, 16, 64, 8, 1)
    with pytest.raises(q4.Q4Error):
        c.backward()
    torch.cuda.synchronize()
    assert torch.isnan(out.float()).all() and torch.isnan(hidden).all()
