"""Router, balance loss and the gradient of the logits against their 64-bit forms on an MI355X."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
from layer_gpu_helpers import check, dev, host, i32, nan_like, replayed
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu


class Call:
    """Buffers of one router call, outputs poisoned."""

    def __init__(self, logits, K, kind, bias=None, mask=None, stats=True, **kw):
        self.M, self.E = logits.shape
        self.K, self.kind, self.kw = K, kind, kw
        self.logits = dev(logits, kind)
        self.bias = None if bias is None else dev(bias)
        self.mask = None if mask is None else torch.from_numpy(np.asarray(mask, np.uint8)).cuda()
        self.ids = torch.full((self.M, K), 777, dtype=torch.int32, device="cuda")
        self.weights = nan_like((self.M, K))
        self.stats = {}
        if stats:
            n = q4.route_workspace_bytes(self.M, self.E)
            ws = aligned_empty(n, 256)
            ws.fill_(0xAB)
            self.stats = dict(counts=torch.full((self.E,), -5, dtype=torch.int32, device="cuda"), loss=nan_like((1,)),
                              loss_grad=nan_like((self.E,)), workspace=ws, workspace_bytes=n)

    def run(self):
        q4.route(self.logits, self.M, self.E, self.K, self.ids, self.weights, select_bias=self.bias,
                 token_mask=self.mask, xdtype=self.kind, **self.kw, **self.stats)

    def outs(self):
        return [self.ids, self.weights] + [self.stats[k] for k in ("counts", "loss", "loss_grad") if self.stats]

    def check(self):
        """Against the 64-bit form on the logits as their type holds them."""
        self.run()
        torch.cuda.synchronize()
        l = host(self.logits)
        mask = None if self.mask is None else host(self.mask)
        bias = None if self.bias is None else host(self.bias)
        ids, w, counts, loss, grad = ref.route(l, self.K, self.kw.get("score", "softmax"),
                                               self.kw.get("renormalize", False), self.kw.get("scale", 1.0), bias, mask)
        assert np.array_equal(host(self.ids), ids)
        # exp's argument is rounded at its own size (up to the spread of the
        # logits), then about 16 + 10 + 16 roundings of sums over lanes, the
        # division and the renormalisation, each 2^-24 relative
        fin = l[np.isfinite(l)]
        spread = float(fin.max() - fin.min()) + float(np.abs(fin).max()) if fin.size else 0.0
        rel = (64 + 2 * spread) * 2.0 ** -24
        check(host(self.weights), w, rel * np.abs(w) + 2.0 ** -120, "weights")
        if self.stats:
            assert np.array_equal(host(self.stats["counts"]), counts)
            check(host(self.stats["loss_grad"]), grad, 2.0 ** -22 * np.abs(grad), "loss_grad")
            # sums of up to M / 4 probabilities a lane, all positive
            check(host(self.stats["loss"]), [loss], (rel + (self.M / 4 + 64) * 2.0 ** -24) * abs(loss), "loss")


def logits_of(seed, M, E, spread=2.0):
    return np.random.default_rng(seed).normal(size=(M, E)) * spread


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,K", [(1, 1, 1), (1, 64, 8), (2, 7, 7), (3, 65, 2), (5, 128, 64), (17, 167, 6), (33, 256, 8),
                                   (9, 384, 4), (4, 1000, 10), (2, 1024, 64), (130, 60, 5), (1100, 33, 3)])
def test_route(M, E, K, score, kind):
    for i, kw in enumerate((dict(), dict(renormalize=True, scale=2.5))):
        rng = np.random.default_rng(M + E + i)
        mask = (rng.random(M) > 0.2) if i else None
        Call(logits_of(M * E + i, M, E), K, kind, mask=mask, score=score, **kw).check()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,K", [(3, 16, 4), (40, 256, 8), (21, 167, 6), (2, 1024, 12)])
def test_route_with_selection_bias(M, E, K, score, kind):
    rng = np.random.default_rng(M)
    Call(logits_of(E, M, E), K, kind, bias=rng.normal(size=E) * 0.2, score=score, renormalize=True).check()
    # equal biases and repeated logits: exact ties, and sums that F32 cannot tell apart
    l = np.repeat(logits_of(E, M, (E + 1) // 2), 2, axis=1)[:, :E]
    Call(l, K, kind, bias=np.full(E, 0.25), score=score).check()
    Call(l, K, kind, bias=1e-9 * np.arange(E), score=score).check()


def test_ties_go_to_the_lowest_index():
    Call(np.zeros((3, 100)), 9, "bf16").check()
    l = np.tile([1.0, 3.0, 3.0, -0.0, 0.0, 3.0], (4, 30))
    Call(l, 64, "f32").check()
    Call(l, 64, "bf16", score="sigmoid").check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_empty_rows(score):
    rng = np.random.default_rng(4)
    l = rng.normal(size=(8, 70))
    l[0, 3:] = -np.inf                  # three experts left for six places
    l[1] = -np.inf                      # nothing left
    l[2] = np.nan                       # masked below
    l[3, 5] = np.inf                    # masked below
    l[4] = np.finfo(np.float32).min     # the type's lowest value is a number
    l[5, :64] = -np.inf
    l[6, 1::2] = np.finfo(np.float32).min
    mask = [1, 1, 0, 0, 1, 1, 1, 1]
    Call(l, 6, "f32", mask=mask, score=score, renormalize=True).check()
    Call(l, 6, "f32", mask=mask, score=score, bias=rng.normal(size=70)).check()
    off = np.zeros(70)
    off[10:] = -np.inf                  # experts taken out by the bias
    Call(rng.normal(size=(5, 70)), 12, "bf16", bias=off, score=score).check()


def test_every_token_masked():
    c = Call(logits_of(1, 6, 40), 4, "bf16", mask=np.zeros(6))
    c.check()
    assert float(c.stats["loss"]) == 0.0 and (c.ids == -1).all()


def test_nan_and_infinite_logits():
    l = logits_of(2, 3, 20)
    l[0, 4] = np.nan
    l[1, 6] = np.inf
    c = Call(l, 3, "f32", stats=False)
    c.run()
    torch.cuda.synchronize()
    ids, w = host(c.ids), host(c.weights)
    assert ids[0, 0] == 4 and np.isnan(w[0]).all()
    assert ids[1, 0] == 6 and np.isnan(w[1, 0])
    good = ref.route(host(c.logits)[2:], 3, "softmax")
    assert np.array_equal(ids[2:], good[0])


def test_extreme_sigmoids():
    l = np.array([[-200.0, -300.0, -400.0], [200.0, 300.0, -300.0], [-80.0, -81.0, 60.0]])
    Call(l, 2, "f32", score="sigmoid", stats=False).check()
    c = Call(l[:1], 2, "f32", score="sigmoid", renormalize=True)   # scores of zero in F32: weights of zero
    c.run()
    torch.cuda.synchronize()
    assert host(c.ids).tolist() == [[0, 1]] and (host(c.weights) == 0).all() and np.isfinite(host(c.stats["loss"])).all()


def test_long_batches_repeat_bit_for_bit():
    c = Call(logits_of(3, 5000, 96), 4, "bf16", mask=np.arange(5000) % 7 != 0)
    c.check()
    first = [o.clone() for o in c.outs()]
    c.stats["workspace"].fill_(0x7F)
    c.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, c.outs()))


def test_each_statistic_alone():
    base = Call(logits_of(8, 50, 24), 3, "f32")
    base.run()
    for name in ("counts", "loss", "loss_grad"):
        c = Call(logits_of(8, 50, 24), 3, "f32")
        for other in ("counts", "loss", "loss_grad"):
            if other != name:
                c.stats[other] = None
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.stats[name], base.stats[name])


def test_odd_addresses():
    l = logits_of(12, 9, 33)
    a = Call(l, 5, "bf16")
    a.run()
    raw = torch.empty(l.size + 1, dtype=torch.bfloat16, device="cuda")
    raw[1:] = a.logits.flatten()
    b = Call(l, 5, "bf16")
    b.logits = raw[1:]
    b.run()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.outs(), b.outs()))


def test_runs_in_a_graph():
    c = Call(logits_of(6, 300, 64), 8, "bf16", renormalize=True)
    c.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in c.outs()]
    for got in replayed(c.run, c.outs()):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- the gradient ----

def backward_case(M, E, K, kind, score, renormalize, scale, use_w=True, use_l=True, seed=0, logits=None):
    rng = np.random.default_rng(seed + M + E)
    l = dev(logits_of(seed, M, E) if logits is None else logits, kind)
    lh = host(l)
    ids, _, _, _, grad = ref.route(lh, K, score, mask=rng.random(M) > 0.15)
    dw, d_loss = rng.normal(size=(M, K)).astype(np.float32), np.float32(0.3)
    grad = grad.astype(np.float32)
    out = nan_like((M, E), kind)
    q4.route_backward(l, M, E, K, i32(ids), out, d_weights=dev(dw) if use_w else None,
                      d_loss=dev([d_loss]) if use_l else None, loss_grad=dev(grad) if use_l else None, score=score,
                      renormalize=renormalize, scale=scale, xdtype=kind)
    torch.cuda.synchronize()
    args = (ids, score, renormalize, scale, dw.astype(np.float64) * use_w, float(d_loss) * use_l, grad.astype(np.float64))
    return lh, host(out), args


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("M,E,K", [(1, 1, 1), (1, 64, 8), (3, 7, 7), (17, 167, 6), (40, 256, 8), (3, 1000, 12), (2, 1024, 64),
                                   (601, 33, 2)])
def test_route_backward(M, E, K, renormalize, score, kind):
    lh, got, args = backward_case(M, E, K, kind, score, renormalize, 2.5)
    want, mag = ref.route_backward(lh, *args)
    # scores within (32 + spread) 2^-24, twice, plus sums over lanes and products
    rel = (128 + 4 * (np.abs(lh).max() * 2)) * 2.0 ** -24
    check(got, want, ref.HALF_STEP[kind] * np.abs(want) + rel * mag + 2.0 ** -120, "d_logits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_parts(score):
    for use in (dict(use_w=False), dict(use_l=False)):
        lh, got, args = backward_case(20, 90, 5, "f32", score, True, 1.0, **use)
        want, mag = ref.route_backward(lh, *args)
        check(got, want, 2.0 ** -16 * mag + 2.0 ** -120, "d_logits")


def test_route_backward_against_differences():
    for score in ("softmax", "sigmoid"):
        lh, got, args = backward_case(3, 11, 3, "f32", score, True, 1.5, seed=2)
        h = 1e-5
        for at in np.ndindex(3, 11):
            up, down = lh.copy(), lh.copy()
            up[at] += h
            down[at] -= h
            num = (ref.route_objective(up, *args) - ref.route_objective(down, *args)) / (2 * h)
            assert abs(num - got[at]) < 1e-5, (score, at)


def test_route_backward_of_far_sigmoids():
    # 1 - sigmoid is formed without cancellation: small gradients keep their digits
    l = np.array([[12.0, 15.0, -14.0, 9.0, 16.0]])
    lh, got, args = backward_case(1, 5, 3, "f32", "sigmoid", False, 1.0, logits=l, seed=3)
    want, mag = ref.route_backward(lh, *args)
    check(got, want, 2.0 ** -15 * mag + 2.0 ** -120, "d_logits")


def test_route_backward_empty_rows_and_foreign_ids():
    l = logits_of(5, 4, 12)
    l[1] = np.nan
    ids = np.array([[3, 99, -1], [-1, -1, -1], [0, 1, 2], [5, -7, 12]])
    dw = np.random.default_rng(1).normal(size=(4, 3)).astype(np.float32)
    out = nan_like((4, 12))
    q4.route_backward(dev(l), 4, 12, 3, i32(ids), out, d_weights=dev(dw), renormalize=True, xdtype="f32")
    torch.cuda.synchronize()
    want, mag = ref.route_backward(host(dev(l)), ids, "softmax", True, 1.0, dw.astype(np.float64), 0.0, np.zeros(12))
    check(host(out), want, 2.0 ** -16 * mag + 2.0 ** -120, "d_logits")
    assert (host(out)[1] == 0).all()


def test_route_backward_in_a_graph():
    l, ids = dev(logits_of(7, 50, 40), "bf16"), i32(np.random.default_rng(2).integers(-1, 40, size=(50, 4)))
    dw, out = dev(np.random.default_rng(3).normal(size=(50, 4))), nan_like((50, 40), "bf16")
    call = lambda: q4.route_backward(l, 50, 40, 4, ids, out, d_weights=dw)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    for got, in replayed(call, [out]):
        assert torch.equal(got, want)


def test_refusals_enqueue_nothing():
    c = Call(logits_of(1, 4, 8), 2, "f32")
    c.stats["workspace_bytes"] = 16
    with pytest.raises(q4.Q4Error):
        c.run()
    with pytest.raises(ValueError):
        q4.route(c.logits, 5, 8, 2, c.ids, c.weights, xdtype="f32")
    torch.cuda.synchronize()
    assert (c.ids == 777).all()
