"""The router over groups of experts against its 64-bit form on an MI355X."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import quantized_moe_expert_q4_amd as q4
import tuning_reference as tune
from layer_gpu_helpers import check, dev, host, i32, nan_like, replayed
from quantized_moe_expert_q4_amd.device import aligned_empty

pytestmark = pytest.mark.gpu


class Call:
    """Buffers of one call, outputs poisoned."""

    def __init__(self, logits, K, groups, top_groups, group_top, kind, bias=None, mask=None, stats=True, **kw):
        self.M, self.E = logits.shape
        self.K, self.kind, self.kw, self.g = K, kind, kw, (groups, top_groups, group_top)
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

    def run(self, stream=None):
        groups, top_groups, group_top = self.g
        q4.route_groups(self.logits, self.M, self.E, self.K, groups, top_groups, self.ids, self.weights,
                        group_top=group_top, select_bias=self.bias, token_mask=self.mask, xdtype=self.kind, stream=stream,
                        **self.kw, **self.stats)

    def outs(self):
        return [self.ids, self.weights] + [self.stats[k] for k in ("counts", "loss", "loss_grad") if self.stats]

    def check(self):
        self.run()
        torch.cuda.synchronize()
        l = host(self.logits)
        mask = None if self.mask is None else host(self.mask)
        bias = None if self.bias is None else host(self.bias)
        score = self.kw.get("score", "softmax")
        ids, w, counts, loss, grad = tune.route_groups(l, self.K, *self.g, score, self.kw.get("renormalize", False),
                                                       self.kw.get("scale", 1.0), bias, mask)
        assert np.array_equal(host(self.ids), ids)
        # exp's argument is rounded at its own size (up to the spread of the
        # logits), then about 16 + 10 + 16 roundings of sums over lanes, the
        # division and the renormalisation, each 2^-24 relative
        fin = l[np.isfinite(l) & (np.abs(l) < 1e30)]
        spread = float(fin.max() - fin.min()) + float(np.abs(fin).max()) if fin.size else 0.0
        rel = (64 + 2 * spread) * 2.0 ** -24
        check(host(self.weights), w, rel * np.abs(w) + 2.0 ** -120, "weights")
        if self.stats:
            assert np.array_equal(host(self.stats["counts"]), counts)
            check(host(self.stats["loss_grad"]), grad, 2.0 ** -22 * np.abs(grad), "loss_grad")
            check(host(self.stats["loss"]), [loss], (rel + 128 * 2.0 ** -24) * abs(loss), "loss")


def logits_of(seed, M, E, spread=2.0):
    return np.random.default_rng(seed).normal(size=(M, E)) * spread


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,K,groups,top", [
    (1, 1, 1, 1, 1), (1, 2, 1, 2, 1), (3, 64, 8, 8, 4), (2, 64, 4, 64, 5), (5, 60, 7, 6, 2), (17, 160, 6, 10, 3),
    (33, 256, 8, 8, 4), (9, 384, 12, 3, 1), (4, 1000, 10, 8, 2), (2, 1024, 64, 32, 5), (2, 1024, 6, 1, 1),
    (130, 21, 5, 7, 3), (1100, 36, 3, 12, 6), (4200, 96, 2, 4, 1)])
def test_route_groups(M, E, K, groups, top, score, kind):
    rng = np.random.default_rng(M + E)
    for group_top, bias, mask in ((1, None, None), (2, None, rng.random(M) > 0.2), (1, rng.normal(size=E) * 0.2, None),
                                  (2, rng.normal(size=E) * 0.2, rng.random(M) > 0.2)):
        Call(logits_of(M * E, M, E), K, groups, top, group_top, kind, bias=bias, mask=mask, score=score, renormalize=True,
             scale=2.5).check()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("M,E,K,groups,top", [(40, 256, 8, 8, 4), (3, 16, 4, 4, 2), (6, 1024, 12, 16, 5), (21, 160, 6, 10, 3)])
def test_ties_and_sums_that_f32_cannot_tell_apart(M, E, K, groups, top, group_top, kind):
    # whole groups alike, then biases of 1e-9 that only 64 bits see
    size = E // groups
    l = np.tile(logits_of(E, M, size), (1, groups))
    for score in ("softmax", "sigmoid"):
        Call(l, K, groups, top, group_top, kind, score=score).check()
        Call(l, K, groups, top, group_top, kind, bias=np.full(E, 0.25), score=score).check()
        # multiples of 2^-30, up to 1e-6: exact in F32 and, beside a score, in 64 bits
        bias = np.random.default_rng(E).permutation(E) * 2.0 ** -30
        Call(l, K, groups, top, group_top, kind, bias=bias, score=score).check()
    Call(np.zeros((M, E)), K, groups, top, group_top, kind).check()


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_empty_groups(score, group_top):
    rng = np.random.default_rng(4)
    E, groups, low = 72, 6, np.finfo(np.float32).min
    l = rng.normal(size=(9, E))
    l[0, 3:] = -np.inf                  # one group with three experts left
    l[1] = -np.inf                      # nothing left
    l[2] = np.nan                       # masked below
    l[3, 5] = np.inf                    # masked below
    l[4] = low                          # the type's lowest value is a number
    l[5, :60] = -np.inf                 # one group left of six
    l[6, 1::2] = low
    l[7, ::12] = 9.0
    l[7, 1:12] = -np.inf                # a group of one expert, the highest
    mask = [1, 1, 0, 0, 1, 1, 1, 1, 1]
    Call(l, 6, groups, 2, group_top, "f32", mask=mask, score=score, renormalize=True).check()
    Call(l, 6, groups, 2, group_top, "f32", mask=mask, score=score, bias=rng.normal(size=E)).check()
    off = np.zeros(E)
    off[10:] = -np.inf                  # experts taken out by the bias
    Call(rng.normal(size=(5, E)), 12, groups, 3, group_top, "bf16", bias=off, score=score).check()
    off[10:] = low                      # biases of the lowest value: two of them add up below F32
    Call(rng.normal(size=(5, E)), 30, groups, 3, group_top, "bf16", bias=off, score=score).check()


def test_a_nan_ranks_its_group_first():
    l = np.tile(np.arange(48.0), (2, 1)) / 8
    l[1, 5] = np.nan
    c = Call(l, 3, 6, 2, 1, "f32", stats=False, score="sigmoid")
    c.run()
    torch.cuda.synchronize()
    assert host(c.ids).tolist() == [[47, 46, 45], [5, 47, 46]]


def test_every_token_masked():
    c = Call(logits_of(1, 6, 40), 4, 5, 2, 2, "bf16", mask=np.zeros(6))
    c.check()
    assert float(c.stats["loss"]) == 0.0 and (c.ids == -1).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_all_groups_kept_is_the_router_without_groups(kind):
    M, E, K = 70, 128, 6
    rng = np.random.default_rng(3)
    c = Call(logits_of(5, M, E), K, 8, 8, 2, kind, bias=0.1 * rng.normal(size=E), score="sigmoid", renormalize=True)
    c.run()
    got = [o.clone() for o in c.outs()]
    q4.route(c.logits, M, E, K, c.ids, c.weights, select_bias=c.bias, xdtype=kind, **c.kw, **c.stats)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, c.outs()))


@pytest.mark.parametrize("M", [5, 5000])
def test_runs_in_a_graph_and_on_another_stream(M):
    c = Call(logits_of(2, M, 256), 8, 8, 4, 2, "bf16", bias=np.zeros(256), score="sigmoid", renormalize=True)
    c.run()
    torch.cuda.synchronize()
    want = [o.clone() for o in c.outs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(c.outs(), want))
    for got in replayed(c.run, c.outs()):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_with_the_ids_of_the_groups():
    # the router's gradient at the ids chosen within groups: the choice has none
    M, E, K = 12, 64, 6
    for score in ("softmax", "sigmoid"):
        c = Call(logits_of(8, M, E), K, 8, 3, 2, "f32", score=score, renormalize=True, scale=2.5)
        c.run()
        rng = np.random.default_rng(1)
        dw, dl = rng.normal(size=(M, K)), 0.3
        d_logits = nan_like((M, E))
        q4.route_backward(c.logits, M, E, K, c.ids, d_logits, d_weights=dev(dw), d_loss=dev([dl]),
                          loss_grad=c.stats["loss_grad"], xdtype="f32", **c.kw)
        torch.cuda.synchronize()
        ids = host(c.ids)
        dw, dl = host(dev(dw)), float(host(dev([dl]))[0])
        grad = host(c.stats["loss_grad"])
        want, mag = ref.route_backward(host(c.logits), ids, score, True, 2.5, dw, dl, grad)
        check(host(d_logits), want, 256 * 2.0 ** -24 * mag, score)
        # and against differences of the objective (step 1e-4: their error is about 1e-8 of its third derivative)
        l, step = host(c.logits), 1e-4
        for t, e in ((0, int(ids[0, 0])), (3, 5), (7, int(ids[7, 2]))):
            up, down = l.copy(), l.copy()
            up[t, e] += step
            down[t, e] -= step
            diff = (tune_objective(up, ids, score, dw, dl, grad) - tune_objective(down, ids, score, dw, dl, grad)) / (2 * step)
            assert abs(diff - want[t, e]) <= 1e-6 * (1 + np.abs(want).max())


def tune_objective(l, ids, score, dw, dl, grad):
    return ref.route_objective(l, ids, score, True, 2.5, dw, dl, grad)


def test_refusals_enqueue_nothing():
    c = Call(logits_of(1, 2, 64), 8, 8, 4, 2, "bf16")
    for groups, top, group_top in ((7, 4, 2), (8, 9, 2), (8, 4, 3), (8, 0, 1), (64, 7, 1)):
        c.g = (groups, top, group_top)
        with pytest.raises(q4.Q4Error):
            c.run()
    torch.cuda.synchronize()
    assert (c.ids == 777).all()
