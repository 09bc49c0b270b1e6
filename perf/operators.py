"""Workloads of the mixture-of-experts layer's operators around the routed experts.

Five passes are described here, each in a plain form (elementary torch
operations) and, with ``own`` true, as calls of the library:

``linear``            tokens times a 4-bit matrix with a scale (and an optional
                      bias) for each group of weights of a row;
``route``             router logits to expert ids and weights, and for training
                      the per-expert counts, the balance loss and its gradient;
``route_backward``    the gradient of the router logits;
``combine``           the weighted sum of a token's expert outputs;
``combine_backward``  the gradients of the expert outputs and of the weights.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token through one projection: the smallest call, latency only
        dict(name="linear_token", op="linear", M=1, N=1536, K=4096, group=64, affine=False, x="bf16", scales="bf16"),
        # one decoded token through a vocabulary head: a long weight stream
        dict(name="linear_head", op="linear", M=1, N=131072, K=4096, group=128, affine=True, x="bf16", scales="bf16"),
        # a few drafted tokens in float32, rows and groups that end inside a tile
        dict(name="linear_draft", op="linear", M=5, N=6147, K=4104, group=32, affine=True, x="f32", scales="f32"),
        # a batch of decoding requests through a wide projection
        dict(name="linear_batch", op="linear", M=64, N=14336, K=7168, group=128, affine=False, x="bf16", scales="f32"),
        # one decoded token, serving: no statistics
        dict(name="route_token", op="route", M=1, E=64, K=8, logits="f32", score="softmax", bias=False, renorm=True,
             scale=1.0, masked=False, stats=False),
        # a training step's tokens over many experts, chosen by sigmoid score plus bias, with padding
        dict(name="route_train", op="route", M=8192, E=256, K=8, logits="bf16", score="sigmoid", bias=True, renorm=True,
             scale=2.5, masked=True, stats=True),
        # an odd batch over an odd number of experts
        dict(name="route_odd", op="route", M=1003, E=167, K=6, logits="f32", score="softmax", bias=False, renorm=False,
             scale=1.0, masked=True, stats=True),
        # the gradients of the two training batches above, the other way round in type
        dict(name="route_back", op="route_backward", M=8192, E=256, K=8, logits="bf16", score="softmax", renorm=True,
             scale=1.0, masked=True),
        dict(name="route_back_odd", op="route_backward", M=1003, E=167, K=6, logits="f32", score="sigmoid", renorm=True,
             scale=2.5, masked=True),
        # one decoded token's eight expert outputs
        dict(name="combine_token", op="combine", M=1, H=4096, K=8, y="bf16", base=True, masked=False),
        # a prompt's expert outputs onto its residual
        dict(name="combine_prompt", op="combine", M=4096, H=7168, K=8, y="bf16", base=True, masked=True),
        # their gradients, for outputs and weights
        dict(name="combine_back", op="combine_backward", M=2048, H=6144, K=8, y="bf16", masked=True),
    ]


def _spread(rng, lo, hi):
    """A whole number whose logarithm is uniform over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "route", "route_backward", "combine", "combine_backward"])
    kind = rng.choice(["bf16", "f32"])
    if op == "linear":
        K = 8 * _spread(rng, 32, 1792)                       # 256 .. 14336
        N = _spread(rng, 64, min(131072, (1 << 29) // K))
        M = _spread(rng, 1, 64)
        # no more weights times tokens than the largest listed case
        M = max(1, min(M, (64 * 14336 * 7168) // (N * K)))
        return dict(op=op, M=M, N=N, K=K, group=rng.choice([32, 64, 128]), affine=rng.random() < 0.5, x=kind,
                    scales=rng.choice(["bf16", "f32"]))
    if op in ("route", "route_backward"):
        E = _spread(rng, 8, 512)
        M = _spread(rng, 1, min(16384, (8192 * 256) // E))
        case = dict(op=op, M=M, E=E, K=rng.randint(1, min(E, 12)), logits=kind, score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.6)
        if op == "route":
            case.update(bias=rng.random() < 0.4, stats=rng.random() < 0.7)
        return case
    H = 8 * _spread(rng, 32, 1024)                           # 256 .. 8192
    K = rng.randint(1, 10)
    size = 4 if kind == "f32" else 2
    M = _spread(rng, 1, min(8192, (2048 * 6144 * 8 * 2) // (H * K * size)))
    case = dict(op=op, M=M, H=H, K=K, y=kind, masked=rng.random() < 0.6)
    if op == "combine":
        case.update(base=rng.random() < 0.6)
    return case


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "linear":
        N, s = case["N"], 2 if case["scales"] == "bf16" else 4
        groups = -(-K // case["group"]) * (2 if case["affine"] else 1)
        b = 2 if case["x"] == "bf16" else 4
        return {"bytes": N * K // 2 + N * groups * s + M * K * b + M * N * b, "flops": 2 * M * N * K}
    if case["op"] in ("route", "route_backward"):
        E, b = case["E"], 2 if case["logits"] == "bf16" else 4
        if case["op"] == "route":
            extra = (4 * E if case["bias"] else 0) + (M if case["masked"] else 0) + (8 * E + 4 if case["stats"] else 0)
            return {"bytes": M * E * b + M * K * 8 + extra, "flops": 6 * M * E}
        return {"bytes": 2 * M * E * b + M * K * 8 + 4 * E + 4, "flops": 10 * M * E}
    H, b = case["H"], 2 if case["y"] == "bf16" else 4
    pairs = M * K * H
    if case["op"] == "combine":
        return {"bytes": pairs * b + M * H * b * (2 if case["base"] else 1) + M * K * 8, "flops": 2 * pairs}
    return {"bytes": 2 * pairs * b + M * H * b + M * K * 12, "flops": 3 * pairs}


# --------------------------------------------------------------- the inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _padding(M, gen):
    """1 for a token, 0 for padding: about one sixteenth of the batch, at random places."""
    return (torch.rand(M, device="cuda", generator=gen) > 1 / 16).to(torch.uint8)


def _linear_inputs(case, gen):
    M, N, K, G = case["M"], case["N"], case["K"], case["group"]
    weights = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    for at in range(0, N, 8192):
        # bell-shaped levels around the middle one, as quantising a weight matrix gives them
        part = weights[at:at + 8192]
        q = torch.randn(part.shape[0], K, device="cuda", generator=gen).mul_(2.7).round_().add_(8).clamp_(0, 15).to(torch.uint8)
        part.copy_(q[:, 0::2] | (q[:, 1::2] << 4))
    groups = -(-K // G)
    kind = _TYPES[case["scales"]]
    scales = (0.005 + 0.015 * torch.rand(N, groups, device="cuda", generator=gen)).to(kind)
    state = dict(weights=weights, scales=scales, biases=None)
    if case["affine"]:
        state["biases"] = (-7.5 * scales.float() + 0.01 * torch.randn(N, groups, device="cuda", generator=gen)).to(kind)
    x = torch.randn(M, K, device="cuda", generator=gen)
    x *= 1 + 15 * (torch.rand(1, K, device="cuda", generator=gen) < 0.01)      # a few channels stand out
    state["x"] = x.to(_TYPES[case["x"]])
    return state


def _route_inputs(case, gen):
    M, E = case["M"], case["E"]
    logits = 1.5 * torch.randn(M, E, device="cuda", generator=gen) + 0.7 * torch.randn(1, E, device="cuda", generator=gen)
    state = dict(logits=logits.to(_TYPES[case["logits"]]), bias=None, mask=None)
    if case.get("bias"):
        state["bias"] = 0.1 * torch.randn(E, device="cuda", generator=gen)
    if case["masked"]:
        state["mask"] = _padding(M, gen)
    return state


def _combine_inputs(case, gen):
    M, K, H, kind = case["M"], case["K"], case["H"], _TYPES[case["y"]]
    y = torch.empty(M, K, H, dtype=kind, device="cuda")
    for at in range(0, M, 512):
        part = y[at:at + 512]
        part.copy_(torch.randn(part.shape, device="cuda", generator=gen))
    weights = torch.rand(M, K, device="cuda", generator=gen) + 0.05
    weights /= weights.sum(1, keepdim=True)
    slots = 64
    ids = torch.rand(M, slots, device="cuda", generator=gen).argsort(1)[:, :K].to(torch.int32)
    if case["masked"]:
        keep = _padding(M, gen).bool()
        ids = torch.where(keep[:, None], ids, -1)
        weights = torch.where(keep[:, None], weights, 0.0)
    state = dict(y=y, weights=weights.contiguous(), ids=ids.contiguous(), slots=slots)
    if case["op"] == "combine":
        state["base"] = torch.randn(M, H, device="cuda", generator=gen).to(kind) if case["base"] else None
    else:
        state["d_out"] = torch.randn(M, H, device="cuda", generator=gen).to(kind)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    M, K = case["M"], case["K"]
    op = case["op"]
    new = lambda shape, kind: torch.empty(shape, dtype=kind, device="cuda")
    if op == "linear":
        state = _linear_inputs(case, gen)
        state["out"] = new((M, case["N"]), state["x"].dtype)
    elif op == "route":
        state = _route_inputs(case, gen)
        state["ids"], state["weights"] = new((M, K), torch.int32), new((M, K), torch.float32)
        if case["stats"]:
            state["counts"], state["loss"] = new((case["E"],), torch.int32), new((1,), torch.float32)
            state["loss_grad"] = new((case["E"],), torch.float32)
            if own:
                import quantized_moe_expert_q4_amd as q4
                from quantized_moe_expert_q4_amd.device import aligned_empty
                state["workspace_bytes"] = q4.route_workspace_bytes(M, case["E"])
                state["workspace"] = aligned_empty(state["workspace_bytes"], 256)
    elif op == "route_backward":
        state = _route_inputs(case, gen)
        # what the forward pass of this batch left: the choice and the loss's gradient
        state["ids"] = _choose(state["logits"].double(), K, state["mask"])
        state["loss_grad"] = _loss_grad(state["ids"], case["E"], K)
        state["d_weights"] = torch.randn(M, K, device="cuda", generator=gen)
        state["d_loss"] = torch.full((1,), 0.01, device="cuda")
        state["d_logits"] = torch.empty_like(state["logits"])
    else:
        state = _combine_inputs(case, gen)
        if op == "combine":
            state["out"] = new((M, case["H"]), state["y"].dtype)
        else:
            state["d_y"], state["d_weights"] = torch.empty_like(state["y"]), new((M, K), torch.float32)
    state["case"] = case
    return state


# ---------------------------------------------------------- the plain forms

def _choose(keys, K, mask):
    """The K highest keys of each row, ties to the lowest index; -1 in the place of a masked token or of -inf."""
    top, ids = torch.sort(keys, dim=1, descending=True, stable=True)
    ids = torch.where(top[:, :K] == -math.inf, -1, ids[:, :K])
    if mask is not None:
        ids = torch.where(mask.bool()[:, None], ids, -1)
    return ids.to(torch.int32)


def _loss_grad(ids, E, K):
    """E c_e / (K T^2) for the counts c of the chosen experts and the T tokens that chose any."""
    chosen = ids >= 0
    counts = torch.zeros(E, dtype=torch.float64, device=ids.device)
    counts.index_add_(0, ids.clamp(min=0).flatten().long(), chosen.flatten().double())
    tokens = chosen.any(1).sum().double()
    return torch.where(tokens > 0, E * counts / (K * tokens * tokens), 0.0).float()


def _scores(logits, score):
    """(score, probability) of every expert: the same for softmax; for sigmoid the probability sums to one."""
    if score == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        return p, p
    s = 1 / (1 + torch.exp(-logits))
    return s, s / s.sum(1, keepdim=True)


def _linear_plain(st):
    case = st["case"]
    N, K, G = case["N"], case["K"], case["group"]
    q = torch.stack((st["weights"] & 15, st["weights"] >> 4), dim=2).view(N, K).float()
    wide = lambda t: t.float().repeat_interleave(G, dim=1)[:, :K]
    if st["biases"] is None:
        w = (q - 8) * wide(st["scales"])
    else:
        w = q * wide(st["scales"]) + wide(st["biases"])
    return (st["x"].float() @ w.t()).to(st["x"].dtype)


def _route_plain(st):
    case = st["case"]
    K, E = case["K"], case["E"]
    logits = st["logits"].float()
    score, prob = _scores(logits, case["score"])
    if st["bias"] is None:
        keys = logits
    else:
        keys = _scores(logits.double(), case["score"])[0] + st["bias"].double()
    ids = _choose(keys, K, st["mask"])
    w = torch.where(ids >= 0, torch.gather(score, 1, ids.clamp(min=0).long()), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    out = [ids, case["scale"] * w]
    if case["stats"]:
        chosen = ids >= 0
        counts = torch.zeros(E, dtype=torch.int32, device=ids.device)
        counts.index_add_(0, ids.clamp(min=0).flatten().long(), chosen.flatten().to(torch.int32))
        there = chosen.any(1, keepdim=True)
        sums = torch.where(there, prob, 0.0).sum(0, dtype=torch.float64)
        grad = _loss_grad(ids, E, K)
        out += [counts, (grad.double() * sums).sum().float().view(1), grad]
    return out


def _route_backward_plain(st):
    case = st["case"]
    ids, logits = st["ids"], st["logits"].float()
    there = ids[:, :1] >= 0
    chosen = ids >= 0
    at = ids.clamp(min=0).long()
    score, prob = _scores(logits, case["score"])
    dw = case["scale"] * torch.where(chosen, st["d_weights"], 0.0)
    if case["renorm"]:
        picked = torch.where(chosen, torch.gather(score, 1, at), 0.0)
        total = picked.sum(1, keepdim=True)
        dw = torch.where(total > 0, (dw - (dw * picked).sum(1, keepdim=True) / total) / total, 0.0)
    d_score = torch.zeros_like(score).scatter_add_(1, at, torch.where(chosen, dw, 0.0))
    d_prob = st["d_loss"] * st["loss_grad"]
    if case["score"] == "softmax":
        g = d_score + d_prob
        d = prob * (g - (prob * g).sum(1, keepdim=True))
    else:
        d_score = d_score + (d_prob - (prob * d_prob).sum(1, keepdim=True)) / score.sum(1, keepdim=True)
        d = d_score * score * (1 - score)
    return torch.where(there, d, 0.0).to(st["logits"].dtype)


def _live(st):
    return ((st["ids"] >= 0) & (st["ids"] < st["slots"]))[:, :, None]


def _combine_plain(st):
    rows = torch.where(_live(st), st["y"].float(), 0.0)
    out = (st["weights"][:, :, None] * rows).sum(1)
    if st["base"] is not None:
        out = out + st["base"].float()
    return out.to(st["y"].dtype)


def _combine_backward_plain(st):
    live = _live(st)
    d_out = st["d_out"].float()[:, None, :]
    d_y = torch.where(live, st["weights"][:, :, None] * d_out, 0.0).to(st["y"].dtype)
    d_w = (torch.where(live, st["y"].float(), 0.0) * d_out).sum(2)
    return [d_y, d_w]


_PLAIN = {"linear": _linear_plain, "route": _route_plain, "route_backward": _route_backward_plain,
          "combine": _combine_plain, "combine_backward": _combine_backward_plain}


# ------------------------------------------------------- the library's calls

def _library(st):
    import quantized_moe_expert_q4_amd as q4
    case = st["case"]
    op, M, K = case["op"], case["M"], case["K"]
    if op == "linear":
        q4.linear(st["weights"], st["scales"], st["x"], M, case["N"], K, case["group"], st["out"], biases=st["biases"],
                  xdtype=case["x"])
        return st["out"]
    if op == "route":
        stats = {k: st[k] for k in ("counts", "loss", "loss_grad", "workspace", "workspace_bytes")} if case["stats"] else {}
        q4.route(st["logits"], M, case["E"], K, st["ids"], st["weights"], score=case["score"], renormalize=case["renorm"],
                 scale=case["scale"], select_bias=st["bias"], token_mask=st["mask"], xdtype=case["logits"], **stats)
        return [st["ids"], st["weights"]] + [st[k] for k in ("counts", "loss", "loss_grad") if case["stats"]]
    if op == "route_backward":
        q4.route_backward(st["logits"], M, case["E"], K, st["ids"], st["d_logits"], d_weights=st["d_weights"],
                          d_loss=st["d_loss"], loss_grad=st["loss_grad"], score=case["score"],
                          renormalize=case["renorm"], scale=case["scale"], xdtype=case["logits"])
        return st["d_logits"]
    if op == "combine":
        q4.combine(st["y"], st["weights"], M, K, case["H"], st["out"], slot_ids=st["ids"], num_slots=st["slots"],
                   base=st["base"], xdtype=case["y"])
        return st["out"]
    q4.combine_backward(st["d_out"], st["y"], st["weights"], M, K, case["H"], d_y=st["d_y"], d_weights=st["d_weights"],
                        slot_ids=st["ids"], num_slots=st["slots"], xdtype=case["y"])
    return [st["d_y"], st["d_weights"]]


def run(state):
    return _library(state) if own else _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------- the definitions in 64 bits

def _exact_linear(st):
    case = st["case"]
    N, K, G = case["N"], case["K"], case["group"]
    x = st["x"].double()
    out = torch.empty(case["M"], N, dtype=torch.float64, device="cuda")
    at = torch.arange(K, device="cuda")
    for lo in range(0, N, 4096):
        byte = st["weights"][lo:lo + 4096].index_select(1, at // 2).int()
        q = torch.bitwise_right_shift(byte, (4 * (at % 2)).int()).bitwise_and(15).double()
        s = st["scales"][lo:lo + 4096].double().index_select(1, at // G)
        off = -8 * s if st["biases"] is None else st["biases"][lo:lo + 4096].double().index_select(1, at // G)
        out[:, lo:lo + 4096] = torch.matmul(x, torch.addcmul(off, q, s).t())
    return out


def _exact_score(logits, score):
    logits = logits.double()
    if score == "sigmoid":
        s = torch.exp(-torch.log1p(torch.exp(-logits.abs())) + logits.clamp(max=0))
        return s, s / s.sum(1, keepdim=True)
    p = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True))
    return p, p


def _exact_ids(keys, K, mask):
    keys = keys.clone()
    index = torch.arange(keys.shape[1], device=keys.device)
    ids = []
    for _ in range(K):
        best = keys.amax(1, keepdim=True)
        first = torch.where(keys == best, index, keys.shape[1]).amin(1, keepdim=True)
        ids.append(torch.where(best > -math.inf, first, -1))
        keys.scatter_(1, first, -math.inf)
    ids = torch.cat(ids, 1)
    if mask is not None:
        ids[mask == 0] = -1
    return ids


def _exact_route(st):
    case = st["case"]
    E, K = case["E"], case["K"]
    score, prob = _exact_score(st["logits"], case["score"])
    keys = st["logits"].double() if st["bias"] is None else score + st["bias"].double()
    ids = _exact_ids(keys, K, st["mask"])
    onehot = torch.zeros(case["M"], E, dtype=torch.float64, device="cuda")
    onehot.scatter_add_(1, ids.clamp(min=0), (ids >= 0).double())
    kept = score * onehot
    if case["renorm"]:
        total = kept.sum(1, keepdim=True)
        kept = torch.where(total > 0, kept / total, 0.0)
    weights = case["scale"] * torch.gather(kept, 1, ids.clamp(min=0)) * (ids >= 0)
    out = [ids.to(torch.int32), weights]
    if case["stats"]:
        counts = onehot.sum(0)
        tokens = float((ids[:, 0] >= 0).sum())
        share = counts / (K * tokens) if tokens else 0 * counts
        mean = prob[ids[:, 0] >= 0].sum(0) / tokens if tokens else 0 * counts
        out += [counts.to(torch.int32), (E * (share * mean).sum()).view(1), E * share / max(tokens, 1.0)]
    return out


def _exact_route_backward(st):
    case = st["case"]
    ids = st["ids"].long()
    score, prob = _exact_score(st["logits"], case["score"])
    E = case["E"]
    picked = torch.zeros_like(score).scatter_add_(1, ids.clamp(min=0), (ids >= 0).double())
    upstream = torch.zeros_like(score).scatter_add_(1, ids.clamp(min=0), (ids >= 0) * st["d_weights"].double())
    upstream *= case["scale"]
    if case["renorm"]:
        total = (score * picked).sum(1, keepdim=True)
        mean = (upstream * score).sum(1, keepdim=True) / total
        upstream = torch.where(total > 0, picked * (upstream - mean) / total, 0.0)
    loss = (st["d_loss"].double() * st["loss_grad"].double()).expand(case["M"], E)
    if case["score"] == "softmax":
        both = upstream + loss
        grad = prob * both - prob * (prob * both).sum(1, keepdim=True)
    else:
        through = (loss - (prob * loss).sum(1, keepdim=True)) / score.sum(1, keepdim=True)
        other, _ = _exact_score(-st["logits"].double(), "sigmoid")
        grad = score * other * (upstream + through)
    return grad * (ids[:, :1] >= 0)


def _exact_combine(st):
    case = st["case"]
    out = torch.zeros(case["M"], case["H"], dtype=torch.float64, device="cuda")
    if st["base"] is not None:
        out += st["base"].double()
    for j in range(case["K"]):
        live = (st["ids"][:, j] >= 0) & (st["ids"][:, j] < st["slots"])
        out[live] += st["weights"][live, j, None].double() * st["y"][live, j].double()
    return out


def _exact_combine_backward(st):
    case = st["case"]
    d_y = torch.zeros(case["M"], case["K"], case["H"], dtype=torch.float64, device="cuda")
    d_w = torch.zeros(case["M"], case["K"], dtype=torch.float64, device="cuda")
    d_out = st["d_out"].double()
    for j in range(case["K"]):
        live = (st["ids"][:, j] >= 0) & (st["ids"][:, j] < st["slots"])
        d_y[live, j] = st["weights"][live, j, None].double() * d_out[live]
        d_w[live, j] = torch.linalg.vecdot(d_out[live], st["y"][live, j].double())
    return [d_y, d_w]


_EXACT = {"linear": _exact_linear, "route": _exact_route, "route_backward": _exact_route_backward,
          "combine": _exact_combine, "combine_backward": _exact_combine_backward}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
