"""Workloads of the operators that serve and tune a mixture-of-experts layer with adapters.

Four passes are described here, each in a plain form (elementary torch
operations) and, with ``own`` true, as calls of the library:

``route_groups``      router logits to expert ids and weights where a token's experts
                      come from its best groups of experts only; for training also
                      the per-expert counts, the balance loss and its gradient;
``adapter``           the low-rank adapters of many requests beside a projection they
                      share: every row has an adapter of its own, or none;
``adapter_backward``  the gradients of the adapters and of their input;
``linear_backward``   the gradient of the input of a 4-bit linear, which is frozen
                      while the adapters beside it are tuned.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token, serving: eight groups of 32 experts, four of them kept, chosen by sigmoid plus bias
        dict(name="groups_token", op="route_groups", M=1, E=256, K=8, groups=8, top_groups=4, group_top=2, logits="f32",
             score="sigmoid", bias=True, renorm=True, scale=2.5, masked=False, stats=False),
        # a training step's tokens over the same experts, with padding and the balance loss
        dict(name="groups_train", op="route_groups", M=8192, E=256, K=8, groups=8, top_groups=4, group_top=2, logits="bf16",
             score="sigmoid", bias=True, renorm=True, scale=2.5, masked=True, stats=True),
        # an odd batch, groups of sixteen ranked by their best expert's softmax score
        dict(name="groups_odd", op="route_groups", M=1003, E=160, K=6, groups=10, top_groups=3, group_top=1, logits="f32",
             score="softmax", bias=False, renorm=False, scale=16.0, masked=True, stats=True),
        # one decoded token of one request: the smallest call, latency only
        dict(name="adapter_token", op="adapter", M=1, N=4096, K=4096, R=16, adapters=8, rows="mixed", x="bf16", base=True,
             hidden=False),
        # a batch of decoding requests, each row with an adapter of its own
        dict(name="adapter_decode", op="adapter", M=64, N=4096, K=7168, R=32, adapters=24, rows="mixed", x="bf16", base=True,
             hidden=False),
        # the prompts of several requests in one batch
        dict(name="adapter_prompts", op="adapter", M=4096, N=4096, K=7168, R=32, adapters=8, rows="segments", x="bf16",
             base=True, hidden=False),
        # a tuning step's forward in float32: odd rows and columns
        dict(name="adapter_odd", op="adapter", M=333, N=6147, K=4104, R=24, adapters=3, rows="segments", x="f32", base=True,
             hidden=True),
        # the backward pass of a tuning step with one adapter
        dict(name="adapter_tune", op="adapter_backward", M=8192, N=4096, K=4096, R=16, adapters=1, rows="segments", x="bf16",
             base=True),
        # the same for several adapters of higher rank that are tuned side by side
        dict(name="adapter_tune_many", op="adapter_backward", M=4096, N=1536, K=7168, R=64, adapters=4, rows="segments",
             x="bf16", base=True),
        # in float32, odd rows and columns
        dict(name="adapter_tune_odd", op="adapter_backward", M=1003, N=2049, K=1544, R=8, adapters=3, rows="mixed", x="f32",
             base=False),
        # a tuning step through a wide frozen projection: one large product
        dict(name="linear_tune", op="linear_backward", M=4096, N=14336, K=7168, group=128, affine=False, x="bf16",
             scales="bf16"),
        # a few rows in float32, rows and groups that end inside a tile
        dict(name="linear_tune_odd", op="linear_backward", M=77, N=6147, K=4104, group=32, affine=True, x="f32", scales="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number whose logarithm is uniform over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["route_groups", "adapter", "adapter", "adapter_backward", "linear_backward"])
    kind = rng.choice(["bf16", "f32"])
    if op == "route_groups":
        size = rng.choice([2, 4, 8, 12, 16, 20, 32, 64])         # experts of a group
        groups = rng.randint(2, max(2, min(32, 512 // size)))
        E, top = size * groups, rng.randint(1, groups)
        M = _spread(rng, 1, min(16384, (8192 * 256) // E))
        return dict(op=op, M=M, E=E, K=rng.randint(1, min(top * size, 12)), groups=groups, top_groups=top,
                    group_top=rng.choice([1, 2]), logits=kind, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    masked=rng.random() < 0.6, stats=rng.random() < 0.6)
    K = 8 * _spread(rng, 32, 1792)                               # 256 .. 14336
    if op == "linear_backward":
        N = _spread(rng, 64, min(65536, (1 << 29) // K))
        M = _spread(rng, 1, max(1, min(8192, (4096 * 14336 * 7168) // (N * K))))
        if kind == "f32":
            M = min(M, max(1, (1024 * 14336 * 7168) // (N * K)))
        return dict(op=op, M=M, N=N, K=K, group=rng.choice([32, 64, 128]), affine=rng.random() < 0.5, x=kind,
                    scales=rng.choice(["bf16", "f32"]))
    N = _spread(rng, 64, 14336)
    size = 4 if kind == "f32" else 2
    M = _spread(rng, 1, max(1, min(8192, (4096 * (4096 + 7168) * 2) // ((K + N) * size))))
    R = rng.choice([8, 16, 24, 32, 64, 128])
    adapters = _spread(rng, 1, max(1, min(64, 4096 // R)))
    case = dict(op=op, M=M, N=N, K=K, R=R, adapters=adapters, x=kind, base=rng.random() < 0.7,
                rows="mixed" if M <= 256 and rng.random() < 0.7 else "segments")
    if op == "adapter":
        case.update(hidden=rng.random() < 0.4)
    return case


def work(case):
    M = case["M"]
    if case["op"] == "route_groups":
        E, b = case["E"], 2 if case["logits"] == "bf16" else 4
        extra = (4 * E if case["bias"] else 0) + (M if case["masked"] else 0) + (8 * E + 4 if case["stats"] else 0)
        return {"bytes": M * E * b + M * case["K"] * 8 + extra, "flops": 6 * M * E}
    N, K, b = case["N"], case["K"], 2 if case["x"] == "bf16" else 4
    if case["op"] == "linear_backward":
        s = 2 if case["scales"] == "bf16" else 4
        groups = -(-K // case["group"]) * (2 if case["affine"] else 1)
        return {"bytes": N * K // 2 + N * groups * s + M * (N + K) * b, "flops": 2 * M * N * K}
    R, used = case["R"], min(M, case["adapters"])
    if case["op"] == "adapter":
        rows = K + N * (2 if case["base"] else 1)
        return {"bytes": M * rows * b + used * R * (K + N) * b + 4 * M + (4 * M * R if case["hidden"] else 0),
                "flops": 2 * M * R * (K + N)}
    rows = N + K * (3 if case["base"] else 2)
    return {"bytes": M * rows * b + used * R * (K + N) * b + case["adapters"] * R * (K + N) * 4 + 4 * M + 4 * M * R,
            "flops": 4 * M * R * (K + N)}


# --------------------------------------------------------------- the inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(M, N, kind, gen, scale=1.0):
    """Normal values [M, N] in that type, made in pieces."""
    out = torch.empty(M, N, dtype=_TYPES[kind], device="cuda")
    for at in range(0, M, 2048):
        part = out[at:at + 2048]
        part.copy_(scale * torch.randn(part.shape, device="cuda", generator=gen))
    return out


def _route_inputs(case, gen):
    M, E = case["M"], case["E"]
    logits = 1.5 * torch.randn(M, E, device="cuda", generator=gen) + 0.7 * torch.randn(1, E, device="cuda", generator=gen)
    state = dict(logits=logits.to(_TYPES[case["logits"]]), bias=None, mask=None)
    if case["bias"]:
        state["bias"] = 0.1 * torch.randn(E, device="cuda", generator=gen)
    if case["masked"]:
        # 1 for a token, 0 for padding: about one sixteenth of the batch, at random places
        state["mask"] = (torch.rand(M, device="cuda", generator=gen) > 1 / 16).to(torch.uint8)
    state["ids"] = torch.empty(M, case["K"], dtype=torch.int32, device="cuda")
    state["weights"] = torch.empty(M, case["K"], device="cuda")
    if case["stats"]:
        state["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        state["loss"], state["loss_grad"] = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
    return state


def _adapter_inputs(case, gen):
    M, N, K, R, n = (case[k] for k in ("M", "N", "K", "R", "adapters"))
    kind = case["x"]
    # -1: a request without an adapter
    ids = torch.randint(0, n, (M,), device="cuda", generator=gen)
    ids = torch.where(torch.rand(M, device="cuda", generator=gen) < (1 / 16 if M > 1 else 0), -1, ids)
    if case["rows"] == "segments":
        # the rows of a request stand together, the requests in any order
        order = torch.randperm(n + 1, device="cuda", generator=gen)
        ids = order[torch.sort(torch.argsort(order)[ids + 1])[0]] - 1
    state = dict(ids=ids.to(torch.int32), x=_rows(M, K, kind, gen))
    state["x"] *= 1 + 15 * (torch.rand(1, K, device="cuda", generator=gen) < 0.01)       # a few channels stand out
    state["a"] = _rows(n * R, K, kind, gen, K ** -0.5).view(n, R, K)
    state["b"] = _rows(n * N, R, kind, gen, 0.05).view(n, N, R)
    state["scales"] = 0.5 + 1.5 * torch.rand(n, device="cuda", generator=gen)
    if case["op"] == "adapter":
        state["base"] = _rows(M, N, kind, gen) if case["base"] else None
        state["out"] = torch.empty(M, N, dtype=_TYPES[kind], device="cuda")
        state["hidden"] = torch.empty(M, R, device="cuda") if case["hidden"] else None
    else:
        # what the forward pass left, and what came back: from the output, and through the projection itself
        state["hidden"] = _hidden(state["x"].float(), state["a"].float(), state["ids"])
        state["d_out"] = _rows(M, N, kind, gen, 1e-3)
        state["base"] = _rows(M, K, kind, gen, 1e-3) if case["base"] else None
        state["d_x"] = torch.empty(M, K, dtype=_TYPES[kind], device="cuda")
        state["d_a"], state["d_b"] = torch.empty(n, R, K, device="cuda"), torch.empty(n, N, R, device="cuda")
    return state


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
    state = dict(weights=weights, scales=scales, biases=None, d_out=_rows(M, N, case["x"], gen, 1e-3))
    if case["affine"]:
        state["biases"] = (-7.5 * scales.float() + 0.01 * torch.randn(N, groups, device="cuda", generator=gen)).to(kind)
    state["d_x"] = torch.empty(M, K, dtype=_TYPES[case["x"]], device="cuda")
    return state


_INPUTS = {"route_groups": _route_inputs, "adapter": _adapter_inputs, "adapter_backward": _adapter_inputs,
           "linear_backward": _linear_inputs}


def prepare(case, seed):
    state = _INPUTS[case["op"]](case, torch.Generator(device="cuda").manual_seed(seed))
    state["case"] = case
    if own:
        import quantized_moe_expert_q4_amd as q4
        from quantized_moe_expert_q4_amd.device import aligned_empty
        M = case["M"]
        if case["op"] == "route_groups":
            size = q4.route_workspace_bytes(M, case["E"]) if case["stats"] else 0
        elif case["op"] == "linear_backward":
            size = q4.linear_backward_workspace_bytes(M, case["N"], case["K"])
        else:
            size = q4.adapter_workspace_bytes(M, case["N"], case["K"], case["R"], case["adapters"])
        state["workspace_bytes"] = size
        state["workspace"] = aligned_empty(size, 256) if size else None
    return state


# ---------------------------------------------------------- the plain forms

def _scores(logits, score):
    """(score, probability) of every expert: the same for softmax; for sigmoid the probability sums to one."""
    if score == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        return p, p
    s = 1 / (1 + torch.exp(-logits))
    return s, s / s.sum(1, keepdim=True)


def _first(keys, count):
    """Indices of the highest keys of each row, ties to the lowest index; -1 in the place of -inf."""
    top, at = torch.sort(keys, dim=1, descending=True, stable=True)
    return torch.where(top[:, :count] == -math.inf, -1, at[:, :count])


def _choose_in_groups(logits, case, bias, mask):
    """The K best experts of the top_groups groups whose group_top best experts add up to most."""
    M, E, groups = case["M"], case["E"], case["groups"]
    # sums and values next to a border: in 64 bits
    keys = _scores(logits.double(), case["score"])[0]
    if bias is not None:
        keys = keys + bias.double()
    keys = torch.where(logits == -math.inf, -math.inf, keys)
    best = torch.sort(keys.view(M, groups, E // groups), dim=2, descending=True)[0][:, :, :case["group_top"]]
    some = best[:, :, 0] > -math.inf
    rank = torch.where(some, torch.where(best > -math.inf, best, 0.0).sum(2), -math.inf)
    kept = _first(rank, case["top_groups"])
    keep = torch.zeros(M, groups + 1, dtype=torch.bool, device=keys.device).scatter_(1, kept % (groups + 1), True)[:, :groups]
    # without a bias the logits order the experts, also where scores are equal in 64 bits
    order = keys if bias is not None else logits.double()
    ids = _first(torch.where(keep.repeat_interleave(E // groups, dim=1), order, -math.inf), case["K"])
    if mask is not None:
        ids = torch.where(mask.bool()[:, None], ids, -1)
    return ids.to(torch.int32)


def _route_groups_plain(st):
    case = st["case"]
    K, E = case["K"], case["E"]
    logits = st["logits"].float()
    score, prob = _scores(logits, case["score"])
    ids = _choose_in_groups(logits, case, st["bias"], st["mask"])
    chosen = ids >= 0
    at = ids.clamp(min=0).long()
    w = torch.where(chosen, torch.gather(score, 1, at), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    out = [ids, case["scale"] * w]
    if case["stats"]:
        counts = torch.zeros(E, dtype=torch.int32, device=ids.device)
        counts.index_add_(0, at.flatten(), chosen.flatten().to(torch.int32))
        there = chosen.any(1, keepdim=True)
        sums = torch.where(there, prob, 0.0).sum(0, dtype=torch.float64)
        tokens = there.sum().double()
        grad = torch.where(tokens > 0, E * counts.double() / (K * tokens * tokens), 0.0)
        out += [counts, (grad * sums).sum().float().view(1), grad.float()]
    return out


def _hidden(x, a, ids):
    """[M, R]: each row through the A of its own adapter, 0 without one; by one product with all of them."""
    n, R, K = a.shape
    every = (x @ a.reshape(n * R, K).t()).view(-1, n, R)
    mine = torch.gather(every, 1, ids.clamp(min=0).long().view(-1, 1, 1).expand(-1, 1, R))[:, 0]
    return torch.where((ids >= 0)[:, None], mine, 0.0)


def _spread_out(h, ids, n):
    """[M, n * R]: h in the columns of the row's own adapter, 0 in the others'."""
    mine = ids[:, None] == torch.arange(n, device=ids.device)
    return torch.where(mine[:, :, None], h[:, None, :], 0.0).view(h.shape[0], -1)


def _adapter_plain(st):
    a, b, ids = st["a"].float(), st["b"].float(), st["ids"]
    n, N, R = b.shape
    h = _hidden(st["x"].float(), a, ids)
    scale = st["scales"][ids.clamp(min=0).long()][:, None]
    out = _spread_out(h * scale, ids, n) @ b.transpose(1, 2).reshape(n * R, N)
    if st["base"] is not None:
        out = out + st["base"].float()
    out = out.to(st["x"].dtype)
    return [out] if st["hidden"] is None else [out, h]


def _adapter_backward_plain(st):
    a, b, ids, x, d = st["a"].float(), st["b"].float(), st["ids"], st["x"].float(), st["d_out"].float()
    n, N, R = b.shape
    d = d * st["scales"][ids.clamp(min=0).long()][:, None]
    g = _spread_out(_hidden(d, b.transpose(1, 2), ids), ids, n)
    d_x = g @ a.reshape(n * R, -1)
    if st["base"] is not None:
        d_x = d_x + st["base"].float()
    d_a = (g.t() @ x).view(n, R, -1)
    d_b = (_spread_out(st["hidden"], ids, n).t() @ d).view(n, R, N).transpose(1, 2).contiguous()
    return [d_x.to(st["x"].dtype), d_a, d_b]


def _linear_backward_plain(st):
    case = st["case"]
    N, K, G = case["N"], case["K"], case["group"]
    q = torch.stack((st["weights"] & 15, st["weights"] >> 4), dim=2).view(N, K).float()
    wide = lambda t: t.float().repeat_interleave(G, dim=1)[:, :K]
    if st["biases"] is None:
        w = (q - 8) * wide(st["scales"])
    else:
        w = q * wide(st["scales"]) + wide(st["biases"])
    return (st["d_out"].float() @ w).to(st["d_out"].dtype)


_PLAIN = {"route_groups": _route_groups_plain, "adapter": _adapter_plain, "adapter_backward": _adapter_backward_plain,
          "linear_backward": _linear_backward_plain}


# ------------------------------------------------------- the library's calls

def _library(st):
    import quantized_moe_expert_q4_amd as q4
    case = st["case"]
    op, M = case["op"], case["M"]
    if op == "route_groups":
        K = case["K"]
        stats = {k: st[k] for k in ("counts", "loss", "loss_grad", "workspace", "workspace_bytes")} if case["stats"] else {}
        q4.route_groups(st["logits"], M, case["E"], K, case["groups"], case["top_groups"], st["ids"], st["weights"],
                        group_top=case["group_top"], score=case["score"], renormalize=case["renorm"], scale=case["scale"],
                        select_bias=st["bias"], token_mask=st["mask"], xdtype=case["logits"], **stats)
        return [st["ids"], st["weights"]] + [st[k] for k in ("counts", "loss", "loss_grad") if case["stats"]]
    N, K, kind, space = case["N"], case["K"], case["x"], (st["workspace"], st["workspace_bytes"])
    if op == "linear_backward":
        q4.linear_backward(st["weights"], st["scales"], st["d_out"], M, N, K, case["group"], st["d_x"], *space,
                           biases=st["biases"], xdtype=kind)
        return st["d_x"]
    R, n = case["R"], case["adapters"]
    if op == "adapter":
        q4.adapter(st["a"], st["b"], st["x"], M, N, K, R, n, st["out"], *space, adapter_ids=st["ids"], scales=st["scales"],
                   base=st["base"], hidden=st["hidden"], xdtype=kind)
        return [st["out"]] if st["hidden"] is None else [st["out"], st["hidden"]]
    q4.adapter_backward(st["d_out"], st["a"], st["b"], M, N, K, R, n, *space, x=st["x"], hidden=st["hidden"], d_x=st["d_x"],
                        d_a=st["d_a"], d_b=st["d_b"], adapter_ids=st["ids"], scales=st["scales"], base=st["base"],
                        xdtype=kind)
    return [st["d_x"], st["d_a"], st["d_b"]]


def run(state):
    return _library(state) if own else _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------- the definitions in 64 bits

def _exact_score(logits, score):
    logits = logits.double()
    if score == "sigmoid":
        s = torch.exp(-torch.log1p(torch.exp(-logits.abs())) + logits.clamp(max=0))
        return s, s / s.sum(1, keepdim=True)
    p = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True))
    return p, p


def _take_best(keys):
    """(best key, its lowest index) of each row, which is then struck out."""
    index = torch.arange(keys.shape[1], device=keys.device)
    best = keys.amax(1, keepdim=True)
    at = torch.where(keys == best, index, keys.shape[1]).amin(1, keepdim=True)
    keys.scatter_(1, at, -math.inf)
    return best, at


def _exact_groups(keys, groups, group_top, top_groups):
    """bool [M, E]: the experts of the kept groups."""
    M, E = keys.shape
    size = E // groups
    rank = torch.empty(M, groups, dtype=torch.float64, device=keys.device)
    for g in range(groups):
        part = keys[:, g * size:(g + 1) * size].clone()
        best, _ = _take_best(part)
        rank[:, g] = best[:, 0]
        if group_top == 2 and size > 1:
            second, _ = _take_best(part)
            rank[:, g] += torch.where(second > -math.inf, second, 0.0)[:, 0]
    keep = torch.zeros(M, E, dtype=torch.bool, device=keys.device)
    inside = torch.arange(size, device=keys.device)
    for _ in range(top_groups):
        best, at = _take_best(rank)
        keep.scatter_(1, at * size + inside, (best > -math.inf).expand(M, size))
    return keep


def _exact_route_groups(st):
    case = st["case"]
    E, K = case["E"], case["K"]
    score, prob = _exact_score(st["logits"], case["score"])
    keys = score if st["bias"] is None else score + st["bias"].double()
    keys = torch.where(st["logits"] == -math.inf, -math.inf, keys)
    keep = _exact_groups(keys, case["groups"], case["group_top"], case["top_groups"])
    left = torch.where(keep, st["logits"].double() if st["bias"] is None else keys, -math.inf)
    ids = []
    for _ in range(K):
        best, at = _take_best(left)
        ids.append(torch.where(best > -math.inf, at, -1))
    ids = torch.cat(ids, 1)
    if st["mask"] is not None:
        ids[st["mask"] == 0] = -1
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
        there = ids[:, 0] >= 0
        tokens = float(there.sum())
        share = counts / (K * tokens) if tokens else 0 * counts
        mean = prob[there].sum(0) / tokens if tokens else 0 * counts
        out += [counts.to(torch.int32), (E * (share * mean).sum()).view(1), E * share / max(tokens, 1.0)]
    return out


def _exact_adapter(st):
    case = st["case"]
    out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    if st["base"] is not None:
        out += st["base"].double()
    hidden = torch.zeros(case["M"], case["R"], dtype=torch.float64, device="cuda")
    for i in range(case["adapters"]):
        at = (st["ids"] == i).nonzero()[:, 0]
        hidden[at] = torch.mm(st["x"][at].double(), st["a"][i].double().t())
        out[at] += st["scales"][i].double() * torch.mm(hidden[at], st["b"][i].double().t())
    return [out] if st["hidden"] is None else [out, hidden]


def _exact_adapter_backward(st):
    case = st["case"]
    d_x = torch.zeros(case["M"], case["K"], dtype=torch.float64, device="cuda")
    if st["base"] is not None:
        d_x += st["base"].double()
    d_a = torch.zeros(st["a"].shape, dtype=torch.float64, device="cuda")
    d_b = torch.zeros(st["b"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["adapters"]):
        at = (st["ids"] == i).nonzero()[:, 0]
        d, s = st["d_out"][at].double(), st["scales"][i].double()
        g = s * torch.mm(d, st["b"][i].double())
        d_x[at] += torch.mm(g, st["a"][i].double())
        d_a[i] = torch.mm(g.t(), st["x"][at].double())
        d_b[i] = s * torch.mm(d.t(), st["hidden"][at].double())
    return [d_x, d_a, d_b]


def _exact_linear_backward(st):
    case = st["case"]
    N, K, G = case["N"], case["K"], case["group"]
    out = torch.zeros(case["M"], K, dtype=torch.float64, device="cuda")
    at = torch.arange(K, device="cuda")
    for lo in range(0, N, 4096):
        byte = st["weights"][lo:lo + 4096].index_select(1, at // 2).int()
        q = torch.bitwise_right_shift(byte, (4 * (at % 2)).int()).bitwise_and(15).double()
        s = st["scales"][lo:lo + 4096].double().index_select(1, at // G)
        off = -8 * s if st["biases"] is None else st["biases"][lo:lo + 4096].double().index_select(1, at // G)
        out.addmm_(st["d_out"][:, lo:lo + 4096].double(), torch.addcmul(off, q, s))
    return out


_EXACT = {"route_groups": _exact_route_groups, "adapter": _exact_adapter, "adapter_backward": _exact_adapter_backward,
          "linear_backward": _exact_linear_backward}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
