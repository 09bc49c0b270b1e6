"""Plain 64-bit forms of the layer operators (numpy), written from their
definitions in include/q4moe.h, with the magnitudes the tolerances scale with."""
import numpy as np

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # rounding of one value, relative


def unpack_q4(weights, N, K):
    """uint8 [N, K/2] -> integer nibbles [N, K]; byte b of a row holds weights 2b (low) and 2b + 1."""
    w = np.asarray(weights, np.uint8).reshape(N, K // 2)
    q = np.empty((N, K), np.int64)
    q[:, 0::2] = w & 15
    q[:, 1::2] = w >> 4
    return q


def linear(weights, scales, biases, group, x, N, K):
    """(out [M, N], magnitude [M, N]): the magnitude is sum_k (31 + 24) s |x| +
    |b| |x|, which bounds every partial sum of the group sums the kernels form
    from 16 + q and its offset."""
    q = unpack_q4(weights, N, K).astype(np.float64)
    wide = lambda a: np.repeat(np.asarray(a, np.float64), group, axis=1)[:, :K]
    s = wide(scales)
    if biases is None:
        W, mag = s * (q - 8), 55 * np.abs(s)
    else:
        W, mag = s * q + wide(biases), 55 * np.abs(s) + np.abs(wide(biases))
    x = np.asarray(x, np.float64)
    return x @ W.T, np.abs(x) @ mag.T


def scores(logits, score):
    """(score, probability) of [E] logits."""
    l = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax":
            e = np.exp(l - l.max())
            return e / e.sum(), e / e.sum()
        s = 1.0 / (1.0 + np.exp(-l))
        total = s.sum()
        return s, (s / total if total else np.zeros_like(s))


def route(logits, K, score, renormalize=False, scale=1.0, bias=None, mask=None):
    """ids [M, K], weights [M, K], counts [E], loss, loss_grad [E], by a loop over tokens."""
    M, E = logits.shape
    ids = np.full((M, K), -1, np.int64)
    weights = np.zeros((M, K))
    counts = np.zeros(E, np.int64)
    sums = np.zeros(E)
    tokens = 0
    for t in range(M):
        l = np.asarray(logits[t], np.float64)
        if (mask is not None and not mask[t]) or np.all(l == -np.inf):
            continue
        s, p = scores(l, score)
        key = l.copy() if bias is None else np.where(l == -np.inf, -np.inf, s + np.asarray(bias, np.float64))
        rank = np.where(np.isnan(key), np.inf, key)
        order = sorted(range(E), key=lambda e: (not np.isnan(key[e]), -rank[e], e))
        chosen = [e for e in order[:K] if rank[e] > -np.inf]
        w = s[chosen]
        if renormalize:
            w = w / w.sum() if w.sum() != 0 else 0 * w
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = scale * w
        counts[chosen] += 1
        sums += p
        tokens += 1
    grad = E * counts / (K * float(tokens) ** 2) if tokens else np.zeros(E)
    return ids, weights, counts, float((grad * sums).sum()), grad


def route_objective(logits, ids, score, renormalize, scale, d_weights, d_loss, loss_grad):
    """sum(d_weights * weights) + d_loss * sum_t <loss_grad, p_t> for fixed ids: its gradient is the backward pass."""
    total = 0.0
    for t in range(logits.shape[0]):
        if ids[t, 0] < 0:
            continue
        s, p = scores(logits[t], score)
        on = (ids[t] >= 0) & (ids[t] < logits.shape[1])
        picked = np.where(on, s[np.where(on, ids[t], 0)], 0.0)
        if renormalize:
            picked = picked / picked.sum() if picked.sum() else 0 * picked
        total += scale * float((np.where(on, d_weights[t], 0.0) * picked).sum()) + d_loss * float((loss_grad * p).sum())
    return total


def route_backward(logits, ids, score, renormalize, scale, d_weights, d_loss, loss_grad):
    """(d_logits, magnitude): the magnitude is the same sum with every term's absolute value."""
    M, E = logits.shape
    out, mag = np.zeros((M, E)), np.zeros((M, E))
    for t in range(M):
        if ids[t, 0] < 0:
            continue
        s, p = scores(logits[t], score)
        g, ga = np.zeros(E), np.zeros(E)
        on = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        S = sum(s[e] for _, e in on)
        mean = sum(scale * d_weights[t, j] * s[e] for j, e in on)
        mean_abs = sum(abs(scale * d_weights[t, j]) * s[e] for j, e in on)
        for j, e in on:
            dw = scale * d_weights[t, j]
            if renormalize:
                g[e] += (dw - mean / S) / S if S else 0.0
                ga[e] += (abs(dw) + mean_abs / S) / S if S else 0.0
            else:
                g[e] += dw
                ga[e] += abs(dw)
        gl = d_loss * np.asarray(loss_grad, np.float64)
        gla = np.abs(gl)
        if score == "softmax":
            out[t] = s * (g + gl - (s * (g + gl)).sum())
            mag[t] = s * (ga + gla + (s * (ga + gla)).sum())
        else:
            q = 1.0 / (1.0 + np.exp(np.asarray(logits[t], np.float64)))
            total = s.sum()
            inv = 1.0 / total if total else 0.0
            out[t] = s * q * (g + (gl - (p * gl).sum()) * inv)
            mag[t] = s * q * (ga + (gla + (p * gla).sum()) * inv)
    return out, mag


def combine(y, weights, ids, num_slots, base):
    """(out [M, H], magnitude)."""
    live = np.ones(weights.shape, bool) if ids is None else (ids >= 0) & (ids < num_slots)
    w = np.where(live, np.asarray(weights, np.float64), 0.0)[:, :, None]
    rows = np.where(live[:, :, None], np.asarray(y, np.float64), 0.0)
    b = 0.0 if base is None else np.asarray(base, np.float64)
    return (w * rows).sum(1) + b, np.abs(w * rows).sum(1) + np.abs(b)


def combine_backward(d_out, y, weights, ids, num_slots):
    """(d_y, d_weights, magnitude of d_weights)."""
    live = np.ones(weights.shape, bool) if ids is None else (ids >= 0) & (ids < num_slots)
    d = np.asarray(d_out, np.float64)[:, None, :]
    w = np.where(live, np.asarray(weights, np.float64), 0.0)[:, :, None]
    rows = np.where(live[:, :, None], np.asarray(y, np.float64), 0.0)
    return w * d, (rows * d).sum(2), np.abs(rows * d).sum(2)
