"""Plain 64-bit forms (numpy) of the router over groups, the adapters and the
linear's gradient, written from their definitions in include/q4moe.h, with the
magnitudes the tolerances scale with."""
import numpy as np

import layer_reference as ref


def kept_groups(logits, groups, top_groups, group_top, score, bias):
    """The kept groups of one token's logits [E], in 64 bits."""
    l = np.asarray(logits, np.float64)
    E = l.size
    if bias is None and group_top == 1:
        key = l.copy()
    else:
        s, _ = ref.scores(l, score)
        key = s + (0.0 if bias is None else np.asarray(bias, np.float64))
    key = np.where(l == -np.inf, -np.inf, key)
    rank = []
    for g in range(groups):
        part = key[g * (E // groups):(g + 1) * (E // groups)]
        part = sorted((v for v in part if not v == -np.inf), key=lambda v: (not np.isnan(v), -v))[:group_top]
        rank.append((sum(part), g) if part else None)
    order = sorted((r for r in rank if r is not None), key=lambda r: (not np.isnan(r[0]), -r[0], r[1]))
    return [g for _, g in order[:top_groups]]


def route_groups(logits, K, groups, top_groups, group_top, score, renormalize=False, scale=1.0, bias=None, mask=None):
    """As layer_reference.route: the experts of the other groups are left out of
    the choice (their logits taken as -inf there), not out of the scores."""
    M, E = logits.shape
    ids = np.full((M, K), -1, np.int64)
    weights, counts, sums, tokens = np.zeros((M, K)), np.zeros(E, np.int64), np.zeros(E), 0
    size = E // groups
    for t in range(M):
        l = np.asarray(logits[t], np.float64)
        if (mask is not None and not mask[t]) or np.all(l == -np.inf):
            continue
        s, p = ref.scores(l, score)
        key = l if bias is None else np.where(l == -np.inf, -np.inf, s + np.asarray(bias, np.float64))
        keep = kept_groups(l, groups, top_groups, group_top, score, bias)
        left = [e for g in sorted(keep) for e in range(g * size, (g + 1) * size) if not key[e] == -np.inf]
        chosen = sorted(left, key=lambda e: (not np.isnan(key[e]), -key[e], e))[:K]
        if not chosen:
            continue
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


def dense_weights(weights, scales, biases, group, N, K):
    """W [N, K] in 64 bits."""
    q = ref.unpack_q4(weights, N, K).astype(np.float64)
    wide = lambda a: np.repeat(np.asarray(a, np.float64), group, axis=1)[:, :K]
    return wide(scales) * (q - 8) if biases is None else wide(scales) * q + wide(biases)


def linear_backward(weights, scales, biases, group, d_out, N, K):
    """(d_x [M, K], magnitude [M, K])."""
    W = dense_weights(weights, scales, biases, group, N, K)
    d = np.asarray(d_out, np.float64)
    return d @ W, np.abs(d) @ np.abs(W)


def adapter(a, b, x, ids, scales, base):
    """(out [M, N], its magnitude, hidden [M, R], its magnitude); scales and base are arrays."""
    M, (n, N, R) = x.shape[0], b.shape
    out, mag = np.array(base, np.float64), np.abs(np.array(base, np.float64))
    h, hm = np.zeros((M, R)), np.zeros((M, R))
    for t in range(M):
        i = ids[t]
        if 0 <= i < n:
            h[t], hm[t] = a[i] @ x[t], np.abs(a[i]) @ np.abs(x[t])
            out[t] += scales[i] * (b[i] @ h[t])
            mag[t] += abs(scales[i]) * (np.abs(b[i]) @ hm[t])
    return out, mag, h, hm


def adapter_backward(d_out, a, b, x, hidden, ids, scales, base):
    """((d_x, d_a, d_b), their magnitudes)."""
    n, N, R = b.shape
    d_x, mx = np.array(base, np.float64), np.abs(np.array(base, np.float64))
    d_a, ma, d_b, mb = np.zeros(a.shape), np.zeros(a.shape), np.zeros(b.shape), np.zeros(b.shape)
    for i in range(n):
        t = np.flatnonzero(np.asarray(ids) == i)
        d, s = d_out[t], scales[i]
        g, gm = s * (d @ b[i]), abs(s) * (np.abs(d) @ np.abs(b[i]))
        d_x[t] += g @ a[i]
        mx[t] += gm @ np.abs(a[i])
        d_a[i], ma[i] = g.T @ x[t], gm.T @ np.abs(x[t])
        d_b[i], mb[i] = s * (d.T @ hidden[t]), abs(s) * (np.abs(d).T @ np.abs(hidden[t]))
    return (d_x, d_a, d_b), (mx, ma, mb)
