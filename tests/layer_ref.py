"""Plain 64-bit forms of the router gate, its losses and gradient, and of the
experts' products with 4-bit weights, written token by token and expert by
expert from the definitions in include/ep.h."""

import numpy as np

EPS = 2.0 ** -24      # one fp32 rounding


def scores(l, score):
    """(s, p, lse) of one token's logits: scores, their share, log sum exp."""
    dead = np.isneginf(l)
    if dead.all():
        z = np.zeros_like(l)
        return z, z, 0.0
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(dead, 0.0, 1.0 / (1.0 + np.exp(-l)))
        return s, s / s.sum() if s.sum() > 0 else s, 0.0
    m = l.max()
    e = np.exp(l - m)
    return e / e.sum(), e / e.sum(), m + np.log(e.sum())


def choose(l, K, score, bias, groups, kept):
    """Experts of one token in order, -1 where none is left."""
    E = len(l)
    s, _, _ = scores(np.where(np.isnan(l), -np.inf, l), score)
    c = l.copy() if score == "softmax" else s + (0.0 if bias is None else bias)
    c = np.where(np.isneginf(l) | np.isnan(l), -np.inf, c)
    if kept < groups:
        per = E // groups
        rank = []
        for g in range(groups):
            top = sorted(c[g * per:(g + 1) * per], reverse=True)[:2]
            v = top[0]
            if score == "sigmoid" and len(top) > 1 and np.isfinite(top[1]):
                v = v + top[1]
            rank.append((-v, g))
        keep = {g for _, g in sorted(rank)[:kept]}
        c = np.array([c[e] if e // per in keep else -np.inf for e in range(E)])
    order = sorted(range(E), key=lambda e: (-c[e], e))[:K]
    return [e if c[e] > -np.inf else -1 for e in order]


def route(l, K, score="softmax", bias=None, groups=1, kept=1, renorm=True, scale=1.0, mask=None):
    T = len(l)
    idx, w = np.full((T, K), -1, np.int64), np.zeros((T, K))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        idx[t] = choose(l[t], K, score, bias, groups, kept)
        s, _, _ = scores(l[t], score)
        w[t] = [s[e] if e >= 0 else 0.0 for e in idx[t]]
        if renorm:
            w[t] = w[t] / w[t].sum() if w[t].sum() != 0 else 0.0
    return idx, w * scale


def balance(l, idx, score, mask, starts):
    """(count, prob, seq_tokens, loss) for given choices."""
    T, E = l.shape
    K, B = idx.shape[1], len(starts) - 1
    count, prob, n = np.zeros((B, E), np.int64), np.zeros((B, E)), np.zeros(B, np.int64)
    z = 0.0
    for b in range(B):
        for t in range(starts[b], starts[b + 1]):
            if mask is not None and not mask[t]:
                continue
            n[b] += 1
            _, p, lse = scores(l[t], score)
            prob[b] += p
            z += lse * lse
            for e in idx[t]:
                if e >= 0:
                    count[b, e] += 1
        prob[b] /= max(1, n[b])
    full = n > 0
    terms = [(count[b] * E / (K * n[b]) * prob[b]).sum() for b in range(B) if full[b]]
    loss = np.array([np.mean(terms) if terms else 0.0, z / max(1, n.sum())])
    return count, prob, np.concatenate([n, [n.sum(), full.sum()]]), loss


def objective(l, idx, gw, gl, score, renorm, scale, mask, starts, count):
    """sum gw w + gl . loss with the choice and the counts held constant."""
    T, E = l.shape
    K, B = idx.shape[1], len(starts) - 1
    valid = [t for t in range(T) if mask is None or mask[t]]
    n = [sum(1 for t in valid if starts[b] <= t < starts[b + 1]) for b in range(B)]
    full = max(1, sum(1 for v in n if v))
    total = 0.0
    for t in valid:
        s, p, lse = scores(l[t], score)
        sel = [(k, e) for k, e in enumerate(idx[t]) if e >= 0]
        S = sum(s[e] for _, e in sel) if renorm else 1.0
        total += sum(gw[t, k] * scale * s[e] / S for k, e in sel if S != 0)
        b = next(b for b in range(B) if starts[b] <= t < starts[b + 1])
        total += gl[0] * (count[b] * E / (K * n[b]) * p).sum() / n[b] / full
        total += gl[1] * lse * lse / len(valid)
    return total


def backward(l, idx, gw, gl, score, renorm, scale, mask, starts, count):
    """(gradient, the sum of its terms' magnitudes) by the logits."""
    T, E = l.shape
    K, B = idx.shape[1], len(starts) - 1
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    valid = [t for t in range(T) if mask is None or mask[t]]
    n = [sum(1 for t in valid if starts[b] <= t < starts[b + 1]) for b in range(B)]
    full = max(1, sum(1 for v in n if v))
    for t in valid:
        s, p, lse = scores(l[t], score)
        b = next(b for b in range(B) if starts[b] <= t < starts[b + 1])
        dq = gl[0] * count[b] * E / (K * n[b] ** 2 * full)
        ds, mag = np.zeros(E), np.zeros(E)
        sel = [(k, e) for k, e in enumerate(idx[t]) if e >= 0]
        S = sum(s[e] for _, e in sel)
        mean = sum(gw[t, k] * s[e] for k, e in sel) / S if S else 0.0
        amean = sum(abs(gw[t, k]) * s[e] for k, e in sel) / S if S else 0.0
        for k, e in sel:
            if renorm:
                ds[e] = scale * (gw[t, k] - mean) / S if S else 0.0
                mag[e] = abs(scale) * (abs(gw[t, k]) + amean) / S if S else 0.0
            else:
                ds[e], mag[e] = scale * gw[t, k], abs(scale * gw[t, k])
        if score == "sigmoid":
            tot = s.sum() or 1.0
            grad[t] = ((dq - (p * dq).sum()) / tot + ds) * s * (1 - s)
            size[t] = ((abs(dq) + (p * abs(dq)).sum()) / tot + mag) * s
        else:
            dz = gl[1] * 2 * lse / len(valid)
            g = dq + ds
            grad[t] = p * (g - (p * g).sum() + dz)
            a = abs(dq) + mag
            size[t] = p * (a + (p * a).sum() + abs(dz))
    return grad, size


def w4_matrix(codes, scales, zeros, group):
    """W [N, H] of one expert from codes [N, H / 2], scales and zeros [N, H / group]."""
    q = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).astype(np.float64)
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, 1)
    return (q - z) * np.repeat(scales.astype(np.float64), group, 1)


def w4(x, W, gated):
    """(y, a bound of its error in fp32 with exact products) of rows x [m, H]."""
    H = x.shape[1]
    a = x @ W.T
    # a rounding a sum of 16 products and one a group, each at most of the
    # terms' magnitudes, with the tensor core's two bits fewer
    da = 4 * EPS * (H / 16 + 8) * (abs(x) @ abs(W).T)
    if not gated:
        return a, da
    half = W.shape[0] // 2
    gate, up, dg, du = a[:, :half], a[:, half:], da[:, :half], da[:, half:]
    with np.errstate(over="ignore"):
        act = gate / (1 + np.exp(-gate))
    # |silu'| <= 1.1; expf, the sum, the quotient and the product round too
    y = act * up
    return y, 1.1 * dg * (abs(up) + du) + abs(act) * du + 16 * EPS * (1 + abs(gate)) * abs(y)
