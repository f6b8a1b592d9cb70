"""Plain 64-bit forms of the gate and the adapters on the CPU (numpy), row by row from the
formulas in include/dg.h, with the error bounds that the fp32 kernels are held to."""
import math

import numpy as np

U = 2.0 ** -24            # unit rounding of fp32


def scores(z, score):
    """(s, 1 - s, p) of one row in 64 bits; a row of -inf only has none."""
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = z.max() if z.size else -math.inf
            if m == -math.inf:
                return np.zeros_like(z), None, np.zeros_like(z)
            e = np.exp(z - m)
            s = e / e.sum()
            return s, None, s
        s = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        c = np.where(z >= 0, np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))), 1 / (1 + np.exp(-np.abs(z))))
        return s, c, s / s.sum() if s.sum() > 0 else np.zeros_like(s)


def choose(z32, bias, k):
    """The k experts by decreasing fp32 key, equal keys by increasing index, -1 past them."""
    with np.errstate(all="ignore"):
        key = z32.astype(np.float32) + (np.float32(0) if bias is None else bias.astype(np.float32))
    ids = []
    left = [e for e in range(len(key)) if key[e] > -math.inf]
    for _ in range(k):
        best = -1
        for e in left:
            if best < 0 or key[e] > key[best]:
                best = e
        ids.append(best)
        if best >= 0:
            left.remove(best)
    return ids


def route(logits, k, bias, valid, score, normalize, scale, balance):
    """logits: T x E float32 (what the dtype holds).  ids, weights, counts, loss, coef."""
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    counts = np.zeros(E, np.int64)
    psum = np.zeros(E)
    live = [t for t in range(T) if valid is None or valid[t]]
    for t in live:
        s, _, p = scores(logits[t].astype(np.float64), score)
        ids[t] = choose(logits[t], bias, k)
        ok = ids[t] >= 0
        w = np.where(ok, s[ids[t]], 0.0)
        with np.errstate(all="ignore"):
            if normalize:
                w = w / w.sum() if w.sum() != 0 else 0 * w
        weights[t] = scale * w
        np.add.at(counts, ids[t][ok], 1)
        psum += p
    if not live:
        return ids, weights, counts, 0.0, np.zeros(E)
    coef = balance * E * counts / (k * float(len(live)) ** 2)
    return ids, weights, counts, float(coef @ psum), coef


def route_loss(z, ids, gw, coef, gl, score, normalize, scale):
    """One row's part of sum(gw * weights) + gl * loss, choice and coef held constant."""
    s, _, p = scores(z, score)
    ok = ids >= 0
    w = np.where(ok, s[ids], 0.0)
    if normalize and w.sum() != 0:
        w = w / w.sum()
    return scale * float((np.where(ok, gw, 0.0) * w).sum()) + gl * float(coef @ p)


def route_grad(logits, ids, gw, coef, gl, valid, score, normalize, scale):
    """The gradient by the logits, and the size of what cancels in each element."""
    T, E = logits.shape
    dz, size = np.zeros((T, E)), np.zeros((T, E))
    u = gl * coef if coef is not None else np.zeros(E)
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        z = logits[t].astype(np.float64)
        s, c, p = scores(z, score)
        d, dm = np.zeros(E), np.zeros(E)
        if gw is not None:
            ok = ids[t] >= 0
            i, g = ids[t][ok], scale * gw[t][ok].astype(np.float64)
            tot = s[i].sum()
            if normalize:
                inv = 1 / tot if tot > 0 else 0.0
                mean = (g * s[i]).sum() * inv
                d[i], dm[i] = (g - mean) * inv, (np.abs(g) + (np.abs(g) * s[i]).sum() * inv) * inv
            else:
                d[i], dm[i] = g, np.abs(g)
        if score == "softmax":
            g, gm = u + d, np.abs(u) + dm
            dz[t], size[t] = s * (g - (g * s).sum()), s * (gm + (gm * s).sum())
        else:
            inv = 1 / s.sum() if s.sum() > 0 else 0.0
            g = (u - (u * p).sum()) * inv + d
            gm = (np.abs(u) + (np.abs(u) * p).sum()) * inv + dm
            dz[t], size[t] = g * s * c, gm * s * c
    return dz, size


def spread(logits):
    """The largest distance of a logit from its row's maximum or from zero: what the
    rounding of exp's argument is proportional to (past 104 exp has nothing left in fp32)."""
    f = logits[np.isfinite(logits)].astype(np.float64)
    return min(float(2 * np.abs(f).max()), 208.0) if f.size else 0.0


def weight_tolerance(logits, E):
    """Relative: exp's argument rounded (spread), exp, a sum of E terms of which a lane
    adds at most 16 and the lanes are added in pairs, the division, the row's sum and its
    division, the factor; twice over."""
    return 2 * U * (spread(logits) + 2 + 16 + math.log2(max(E, 2)) + 2 + 5 + 2)


def lora(x, A, B, ids, scales, ranks, base):
    """The result in 64 bits and the sum of the magnitudes that it is made of."""
    T, N = len(x), B.shape[1]
    out = np.zeros((T, N)) if base is None else base.astype(np.float64)
    size = np.zeros((T, N))
    L, R = A.shape[:2]
    for t in range(T):
        i = int(ids[t])
        if not 0 <= i < L:
            continue
        r = R if ranks is None else min(max(int(ranks[i]), 0), R)
        a, b = A[i, :r].astype(np.float64), B[i, :, :r].astype(np.float64)
        s = 1.0 if scales is None else float(scales[i])
        xt = x[t].astype(np.float64)
        out[t] += s * (b @ (a @ xt))
        size[t] += abs(s) * (np.abs(b) @ (np.abs(a) @ np.abs(xt)))
    return out, size


def lora_tolerance(ref, size, K):
    """One rounding to bf16 (2^-9 of the result, doubled); the inner product as two bf16
    numbers (2^-18, doubled); fp32 sums of K and of R terms, 32 to an instruction."""
    return 2.0 ** -8 * np.abs(ref) + size * (2.0 ** -17 + 2 * U * (K / 32 + 64)) + 1e-37
