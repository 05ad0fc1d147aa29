"""Plain 64-bit references of the residual norm, the routing and the products with 4-bit weights."""

import numpy as np

from attn_ref import e2m1_values, e4m3_values
from oracle import mx_oracle as O


def act_values(codes, sf):
    """codes [T, K], sf [T, ceil(K/128)] -> [T, K] float64 (scale byte 255: NaN)."""
    s = np.where(sf == 255, np.nan, np.exp2(sf.astype(np.float64) - 127))
    return e4m3_values(codes) * np.repeat(s, 128, axis=1)[:, :codes.shape[1]]


def weight_values(codes, sf):
    return e2m1_values(codes, sf)


def norm(s, weight, eps):
    """s [T, D], weight [D] or None, float64 -> y."""
    y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    return y if weight is None else y * weight


def scores(logits, scoring):
    """float64 scores; masked logits (-inf, NaN) count for nothing."""
    l = np.where(np.isnan(logits), -np.inf, np.minimum(logits, 3.4028234663852886e38))
    with np.errstate(all="ignore"):
        if scoring == "softmax":
            m = np.max(l, axis=1, keepdims=True)
            e = np.exp(l - np.where(np.isfinite(m), m, 0.0))
            return e / np.maximum(e.sum(1, keepdims=True), 1e-300)
        if scoring == "sigmoid":
            return 1 / (1 + np.exp(-l))
        return np.sqrt(np.maximum(l, 0) + np.log1p(np.exp(-np.abs(l))))


def _undecided(values, keys):
    """Whether neighbours among the descending `values` are nearer than 64-bit scores tell: an exponential or a
    logarithm is off by an ulp or two (2^-51), the quotient, the root and the sums of two by half of one each, a
    softmax's denominator of up to 1024 terms by 2^-47 at most: below 2^-46 of the value (nothing of a score that is
    zero).  Equal keys (the numbers that the value is computed from) give equal values in any arithmetic."""
    return any(a - b < 2.0 ** -46 * (abs(a) + abs(b)) and p != q
               for a, b, p, q in zip(values, values[1:], keys, keys[1:]))


def route(logits, k, scoring, bias=None, groups=1, topk_groups=1, group_top=2, renormalise=True, scale=1.0):
    """logits [T, E] float64 -> (ids [T, k], weights [T, k], sure [T]: the rows whose choice 64-bit scores
    decide)."""
    T, E = logits.shape
    n = E // groups
    p = scores(logits, scoring)
    shut = np.isnan(logits) | (logits == -np.inf)
    b = np.zeros(E)
    if bias is not None:
        shut = shut | (np.isnan(bias) | (bias == -np.inf))[None]
        b = np.minimum(np.where(np.isfinite(bias) | (bias > 0), bias, 0.0), np.float32(1e30).astype(np.float64))
    c = p + b
    ids, w, sure = np.full((T, k), -1, np.int64), np.zeros((T, k)), np.ones(T, bool)
    for t in range(T):
        open_ = [e for e in range(E) if not shut[t, e]]
        if topk_groups < groups:
            best = []
            for g in range(groups):
                v = sorted(((c[t, e], logits[t, e], b[e]) for e in open_ if e // n == g), reverse=True)[:group_top]
                if v:
                    best.append((-sum(x[0] for x in v), g, [x[1:] for x in v]))
            best.sort(key=lambda x: x[:2])
            edge = best[topk_groups - 1:topk_groups + 1]
            sure[t] &= not _undecided([-x[0] for x in edge], [x[2] for x in edge])
            kept = {x[1] for x in best[:topk_groups]}
            open_ = [e for e in open_ if e // n in kept]
        order = logits[t] if bias is None else c[t]
        pick = sorted(open_, key=lambda e: (-order[e], e))[:k + 1]
        if bias is not None:
            sure[t] &= not _undecided(order[pick], [(logits[t, e], b[e]) for e in pick])
        pick = pick[:k]
        pw = p[t, pick]
        ids[t, :len(pick)] = pick
        w[t, :len(pick)] = scale * (pw / (pw.sum() + 1e-20) if renormalise else pw)
    return ids, w, sure


def linear(a, w):
    """[T, K], [N, K] -> (products, sums of the magnitudes)."""
    return a @ w.T, np.abs(a) @ np.abs(w).T


def _step(v, e):
    """Distance of the E4M3 codes around v at scale 2^e."""
    x = np.maximum(np.abs(v) * np.exp2(-e), 2.0 ** -6)
    return np.exp2(np.floor(np.log2(x)) - 3 + e)


def _round(v, e):
    s = _step(v, e)
    return np.clip(np.rint(v / s) * s, -448 * np.exp2(e), 448 * np.exp2(e))


def quant_with_slack(h, err):
    """The E4M3 values of h [R, I] (groups of 128), and how far those of h +- err may lie from them: nothing
    where both ends round alike, a step where they do not, and a step of the coarser scale all over a group
    whose scale they do not agree on."""
    q, slack = np.empty_like(h), np.empty_like(h)
    for i in range(0, h.shape[1], 128):
        v, d = h[:, i:i + 128], err[:, i:i + 128]
        a = np.abs(v)
        e = O.e8m0_exponent(a.max(1, keepdims=True)).astype(np.float64)
        lo = O.e8m0_exponent(np.maximum(a - d, 0).max(1, keepdims=True)).astype(np.float64)
        hi = O.e8m0_exponent((a + d).max(1, keepdims=True)).astype(np.float64)
        q[:, i:i + 128] = _round(v, e)
        near = _round(v - d, e) != _round(v + d, e)
        s = np.where(near, _step(a + d, e), 0.0)
        slack[:, i:i + 128] = np.where(lo != hi, _step(a + d, hi) + d, s)
    return q, slack


def experts(a, ids, wt, w13, w2):
    """a [T, K], ids/wt [T, k], w13 [E, 2, I, K], w2 [E, N, I], all float64 -> (out, tolerance).  The tolerance
    takes 1e-5 of the magnitudes for each product's FP32 sums, what these and the fast exponential and quotient
    (2^-22 + 2^-23 |g| and 2^-22, on operands that are off by 2^-24: below 2^-20 + 2^-22 |g| of h) can move the 8-bit
    codes in between, half a step of a weighted result (a step is 2^-13 of the largest of 32 columns at most, which the
    other errors can raise to the next power of two) and half a BF16 step."""
    T, N = a.shape[0], w2.shape[1]
    out, tol = np.zeros((T, N)), np.zeros((T, N))
    for e in range(w2.shape[0]):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        g, sg = linear(a[t], w13[e, 0])
        u, su = linear(a[t], w13[e, 1])
        silu = g / (1 + np.exp(-g))
        h = silu * u
        err = 1.1 * np.abs(u) * 1e-5 * sg + np.abs(silu) * 1e-5 * su + (2.0 ** -20 + 2.0 ** -22 * np.abs(g)) * np.abs(h)
        q, slack = quant_with_slack(h, err)
        y, sy = linear(q, w2[e])
        w = wt[t, j][:, None]
        off = 1e-5 * sy + slack @ np.abs(w2[e]).T
        top = np.pad(np.abs(y) + off, ((0, 0), (0, -N % 32))).reshape(len(t), -1, 32).max(2)
        np.add.at(out, t, w * y)
        np.add.at(tol, t, np.abs(w) * (off + 2.0 ** -14 * np.repeat(top, 32, 1)[:, :N]))
    return out, tol + np.abs(out) * 2.0 ** -8 + 2.0 ** -126
