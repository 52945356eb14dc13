"""CPU oracle of what surrounds the experts' products: the router, the gated
activation with its 8-bit checkpoint, the weighted sum over a token's experts.

TEST INFRASTRUCTURE ONLY: numpy in fp64, no code shared with the HIP path.
"""

from __future__ import annotations

import numpy as np

from .mxfp8 import BLOCK, E8M0_NAN, e4m3_decode, e4m3_encode, e8m0_from_amax, e8m0_value


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


def scores(logits, masked, score):
    """fp64 scores [T, E]; masked experts (and rows of nothing else) 0."""
    l = np.asarray(logits, dtype=np.float64)
    if score == "sigmoid":
        return np.where(masked, 0.0, sigmoid(l))
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        on = ~masked[t]
        if on.any():
            with np.errstate(invalid="ignore"):
                e = np.exp(l[t, on] - l[t, on].max())
            out[t, on] = e / e.sum()
    return out


def shares(l, masked, ids, score):
    """Chosen scores over their sum, by their logarithms: scores below fp64's range
    have shares all the same.  0 for masked experts."""
    x = np.take_along_axis(l, ids, 1)
    if score == "sigmoid":
        x = np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
    out = np.zeros(ids.shape)
    for t in range(l.shape[0]):
        on = ~masked[t, ids[t]]
        if on.any():
            e = np.exp(x[t, on] - x[t, on].max())
            out[t, on] = e / e.sum()
    return out


def router(logits, lowest, k, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renormalize=True,
           scale=1.0):
    """(ids [T, k], weights fp64 [T, k]): token by token, sorting (value, index) pairs.
    `lowest`: the lowest finite value of the logits' type."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    masked = l <= lowest
    s = scores(l, masked, score)
    c = l.copy() if bias is None and (groups == 1 or group_score == "max") else s + (0.0 if bias is None else
                                                                                       np.asarray(bias, np.float64))
    last = masked | np.isnan(c)
    n = E // groups
    ids = np.zeros((T, k), dtype=np.int32)
    for t in range(T):
        key = lambda e: (last[t, e], -c[t, e] if not last[t, e] else 0.0, e)  # noqa: E731
        value = []
        for g in range(groups):
            live = sorted((c[t, e] for e in range(g * n, g * n + n) if not last[t, e]), reverse=True)
            v = live[:1] if group_score == "max" else live[:2]
            value.append((not v, -sum(v) if v else 0.0, g))
        kept = sorted(g for _, _, g in sorted(value)[:topk_groups])
        ids[t] = sorted((e for g in kept for e in range(g * n, g * n + n)), key=key)[:k]
    return ids, scale * (shares(l, masked, ids, score) if renormalize else np.take_along_axis(s, ids, 1))


def router_weights(l, ids, score, renormalize, scale):
    """Weights of one token as a function of its logits (ids fixed): what the gradient is of."""
    s = sigmoid(l) if score == "sigmoid" else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
    w = s[ids]
    return scale * (w / w.sum() if renormalize else w)


def router_grad(logits, lowest, ids, dw, score, renormalize, scale):
    """(dlogits fp64 [T, E], the sum of the magnitudes that each was added from)."""
    l = np.asarray(logits, dtype=np.float64)
    masked = l <= lowest
    s = scores(l, masked, score)
    T, E = l.shape
    p = shares(l, masked, ids, score)
    out, mag = np.zeros_like(l), np.zeros_like(l)
    for t in range(T):
        i, si = ids[t], s[t, ids[t]]
        rest = sigmoid(-l[t, i])                    # 1 - s, of which nothing is lost where s is close to 1
        g = scale * np.asarray(dw[t], np.float64)
        if renormalize:
            # through the shares, whose derivative by the logarithm of score m is p_j (delta - p_m)
            d, m = p[t] * (g - (g * p[t]).sum()), p[t] * (np.abs(g) + (np.abs(g) * p[t]).sum())
            out[t, i], mag[t, i] = (d * rest, m * rest) if score == "sigmoid" else (d, m)
        elif score == "sigmoid":
            out[t, i], mag[t, i] = g * si * rest, np.abs(g) * si * rest
        else:
            ds, dm = np.zeros(E), np.zeros(E)
            ds[i], dm[i] = g, np.abs(g)
            out[t], mag[t] = s[t] * (ds - (s[t] * ds).sum()), s[t] * (dm + (s[t] * dm).sum())
    return out, mag


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_grad(dh, g, u):
    """(dg, du, the magnitudes that dg was added from)."""
    s = sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s, np.abs(dh * u) * s * (1 + np.abs(g) * (1 - s))


def combine(y, w, routed):
    """(out [T, N], sums of magnitudes); y [T, k, N]; items that are not routed add nothing."""
    y = np.where(routed[:, :, None], y, 0.0)
    w = np.where(routed, w, 0.0)[:, :, None]
    return (w * y).sum(1), (np.abs(w) * np.abs(y)).sum(1)


def combine_grad(dout, y, w, routed):
    """(dy, dcombine, sums of magnitudes of dcombine)."""
    y = np.where(routed[:, :, None], y, 0.0)
    p = dout[:, None, :] * y
    return np.where(routed, w, 0.0)[:, :, None] * dout[:, None, :], p.sum(2), np.abs(p).sum(2)


def codes_reached(q, s, x, d):
    """Which codes may stand for x, known to within d: truth values like q.

    q, s: codes [R, C] and row-major scale bytes [R, C/32] of values x [R, C] in
    1x32 blocks.  A block's byte has to be that of a largest magnitude within
    reach, a code (with that byte) lie between those of x - d and x + d."""
    R, C = x.shape
    xb, db, qb = (a.reshape(R, C // BLOCK, BLOCK) for a in (x, d, q))
    none = np.zeros((R, C // BLOCK), dtype=bool)
    lo = e8m0_from_amax(np.maximum(np.abs(xb) - db, 0).max(2), none)
    hi = e8m0_from_amax((np.abs(xb) + db).max(2), none)
    nan = ~np.isfinite(xb).all(2)
    byte_ok = np.where(nan, s == E8M0_NAN, (s >= lo) & (s <= hi))
    with np.errstate(invalid="ignore"):
        inv = 1.0 / e8m0_value(s)[:, :, None]
        a, v, b = (e4m3_decode(e4m3_encode(np.nan_to_num((xb + e) * inv))) for e in (-db, 0 * db, db))
        got = e4m3_decode(qb)
        ok = np.where(nan[:, :, None], (qb & 0x7F) == 0x7F, (got >= np.minimum(a, v)) & (got <= np.maximum(b, v)))
    return (ok & byte_ok[:, :, None]).reshape(R, C)
