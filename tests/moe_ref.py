"""The mixture-of-experts layer in numpy and 64 bits, with a bound on what the library may be off by."""
import numpy as np
from scipy.special import erfc


def routing(x, router, k):
    """(logits, what they may be off by, order of the experts, gap): the router adds the products of a logit in
    32 chains and a tree of them."""
    z = x @ router.T
    dz = (x.shape[1] / 32 + 16) * 2.0 ** -24 * (np.abs(x) @ np.abs(router).T)
    order = np.argsort(-z, axis=1, kind="stable")
    if k == router.shape[0]:
        return z, dz, order, np.inf
    lo = np.take_along_axis(z - dz, order, 1)[:, :k].min(1)
    hi = np.take_along_axis(z + dz, order, 1)[:, k:].max(1)
    return z, dz, order, (lo - hi).min()


def layer(x, router, w1, w2, k, act, normalize, u):
    """(y, bound, ids, weights, gap) for float64 inputs; u: half a step of the 16-bit type, relative.

    The bound follows the computation: FP32 sums of n exact products are off by at most n 2^-24 times
    the sum of magnitudes in any order (2^-23 where the tensor core truncates), expf by 2 units in the last
    place; h is held in two 16-bit parts (off by u of the second, which is at most u of h), and y is rounded once.  gap: the least difference between a chosen and a
    passed-over logit, less what both may be off by (a choice is certain where it is positive).
    """
    T, H = x.shape
    E, I = router.shape[0], w2.shape[2]
    z, dz, order, gap = routing(x, router, k)
    ids = order[:, :k]
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, ids, 1)
    if normalize:
        w = w / w.sum(1, keepdims=True)
    # weights: every exponent off by its logit and the maximum's, the sums by E additions
    dw = w * (4 * dz.max(1, keepdims=True) + (E + 16) * 2.0 ** -23)
    y, b = np.zeros((T, H)), np.zeros((T, H))
    n1, n2 = (H + 64) * 2.0 ** -23, (2 * I + 64) * 2.0 ** -23
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        a = x[t] @ w1[e].T
        da = n1 * (np.abs(x[t]) @ np.abs(w1[e]).T)
        if act == "swiglu":
            g, up, dg, dup = a[:, :I], a[:, I:], da[:, :I], da[:, I:]
            with np.errstate(over="ignore"):
                sg = g / (1 + np.exp(-g))
            h = sg * up  # silu' stays below 1.1 in magnitude
            dh = 1.1 * dg * np.abs(up) + np.abs(sg) * dup + 1.1 * dg * dup + 2.0 ** -20 * np.abs(h)
        elif act == "gelu":
            h = 0.5 * a * erfc(-a / np.sqrt(2))  # slope below 1.13; erff 2 units in the last place
            dh = 1.13 * da + 2.0 ** -21 * np.abs(a)
        else:
            h, dh = np.maximum(a, 0), da
        dh = dh + u * u * (np.abs(h) + dh) + 2.0 ** -24  # (FP16: below the normal range a step is 2^-24)
        o = h @ w2[e].T
        do = dh @ np.abs(w2[e]).T + n2 * ((np.abs(h) + dh) @ np.abs(w2[e]).T)
        y[t] += w[t, j][:, None] * o
        b[t] += w[t, j][:, None] * do + dw[t, j][:, None] * (np.abs(o) + do)
        b[t] += 2.0 ** -22 * w[t, j][:, None] * np.abs(o)
    return y, b + u * (np.abs(y) + b) + 2.0 ** -24, ids, w, gap
