"""A mixture of experts in 64 bits on the CPU, with what its fp32 sums may be off
by.  Test infrastructure; shares nothing with the library."""
import numpy as np

from tests import _w4


def choose(logits, top_k, renormalize):
    """Ids (descending logits, the lower id of equal ones) and weights; NaN is
    below every other."""
    key = np.where(np.isnan(logits), -np.inf, logits)
    nan = np.isnan(logits)
    ids = np.stack([np.lexsort((np.arange(logits.shape[1]), -k, n))[:top_k]
                    for k, n in zip(key, nan)])
    v = np.take_along_axis(logits, ids, 1)
    with np.errstate(all="ignore"):
        over = v if renormalize else logits
        p = np.exp(v - v[:, :1]) / np.exp(over - v[:, :1]).sum(1, keepdims=True)
    return ids, p


def layer(x, ids, weights, up, down, terms, act_eps):
    """out [tokens, hidden] and a bound of the error before its rounding."""
    x = np.asarray(x, dtype=np.float64)
    out, bound = np.zeros_like(x), np.zeros_like(x)
    inner = up.codes.shape[1] // 2
    hidden = x.shape[1]
    # four waves or more share K, once it has a unit for each
    r_up = terms * max(hidden / 4, 256) + 16
    r_down = 3 * max(inner / 4, 256) + 16
    experts = up.codes.shape[0]
    for e in range(experts):
        share = np.where(ids == e, weights, 0.0).sum(1)
        rows = np.nonzero((ids == e).any(1))[0]
        if rows.size == 0:
            continue
        wu, wd = up.values(e) * up.factor(e), down.values(e) * down.factor(e)
        h = x[rows] @ wu.T
        dh = _w4.product_bound(r_up, np.abs(x[rows]) @ np.abs(wu).T) + 2.0 ** -24 * np.abs(h)
        g, u, dg, du = h[:, :inner], h[:, inner:], dh[:, :inner], dh[:, inner:]
        with np.errstate(over="ignore"):
            silu = g / (1 + np.exp(-g))
        a = silu * u
        # |silu'| < 1.1; the exponential, the quotient and the product are a few units off
        da = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du
        da = da + (8 * 2.0 ** -23 + act_eps) * np.abs(a)
        w = np.abs(share[rows])[:, None]
        size = np.abs(a) @ np.abs(wd).T
        out[rows] += share[rows][:, None] * (a @ wd.T)
        bound[rows] += w * (da @ np.abs(wd).T + _w4.product_bound(r_down + experts, size))
    return out, bound
