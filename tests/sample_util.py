"""The sampler's definition in 64 bits, on the CPU, row by row."""
import math

import numpy as np


def reference(logits, u, temperature, top_k, top_p, min_p):
    """For one row of float64 logits: (the kept indexes in order, their running sums of weights, token, logprob, margin), or None
    for a row without an answer. margin: how far u times the whole is from the borders next to it, and top_p's sums from
    theirs, relative to the whole: a token is decided where that is well above the weights' rounding (0 where a weight is
    as near to min_p as the exponential is exact)."""
    l = np.asarray(logits, np.float64) + 0.0
    if np.isnan(l).any() or not (l > -np.inf).any() or not temperature >= 0 or any(math.isnan(x) for x in (u, top_p, min_p)):
        return None
    top = l.max()
    if temperature == 0:
        return np.array([l.argmax()]), np.ones(1), int(l.argmax()), 0.0, 1.0
    if top == np.inf:
        w = (l == np.inf).astype(np.float64)
    else:
        with np.errstate(all="ignore"):
            w = np.exp(np.where(l == top, 0.0, np.where(l == -np.inf, -np.inf, (l - top) / temperature)))
    order = np.argsort(-l, kind="stable")
    margin = 1.0
    if top_p <= 0:
        top_k, top_p = 1, 1.0
    if 0 < top_k < len(l):
        order = order[:top_k]
    if top_p < 1:
        sums = np.cumsum(w[order])
        need = int((sums < top_p * sums[-1]).sum()) + 1
        margin = min(margin, np.abs(sums / sums[-1] - top_p).min())
        order = order[:need]
    m = min(max(min_p, 0.0), 1.0)
    # one weight against min_p: no sum, so the exponential's own error decides, 2^-44.6 relative here and less there
    if m > 0 and (np.abs(w[order][w[order] != 1] / m - 1) < 1e-12).any():
        margin = 0.0
    order = order[w[order] >= m]
    index = np.sort(order)
    sums = np.cumsum(w[index])
    x = min(max(u, 0.0), 1.0 - 2.0 ** -53)
    margin = min(margin, np.abs(sums[:-1] / sums[-1] - x).min(initial=1.0))
    token = int(index[min(int((sums <= x * sums[-1]).sum()), len(index) - 1)])
    with np.errstate(all="ignore"):
        return index, sums, token, float(np.log(w[token] / sums[-1])), margin
