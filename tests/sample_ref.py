"""Plain 64-bit form of sampling, a row at a time."""
import itertools

import numpy as np

EPS = 2.0 ** -28  # a weight's relative error is near 2^-30: borders as near as this may go either way


def token(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """The token drawn from logits x (a 64-bit array) by the number u; -1 where there is none."""
    x = np.where(np.isnan(x), -np.inf, x)
    ids = np.flatnonzero(x > -np.inf)
    if ids.size == 0:
        return -1
    ids = ids[np.argsort(-x[ids], kind="stable")]
    if not t > 0:
        return int(ids[0])
    v, top = x[ids], x[ids[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(v == top, 1.0, np.exp((v - top) / t))
    if 0 < k < x.size:
        ids, w = ids[:k], w[:k]
    mass = np.cumsum(w)
    n = ids.size
    if p < 1:
        n = min(n, 1 + int(np.searchsorted(mass, p * mass[-1], side="left")))
    n = min(n, max(1, int(np.count_nonzero(w >= min(m, 1.0)))))
    mass = mass[:n]
    return int(ids[min(n - 1, int(np.searchsorted(mass, u * mass[-1], side="right")))])


def tokens(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """Every token that borders within EPS of the numbers allow."""
    out = {token(x, u, t, k, p, m)}
    for a, b, c in itertools.product((-EPS, EPS), repeat=3):
        out.add(token(x, max(0.0, u * (1 + a)), t, k, p * (1 + b), m * (1 + c)))
    return out
