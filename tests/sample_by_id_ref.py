"""Plain 64-bit form of sampling whose draw walks the kept tokens by rising id, a row at a time."""
import itertools

import numpy as np

# What the borders may be off by.  A weight is off by less than 2^-28 of itself (its exponent's parts and series), and is a
# whole number of 2^-44, so a mass of n weights, the largest of them 1, by less than n 2^-44 more.
EPS, UNIT = 2.0 ** -28, 2.0 ** -44


def kept(x, t=1.0, k=0, p=1.0, m=0.0):
    """(ids by rising id, their weights) of the tokens that the filters keep of logits x (a 64-bit array)."""
    w = np.zeros(x.size)
    top = np.nanmax(np.where(np.isnan(x), -np.inf, x), initial=-np.inf)
    if top == -np.inf:
        return np.empty(0, int), np.empty(0)
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / t) if t > 0 else 0.0)
    w = np.where(np.isnan(x) | np.isnan(w), 0.0, w)
    order = np.argsort(-np.where(np.isnan(x), -np.inf, x), kind="stable")
    n = int(np.count_nonzero(x > -np.inf)) if t > 0 else 1
    if 0 < k < x.size:
        n = min(n, k)
    mass = np.cumsum(w[order[:n]])
    if p < 1:
        n = min(n, 1 + int(np.searchsorted(mass, p * mass[-1], side="left")))
    n = min(n, max(1, int(np.count_nonzero(w >= min(m, 1.0)))))
    ids = np.sort(order[:n])
    return ids, w[ids]


def drawn(ids, w, u):
    mass = np.cumsum(w)
    at = int(np.searchsorted(mass, u * mass[-1], side="right"))
    return int(ids[at]) if at < ids.size else int(ids[np.flatnonzero(w)[-1]])


def token(x, u, **filters):
    ids, w = kept(x, **filters)
    return drawn(ids, w, u) if ids.size else -1


def tokens(x, u, t=1.0, k=0, p=1.0, m=0.0):
    """Every token that the numbers' errors allow."""
    out, room = set(), x.size * UNIT
    for b, c in itertools.product((-1, 0, 1), repeat=2):
        ids, w = kept(x, t, k, p * (1 + b * EPS) + b * room if p < 1 else p, m * (1 + c * EPS))
        if ids.size == 0:
            return {-1}
        out |= {drawn(ids, w, max(0.0, u * (1 + a * EPS) + a * room)) for a in (-1, 0, 1)}
    return out
