"""Plain float64 implementation of drawing a token (numpy only), one row at a time."""
import numpy as np


def sample(l, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, near=2.0 ** -32):
    """(token, clear): clear is False where a border lies within `near` of the sums that decide."""
    l = np.asarray(l, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    n = int((l > -np.inf).sum())
    if n == 0:
        return -1, True
    best = int(np.argmax(l))
    if not temperature >= 2.0 ** -126:
        return best, True
    order = np.argsort(-l, kind="stable")[:n]
    if l[best] == np.inf:
        w = (l[order] == np.inf).astype(np.float64)
    else:
        w = np.exp((l[order] - l[best]) / np.float64(temperature))
    clear = True
    keep = n
    if 1 <= top_k < keep:
        keep = top_k
    if top_p < 1:
        cum = np.cumsum(w[:keep])
        goal = max(top_p, 0.0) * cum[-1]
        at = int(np.searchsorted(cum, goal))  # the first that reaches it
        keep = min(at, keep - 1) + 1
        clear &= goal == 0 or bool(np.abs(cum - goal).min() > near * cum[-1]) or (w == w[0]).all()
    if min_p > 0:
        # by the exponents: exp(-1e-29), a weight below 1, is 1 in 64 bits
        with np.errstate(invalid="ignore"):
            x = np.where(l[order[:keep]] == l[best], 0.0, (l[order[:keep]] - l[best]) / np.float64(temperature))
        m = np.log(min(float(min_p), 1.0))
        clear &= bool(np.abs(x - m).min() > 1e-12) or m == 0
        keep = int((x >= m).sum())
    kept = np.sort(order[:keep])
    by = np.empty(len(l))
    by[order] = w
    cum = np.cumsum(by[kept])
    goal = min(max(float(u) if u == u else 0.0, 0.0), 1 - 2.0 ** -24) * cum[-1]
    at = int(np.searchsorted(cum, goal, side="right"))
    if goal > 0 and not (w == w[0]).all():
        clear &= bool(np.abs(cum[:-1] - goal).min() > near * cum[-1]) if keep > 1 else True
    return int(kept[min(at, keep - 1)]), clear
