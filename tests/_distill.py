"""Plain float64 implementation of the softmax layer's loss against a teacher (numpy only), row by row."""
import numpy as np


def softmax(x):
    """Probabilities and their logarithms; a row of nothing but -infinity has probability 0 everywhere."""
    if not (x > -np.inf).any() and not np.isnan(x).any():
        return np.zeros_like(x), np.full_like(x, -np.inf)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = x - x.max()
        lse = np.log(np.exp(d).sum())
        return np.exp(d - lse), d - lse


def distill(z, idx, t, targets, weight, temperature, soft, hard, scale):
    """(loss [T], gradient [T][V], room [T], grad_room [T][V]): the last two are the sums of magnitudes that
    rounding errors are relative to. All inputs float64 or integer arrays; idx, t, targets, weight may be None."""
    T, V = z.shape
    loss, grad, room, groom = np.zeros(T), np.zeros((T, V)), np.zeros(T), np.zeros((T, V))
    for r in range(T):
        w = 1.0 if weight is None else weight[r]
        if w == 0:
            continue
        one, d = 0.0, np.zeros(V)
        if idx is not None and soft != 0:
            ok = (idx[r] >= 0) & (idx[r] < V)
            i, x = idx[r][ok], t[r][ok] / temperature
            q, logq = softmax(x)
            if (q > 0).any() or np.isnan(q).any():
                p, logp = softmax(z[r] / temperature)
                qi = np.zeros(V)
                np.add.at(qi, i, q)
                some = ~(q == 0)
                one += soft * (q[some] * (logq[some] - logp[i[some]])).sum()
                d += soft / temperature * (p - qi)
                groom[r] += soft / temperature * (p + qi)
                with np.errstate(invalid="ignore"):
                    room[r] += soft * (q[some] * (np.abs(logq[some]) + np.abs(logp[i[some]]) + 1)).sum()
        if targets is not None and hard != 0 and 0 <= targets[r] < V:
            p, logp = softmax(z[r])
            y = targets[r]
            one -= hard * logp[y]
            d += hard * p
            d[y] -= hard
            groom[r] += hard * p
            groom[r][y] += hard
            room[r] += hard * (np.abs(logp[y]) + 1)
        loss[r] = w * one
        grad[r] = w * scale * d
        groom[r] *= abs(w * scale)
        room[r] *= abs(w)
    return loss, grad, room, groom
