"""GPU tests of what s2_sample's weights are: whole numbers of a unit of 2^-43 of the largest, rounded to nearest (twice
that for each factor of two of V above 2^19), so that a token below half a unit is never drawn, not even with u = 0.

The rule is followed here in exact integers. A weight is right to 2^-35 of itself before it is rounded, so each lies
between two whole numbers, and so do the sums A of the weights up to a border and R of those behind it, which have no
weight in common. A exceeds u times the sum of both where (1 - u) A exceeds u R; rows in which the ends of A and R leave
that open are not compared, one at most.
"""
from fractions import Fraction
from math import floor

import numpy as np
import pytest
import torch

from tests._sample import sample

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2

DEV = "cuda"


def drawn(l, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, clear) of a row of finite or -infinite logits."""
    l = l.astype(np.float64)
    best, V = int(np.argmax(l)), len(l)
    x = (l - l[best]) / np.float64(temperature)
    unit = 2.0 ** (43 - max(0, (V - 1).bit_length() - 19))
    low, high = (np.rint(np.exp(x) * (1 + e) * unit).astype(np.int64) for e in (-2.0 ** -35, 2.0 ** -35))
    middle = np.rint(np.exp(x) * unit).astype(np.int64)

    def sums(of, at):
        """Ends of A and of R around the border behind of[at], as whole numbers."""
        return [[int(w[of[:at + 1]].sum()), int(w[of[at + 1:]].sum())] for w in (low, high)]

    order, clear = np.argsort(-l, kind="stable"), True
    order = order[:int((l > -np.inf).sum())]
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:  # the first A that is p of A + R or more
        p, a = Fraction(float(top_p)), np.cumsum(middle[order])
        at = min(int(np.searchsorted(a, float(p) * float(a[-1]))), len(a) - 1)
        (a0, r0), (a1, r1) = sums(order, at)
        clear &= (1 - p) * a0 >= p * r1
        if at:
            (a0, r0), (a1, r1) = sums(order, at - 1)
            clear &= (1 - p) * a1 < p * r0
        order = order[:at + 1]
    if min_p > 0:
        keep = x[order] >= np.log(np.float64(min_p))
        clear &= bool(np.abs(x[order] - np.log(np.float64(min_p))).min() > 1e-12)
        order = order[keep]
    kept = np.sort(order)
    v = Fraction(min(float(u), 1 - 2.0 ** -24)) if u > 0 else Fraction(0)  # (NaN: 0)
    a = np.cumsum(middle[kept])
    at = int(np.searchsorted(a, floor(v * int(a[-1])), side="right"))
    (a0, r0), (a1, r1) = sums(kept, at)
    clear &= (1 - v) * a0 > v * r1
    if at:
        (a0, r0), (a1, r1) = sums(kept, at - 1)
        clear &= (1 - v) * a1 <= v * r0
    return int(kept[at]), clear


def logits(T, V, rng):
    """A Zipf prior over the words in some order, noise, and a few words that the context makes likely."""
    z = rng.normal(size=(T, V)) * 1.2 - 1.1 * np.log(1.0 + np.stack([rng.permutation(V) for _ in range(T)]))
    for r in z:
        r[rng.integers(0, V, 12)] += 6 + 2 * rng.normal(size=12)
    return z.astype(np.float32)


@pytest.mark.parametrize("T,V", [(300, 1003), (120, 33278), (40, 267735), (10, 1000003)])
def test_smallest_random_numbers_on_peaked_rows(T, V):
    rng = np.random.default_rng([T, V])
    z = logits(T, V, rng)
    z[::7, ::3] = -np.inf
    u = rng.choice(np.float32([0.0, 0.0, -0.0, 2.0 ** -24, 2.0 ** -23, 1e-30, np.nan, -1.0, 0.25, 1 - 2.0 ** -24, 1.0]), T)
    for kw in (dict(), dict(top_k=rng.choice([0, 1000, V // 2, V - 1], T)), dict(top_p=rng.choice([0.9, 0.999, 1 - 2.0 ** -24], T)),
               dict(min_p=rng.choice([1e-30, 2.0 ** -50, 1e-3], T)),
               dict(top_k=rng.choice([0, V // 3], T), top_p=rng.choice([0.99, 1 - 2.0 ** -20], T), min_p=rng.choice([0.0, 1e-12], T))):
        kw["temperature"] = rng.choice([0.1, 0.2, 0.3, 1.0], T)
        kw = {k: v.astype(np.int32 if k == "top_k" else np.float32) for k, v in kw.items()}
        out = torch.full((T,), -7, dtype=torch.int32, device=DEV)
        s2.s2_sample(torch.from_numpy(z).to(DEV), torch.from_numpy(u).to(DEV), out, **{k: torch.from_numpy(v).to(DEV) for k, v in kw.items()})
        got, unclear = out.cpu().numpy(), 0
        for i in range(T):
            want, clear = drawn(z[i], u[i], **{k: v[i] for k, v in kw.items()})
            assert got[i] == want or not clear, (i, got[i], want, u[i], {k: v[i] for k, v in kw.items()})
            unclear += not clear
        assert unclear <= 1


def test_tokens_that_weigh_nothing_are_not_drawn():
    """A token of weight 2^-45 is left out, one of 2^-43 is drawn with u = 0; without units the first would be."""
    z = np.zeros((2, 40), np.float32)
    z[0] = -45 * np.log(2.0)
    z[1] = -43 * np.log(2.0)
    z[:, 30] = 0
    out = torch.empty(2, dtype=torch.int32, device=DEV)
    s2.s2_sample(torch.from_numpy(z).to(DEV), torch.zeros(2, device=DEV), out)
    assert out.tolist() == [30, 0]
    assert [sample(r, 0.0)[0] for r in z] == [0, 0]
