"""GPU tests of s2_distill where a cluster of blocks goes through many rows, one after the other.

At most 456 clusters are on the device at once, so 2600 rows give each of them five or six; rows of
1,000,003 float32 take sixteen blocks each, of which nine at most are there.

Rounding. A thread of 192 of a block takes ceil(n / 192) of a row's n groups of eight logits (fewer where
blocks share the row) and adds four exponentials of each to either of two sums: ceil(n / 192) * 4 additions
of positive numbers, each off by at most 2^-24, and 20 more until the row's sum is there. An exponential
exp2(x) is off by 2^-22, and by 2^-24 |x| as x was rounded. The numbers of a sum lie over a base that is at
most 30 factors of two away from it, and the mean of |x| under the probabilities is at most that and log2 V
more. So a sum is off by at most
    E = (4 + 30 + log2 V + 4 ceil(n / 192) + 20 + 12) * 2^-24
of itself (12: the logarithm, the base moved to the sum, the teacher's probabilities and their sums), the
loss by E times the sums of magnitudes that tests/_distill.py gives, and a gradient by E and its own
exponential's (4 + |x|) * 2^-24 times the magnitudes that make it up, and half a step of its type.
"""
import math

import numpy as np
import pytest
import torch

from tests import _distill as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def bound(V):
    return (66 + math.log2(V) + 4 * -(-((V + 14) // 8) // 192)) * 2.0 ** -24


def dev(a, dtype):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def check(z, idx, t, y, w, dtype, ddtype, temperature, soft, hard, ld):
    T, V = z.shape
    flat = torch.full((T * ld + 9,), 5.0, dtype=DT[dtype], device=DEV)
    logits = flat[:T * ld].reshape(T, ld)[:, :V]
    logits.copy_(dev(z, torch.float32))
    z64 = logits.double().cpu().numpy()
    t = None if t is None else t.astype(np.float32).astype(np.float64)
    w = None if w is None else w.astype(np.float32).astype(np.float64)
    want, dwant, room, droom = ref.distill(z64, idx, t, y, w, temperature, soft, hard, 1.0)
    args = dict(targets=dev(y, torch.int32), row_weight=dev(w, torch.float32), temperature=temperature, soft=soft, hard=hard)
    loss = torch.full((T + 1,), 7.0, device=DEV)
    out = torch.full((T * ld + 9,), 5.0, dtype=DT[ddtype], device=DEV)
    d = out[:T * ld].reshape(T, ld)[:, :V]
    E, losses = bound(V), []
    for grad in (d, None):
        loss.fill_(7.0)
        s2.s2_distill(logits, dev(idx, torch.int32), dev(t, torch.float32), loss, grad, **args)
        got = loss.double().cpu().numpy()
        assert got[T] == 7.0
        got = got[:T]
        losses.append(got)
        same = np.isfinite(want)
        np.testing.assert_array_equal(got[~same], want[~same])
        np.testing.assert_array_less(np.abs(got[same] - want[same]), (E * room + 2.0 ** -24 * np.abs(want))[same] + 1e-37)
    dgot = d.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(dgot), np.isnan(dwant))
    for r in range(T):
        fine = np.isfinite(dwant[r])
        if not fine.any():
            continue
        with np.errstate(invalid="ignore"):
            x = (z64[r].max() - z64[r]) / min(1.0, temperature) / math.log(2) + math.log2(V)
        x = np.where(np.isfinite(x), np.minimum(x, 150.0), 150.0)
        tol = (E + (4 + x) * 2.0 ** -24) * droom[r] + STEP[ddtype] * np.abs(dwant[r]) * 1.01 + 1e-37
        assert (np.abs(dgot[r] - dwant[r]) <= tol)[fine].all(), (r, np.max((np.abs(dgot[r] - dwant[r]) / tol)[fine]))
    d.fill_(5.0)
    assert bool((out == 5.0).all()), "wrote outside dlogits"
    return losses


def make(T, V, K, far=100.0, tag=0):
    """Rows at levels up to `far` from one another, some of them without weight, masked, NaN or infinite."""
    rng = np.random.default_rng([T, V, K, tag])
    z = rng.normal(size=(T, V)) * rng.choice([0.01, 1.0, 4.0], (T, 1)) + rng.uniform(-far, far, (T, 1)) * (rng.random((T, 1)) < 0.7)
    idx = rng.integers(0, V, (T, K))
    if K > 2:
        idx[rng.random(T) < 0.3, 1] = V  # a shorter list
        some = rng.random(T) < 0.3
        idx[some, 2] = idx[some, 0]      # an index twice
    t, y = rng.normal(size=(T, K)) * 3, rng.integers(0, V, T)
    y[rng.random(T) < 0.2] = -1
    if K:
        some = rng.random(T) < 0.2
        y[some] = np.minimum(idx[some, 0], V - 1)
    w = rng.random(T) + 0.5
    w[rng.random(T) < 0.2] = 0
    kind = rng.integers(0, 40, T)
    z[kind == 0] = -np.inf
    z[kind == 1] = np.nan
    z[np.nonzero(kind == 2)[0], rng.integers(0, V, int((kind == 2).sum()))] = np.inf
    z[kind == 3] = np.where(rng.random((int((kind == 3).sum()), V)) < 0.9, -np.inf, z[kind == 3])
    z[kind == 4] = np.finfo(np.float32).min
    return z, idx, t, y, w


FORMS = [(1.0, 1.0, 0.5), (2.0, 4.0, 0.3), (3.0, 2.0, 0.3), (0.7, 1.0, 0.0)]  # one sum, a sum and its squares', two sums


@pytest.mark.parametrize("dtype,ddtype", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("K,ld", [(9, 1003), (9, 1016), (300, 1007)])
def test_many_rows_of_a_cluster(form, K, ld, dtype, ddtype):
    temperature, soft, hard = form
    z, idx, t, y, w = make(2600, 1003, K)
    a, b = check(z, idx, t, y, w, dtype, ddtype, temperature, soft, hard, ld)
    if K < 300:  # the sums do not depend on whether a gradient is wanted
        np.testing.assert_allclose(a, b, rtol=4 * bound(1003), atol=1e-5)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("far", [3e3, 1e5, 1e6, 1e8])
def test_many_rows_far_from_zero(form, far):
    """Logits of that size, whose sums' bases are floats up to 8 apart: what a base is rounded by is not lost."""
    temperature, soft, hard = form
    z, idx, t, y, w = make(2600, 1003, 9, far=far)
    check(z, idx, t, y, w, "f32", "f32", temperature, soft, hard, 1003)


def test_many_rows_without_a_teacher():
    z, _, _, y, w = make(2600, 1003, 0)
    check(z, None, None, y, w, "f32", "f32", 1.0, 0.0, 1.0, 1003)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,V,K", [("f32", 1000003, 9), ("bf16", 300007, 9), ("f32", 1000003, 300)])
def test_many_rows_of_large_clusters(form, dtype, V, K):
    """Sixteen and eight blocks a row; the larger rows do not stay in shared memory as a whole."""
    temperature, soft, hard = form
    if K > 256 and temperature != 2.0:
        return
    z, idx, t, y, w = make(40, V, K)
    check(z, idx, t, y, w, dtype, dtype, temperature, soft, hard, V)
