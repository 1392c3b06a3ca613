"""s2_distill takes a row's sums over the log-sum of the row before: a test that no row's result depends on it."""
import math

import numpy as np
import pytest
import torch

from tests import _distill as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2

DEV = "cuda"


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


@pytest.mark.parametrize("level", [0.0, 1e3, 2e4, 3e5, -4e6, 3e7])
@pytest.mark.parametrize("form", [(1.0, 0.0, 1.0), (1.0, 1.0, 0.0), (2.0, 1.0, 1.0), (3.0, 1.0, 1.0)])
def test_a_row_does_not_depend_on_the_level_of_the_one_before(form, level):
    """Rows that one word (or two of like weight) dominates, at levels 0 to 50 apart, around 0 and far from it (a logit
    is a float exactly there too, and so is its distance from one beside it). With x the exponent of that
    word over the base of its sums, at most 30, its exponential is off by 2^-22 + 2^-20 ln 2 (half a step of numbers below
    32), and 2^-22 more for what follows: 1.15e-6, and a loss (of little more than 0, or log 2) or a probability by no
    more. At temperature 2 the cross entropy's sum is of the squares of those exponentials: twice that."""
    temperature, soft, hard = form
    T, V = 2600, 1003
    rng = np.random.default_rng(3)
    z = np.full((T, V), -60.0 * max(1.0, temperature)) + rng.random((T, V))
    at = np.stack([rng.permutation(V)[:2] for _ in range(T)])
    rows = np.arange(T)
    z[rows, at[:, 0]] = rng.random(T)
    two = rows % 2 == 0
    z[rows[two], at[two, 1]] = z[rows[two], at[two, 0]]
    z = (z + rng.uniform(0, 50 * max(1.0, temperature), (T, 1)) + level).astype(np.float32)
    idx, t = at[:, :1], np.zeros((T, 1))
    teacher = (dev(idx, torch.int32), dev(t, torch.float32)) if soft else (None, None)
    loss, d = torch.empty(T, device=DEV), torch.empty((T, V), device=DEV)
    s2.s2_distill(dev(z, torch.float32), *teacher, loss, d, targets=dev(at[:, 0], torch.int32), temperature=temperature, soft=soft, hard=hard)
    want, dwant, _, _ = ref.distill(z.astype(np.float64), idx if soft else None, t, at[:, 0], None, temperature, soft, hard, 1.0)
    most = (soft + (2 if temperature == 2.0 else 1) * hard) * (2.0 ** -21 + 2.0 ** -20 * math.log(2))
    off, doff = np.abs(loss.double().cpu().numpy() - want), np.abs(d.double().cpu().numpy() - dwant).max(axis=1)
    assert off.max() <= most, (off.max() / most, np.mean(off) / most)
    assert doff.max() <= 2 * most, doff.max() / most
