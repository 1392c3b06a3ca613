"""GPU tests of s2_sample where a cluster of blocks goes through many rows of unlike settings, one after the other,
against the plain float64 implementation in tests/_sample.py."""
import numpy as np
import pytest

from tests.test_gpu_sample import check, normal, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,ld", [(1900, 1003, 1003), (300, 40009, 40016), (40, 1000003, 1000003)])
def test_rows_of_all_kinds_follow_one_another(T, V, ld, dtype):
    """At most 304 clusters are on the device at once. (Rows in which a border lies within 2^-32 of what decides
    are not compared: at most one in fifty, as in the tests of single calls.)"""
    rng = np.random.default_rng([T, V])
    z = normal(T, V, 21) * rng.choice([0.05, 1.0, 3.0], (T, 1)) + rng.uniform(-100, 100, (T, 1))
    kind = rng.integers(0, 25, T)
    z[kind == 0] = -np.inf
    z[kind == 1] = np.nan
    z[kind == 2, ::2] = -np.inf
    some = np.nonzero(kind == 3)[0]
    z[some, rng.integers(0, V, len(some))] = np.inf
    if dtype == "f32":  # (bfloat16 numbers that far from zero are too few: most would be equal)
        z[kind == 4] += 1e5
    check(z, rng.random(T), dtype, ld=ld, off=3, **settings(T, V + 1))
