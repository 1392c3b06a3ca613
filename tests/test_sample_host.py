"""s2_sample without a GPU: the plain implementation that the GPU tests compare with, and the refusals of
the entry point (no call here reaches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

from tests._sample import sample

VP, U64, I32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int
OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
A = 0x10000000  # fake, aligned device addresses; never dereferenced
G = 1 << 32     # far apart


def test_plain_by_hand():
    l = np.log([0.1, 0.4, 0.2, 0.3])
    draw = lambda u, **kw: sample(l, u, **kw)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.999, 1.0, float("nan"))] == [0, 0, 1, 1, 2, 2, 3, 3, 3, 0]
    assert [draw(u, top_k=2) for u in (0.0, 0.57, 0.58)] == [1, 1, 3]              # 4/7 and 3/7
    assert [draw(u, top_p=0.7 - 1e-9) for u in (0.0, 0.58)] == [1, 3]
    assert [draw(u, top_p=0.7 + 1e-9) for u in (0.0, 0.45, 0.67)] == [1, 2, 3]     # 4/9, 2/9, 3/9
    assert [draw(u, min_p=0.6) for u in (0.0, 0.58)] == [1, 3]
    assert [draw(u, top_k=3, top_p=0.5) for u in (0.0, 0.58)] == [1, 3]            # 4/9 is not enough
    assert draw(0.99, top_p=0.0) == 1 and draw(0.99, temperature=0.0) == 1 and draw(0.99, temperature=float("nan")) == 1
    assert draw(0.99, min_p=5.0) == 1 and draw(0.5, top_k=-3) == draw(0.5)
    assert sample([-np.inf, np.nan], 0.5)[0] == -1
    assert sample([0.0, np.inf, 3.0, np.inf], 0.6)[0] == 3
    assert sample([2.0, 2.0, 2.0, 1.0], 0.9, top_k=2)[0] == 1


def test_plain_frequencies():
    """Over an even grid of u every token comes as often as its probability says."""
    l = np.random.default_rng(0).normal(size=20)
    got = np.bincount([sample(l, (i + 0.5) / 4000, temperature=0.7)[0] for i in range(4000)], minlength=20) / 4000
    p = np.exp(l / 0.7) / np.exp(l / 0.7).sum()
    assert np.abs(got - p).max() <= 1 / 4000 + 1e-12


@pytest.fixture(scope="module")
def call():
    from sketch_compressed_sparse_gb300 import build

    f = ctypes.CDLL(build.build()).s2_sample
    f.argtypes, f.restype = [VP, I32, U64, U64, U64, VP, VP, VP, VP, VP, VP, VP], I32

    def one(z=A, dt=0, T=10, V=100, ld=100, t=A + G, k=A + 2 * G, p=A + 3 * G, m=A + 4 * G, u=A + 5 * G, out=A + 6 * G):
        return f(z, dt, T, V, ld, t, k, p, m, u, out, None)

    return one


def test_refusals(call):
    assert call(dt=2) == INVALID and call(ld=99) == INVALID
    assert call(z=None) == INVALID and call(u=None) == INVALID and call(out=None) == INVALID
    assert call(z=A + 2) == ALIGN and call(dt=1, z=A + 1) == ALIGN
    for name, at in (("t", 1), ("k", 2), ("p", 3), ("m", 4), ("u", 5), ("out", 6)):
        assert call(**{name: A + at * G + 2}) == ALIGN
    assert call(out=A + 36) == INVALID
    for at in range(1, 6):
        assert call(out=A + at * G + 36) == INVALID
    assert call(T=1 << 31) == UNSUP and call(V=1 << 31, ld=1 << 31) == UNSUP
    assert call(T=0) == OK and call(T=0, z=None, u=None, out=None) == OK


def test_binding_refusals():
    import sketch_compressed_sparse_gb300 as s2

    with pytest.raises(ValueError, match="CUDA"):
        s2.s2_sample(torch.zeros(2, 8), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
