"""s2_distill without a GPU: the plain implementation that the GPU tests compare with, against torch's
own functions and differences, and the refusals of the entry point (no call here reaches a kernel)."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import _distill as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VP, U64, I32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int
OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
A = 0x10000000  # fake, aligned device addresses; never dereferenced
G = 1 << 32     # far apart
F32, BF16 = 0, 1


def inputs(T=5, V=40, K=7):
    rng = np.random.default_rng(T + V + K)
    return (rng.normal(size=(T, V)) * 3, rng.integers(0, V, size=(T, K)), rng.normal(size=(T, K)) * 2, rng.integers(0, V, size=T),
            rng.random(T))


def test_plain_loss_matches_torch():
    z, idx, t, y, w = inputs()
    for temp, soft, hard in [(1.0, 1.0, 0.0), (2.0, 4.0, 0.5), (0.7, 0.0, 1.0)]:
        loss, grad, _, _ = ref.distill(z, idx, t, y, w, temp, soft, hard, 0.25)
        zt = torch.from_numpy(z).requires_grad_()
        q = torch.zeros(z.shape, dtype=torch.float64)
        q.scatter_add_(1, torch.from_numpy(idx), torch.softmax(torch.from_numpy(t) / temp, 1))
        logq = torch.log_softmax(torch.from_numpy(t) / temp, 1)
        own = (torch.softmax(torch.from_numpy(t) / temp, 1) * logq).sum(1)
        kl = own - (q * torch.log_softmax(zt / temp, 1)).sum(1)
        ce = torch.nn.functional.cross_entropy(zt, torch.from_numpy(y), reduction="none")
        want = torch.from_numpy(w) * (soft * kl + hard * ce)
        (want.sum() * 0.25).backward()
        np.testing.assert_allclose(loss, want.detach().numpy(), rtol=1e-12, atol=1e-14)
        np.testing.assert_allclose(grad, zt.grad.numpy(), rtol=1e-10, atol=1e-14)


def test_plain_gradient_matches_differences():
    z, idx, t, y, w = inputs(3, 9, 4)
    _, grad, _, _ = ref.distill(z, idx, t, y, w, 1.5, 2.0, 0.5, 1.0)
    for j in range(9):
        d = np.zeros_like(z)
        d[:, j] = 1e-5
        up, down = (ref.distill(z + s * d, idx, t, y, w, 1.5, 2.0, 0.5, 1.0)[0] for s in (1, -1))
        np.testing.assert_allclose((up - down) / 2e-5, grad[:, j], rtol=1e-6, atol=1e-9)


class Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_float) for n in ("temperature", "soft", "hard", "scale")]


@pytest.fixture(scope="module")
def call():
    from sketch_compressed_sparse_gb300 import build

    f = ctypes.CDLL(build.build()).s2_distill
    f.argtypes, f.restype = [VP, I32, U64, U64, U64, VP, VP, U64, VP, VP, Params, VP, VP, I32, U64, VP], I32

    def one(z=A, dt=F32, T=10, V=100, ld=100, idx=A + G, t=A + 2 * G, K=5, y=A + 3 * G, w=A + 4 * G, temp=2.0, soft=1.0,
            hard=0.5, scale=1.0, loss=A + 5 * G, dz=A + 6 * G, ddt=BF16, ldd=100):
        return f(z, dt, T, V, ld, idx, t, K, y, w, Params(temp, soft, hard, scale), loss, dz, ddt, ldd, None)

    return one


def test_refusals(call):
    assert call(dt=2) == INVALID and call(ddt=-1) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        assert call(temp=bad) == INVALID
    for bad in (float("nan"), float("inf")):
        assert call(soft=bad) == INVALID and call(hard=bad) == INVALID and call(scale=bad) == INVALID
    assert call(ld=99) == INVALID and call(ldd=99) == INVALID
    assert call(z=None) == INVALID and call(idx=None) == INVALID and call(t=None) == INVALID and call(loss=None) == INVALID
    assert call(z=A + 2) == ALIGN and call(dz=A + 6 * G + 1) == ALIGN and call(dt=BF16, z=A + 1) == ALIGN
    for name, at in (("idx", 1), ("t", 2), ("y", 3), ("w", 4), ("loss", 5)):
        assert call(**{name: A + at * G + 2}) == ALIGN
    assert call(dz=A) == INVALID and call(dz=A + 3996) == INVALID  # over the logits
    assert call(loss=A + 6 * G + 16) == INVALID and call(loss=A + 3 * G) == INVALID and call(loss=A + 4 * G + 36) == INVALID
    assert call(dz=A + G + 196) == INVALID and call(dz=A + 2 * G) == INVALID
    assert call(K=8193) == UNSUP and call(T=1 << 31) == UNSUP and call(V=1 << 31, ld=1 << 31, ldd=1 << 31) == UNSUP
    assert call(T=0) == OK and call(T=0, z=None, loss=None) == OK


def test_binding_refusals():
    import sketch_compressed_sparse_gb300 as s2

    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        s2.s2_distill(z, None, None, torch.zeros(2))


def test_both_ways_of_calling_agree():
    """The extension's call and that by ctypes refuse the same: the parameters arrive."""
    code = ("import sketch_compressed_sparse_gb300 as s2\n"
            "if {0}: s2._CALLS_PATH = '/nowhere'\n"
            "f = s2._f('s2_distill')\n"
            "one = lambda t, so, h, sc: f(None, 0, 0, 5, 5, None, None, 0, None, None, t, so, h, sc, None, None, 0, 0, None)\n"
            "inf = float('inf')\n"
            "print([one(*v) for v in ((1.0, 1, 0.0, 2.0), (0.0, 1.0, 0.0, 1.0), (1.0, inf, 0.0, 1.0), (1.0, 0.0, inf, 1.0), (2, 0.0, 0.0, inf))])\n")
    for own in (0, 1):
        r = subprocess.run([sys.executable, "-c", code.format(own)], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.strip() == "[0, 1, 1, 1, 1]", r.stdout + r.stderr
