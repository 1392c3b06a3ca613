"""The GPU tests of s2_sample may leave out rows whose answer hangs on a rounding. No row of these inputs does, by the
64-bit implementation alone: every one is compared."""
import numpy as np
import pytest
import torch

from tests import test_gpu_sample as gpu
from tests._sample import sample


@pytest.fixture
def unclear(monkeypatch):
    """The tests' check without a GPU: rows that it would leave out."""
    rows = []

    def check(z, u, dtype="f32", ld=None, off=0, cleared=0.02, **kw):
        z = z if isinstance(z, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(z, dtype=np.float32))
        got = []
        for i, (l, v) in enumerate(zip(z.to(gpu.DT[dtype]).float().numpy(), np.asarray(u, np.float32))):
            token, clear = sample(l, v, **{k: a[i] for k, a in kw.items() if a is not None})
            got.append(token)
            if not clear:
                rows.append((i, {k: a[i] for k, a in kw.items()}))
        return np.array(got)

    monkeypatch.setattr(gpu, "check", check)
    return rows


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 3000])
def test_equal_logits(unclear, V, dtype):
    gpu.test_equal_logits(V, dtype)
    assert unclear == []


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 5000])
def test_masks_and_special_numbers(unclear, V, dtype):
    gpu.test_masks_and_special_numbers(V, dtype)
    assert unclear == []


@pytest.mark.filterwarnings("ignore")
def test_extreme_settings(unclear):
    gpu.test_extreme_settings()
    assert unclear == []
