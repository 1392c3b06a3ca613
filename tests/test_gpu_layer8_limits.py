"""GPU tests of the 8-bit layer at the edges of what its calls take: the longest
sums."""
import pytest
import torch

from tests.test_gpu_layer8 import DEV

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2


def test_wgrad_of_many_tokens():
    """2^27 tokens, 262144 stages in each block of a cluster of eight. Output n has a gradient at every
    eighth token and feature k is 1 or 2, so every chunk's sum is a multiple of eight and the sums, at most
    2^25, are exact: all tokens are in them, once."""
    T, N, K = 1 << 27, 8, 16
    dy = torch.eye(8, dtype=torch.bfloat16, device=DEV).repeat(T // 8, 1)
    codes = torch.tensor([0x38, 0x40], dtype=torch.uint8, device=DEV).repeat(T, K // 2)
    scales = torch.full((T, 1), 127, dtype=torch.uint8, device=DEV)
    want = torch.tensor([1.0, 2.0], device=DEV).repeat(N, K // 2) * (T // 8)
    for dtype in (torch.float32, torch.bfloat16):
        dw = torch.empty((N, K), dtype=dtype, device=DEV)
        s2.s2_wgrad8(dy, codes, scales, dw)
        assert torch.equal(dw.float(), want)
    assert s2.s2_wait_faults() == 0
