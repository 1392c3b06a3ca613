"""GPU tests of the 8-bit layer at the edges of what its calls take: the longest
sums, single rows of any stride, and the count of waits that ran out."""
import numpy as np
import pytest
import torch

from tests import _layer8 as ref
from tests.test_gpu_layer8 import DEV, make

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


def one_row(codes, ld):
    """The same single row, as a matrix whose row stride is ld."""
    return codes.reshape(-1).as_strided((1, codes.shape[1]), (ld, 1))


@pytest.mark.parametrize("ld", [0, 1, 140, 141, 144])
def test_single_rows_of_any_stride(ld):
    """A matrix of one row has no next row: its row stride does not matter, as a contiguous [1, 140]
    has it. The products with one of 1.0 as the other factor are exact."""
    K = 140
    x = make(1, K, 1)
    want, want_s = ref.pack(x.double().numpy(), False)
    values = ref.unpack(want, want_s, False)
    room = torch.zeros((1, 256), dtype=torch.uint8, device=DEV)
    codes = one_row(room[:, :K], ld)
    scales = torch.empty((1, 2), dtype=torch.uint8, device=DEV)
    s2.s2_pack8(one_row(x.to(DEV), ld), codes, scales)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    out = one_row(torch.empty((1, 256), device=DEV)[:, :K], ld)
    s2.s2_unpack8(codes, scales, out)
    np.testing.assert_array_equal(out.double().cpu().numpy(), values)
    for N in (1, 24):
        dw = torch.empty((N, K), device=DEV)
        dy = one_row(torch.ones((1, 64), dtype=torch.bfloat16, device=DEV)[:, :N], ld)
        s2.s2_wgrad8(dy, codes, scales, dw)
        np.testing.assert_array_equal(dw.double().cpu().numpy(), np.repeat(values, N, 0))
    y = one_row(torch.empty((1, 256), device=DEV)[:, :1], ld)
    s2.s2_matmul8(codes, scales, codes, scales, y, "rows")
    sq = (values * values).sum()
    assert abs(y.item() - sq) <= (K + 41) * 2.0 ** -23 * sq


def test_wait_faults_waits_for_every_stream():
    """The count covers every call made before: also those on streams that do not wait for the default stream."""
    busy = torch.randn((8192, 8192), device=DEV)
    out = busy @ busy
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert s2.s2_wait_faults() == 0
    with torch.cuda.stream(side):
        for _ in range(30):
            torch.mm(busy, busy, out=out)
    assert s2.s2_wait_faults() == 0
    assert side.query()
