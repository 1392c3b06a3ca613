"""Sizes that no memory holds are refused as unsupported, before any launch (no GPU needed: the
addresses are fake and never dereferenced)."""
import ctypes

import pytest

UNSUP = 3
VP, U64, I32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int
F32, BF16, ROWS, TILES = 0, 1, 0, 1
# 2^58 apart, so that even these matrices lie beside one another
A = [0x10000000 + (i << 58) for i in range(6)]
MOST = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    from sketch_compressed_sparse_gb300 import build

    lib = ctypes.CDLL(build.build())
    for name, args in (("s2_pack8", [VP, I32, U64, U64, U64, I32, VP, U64, VP, VP, U64, VP, VP]),
                       ("s2_unpack8", [VP, U64, VP, I32, U64, U64, VP, I32, U64, VP]),
                       ("s2_matmul8", [VP, U64, VP, VP, U64, VP, I32, U64, U64, U64, VP, I32, U64, VP]),
                       ("s2_wgrad8", [VP, U64, VP, U64, VP, U64, U64, U64, VP, I32, U64, I32, VP])):
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, I32
    return lib


def up16(n):
    return -(-n // 16) * 16


@pytest.mark.parametrize("M,N", [(1 << 30, 1 << 30), (MOST, 1 << 20), (1 << 20, MOST), (1 << 21, 1 << 21)])
def test_matmul_tiles(lib, M, N):
    """ceil(M / 16) * ceil(N / 128) has to be below 2^31."""
    assert lib.s2_matmul8(A[0], 128, A[1], A[2], 128, A[3], TILES, M, N, 128, A[4], BF16, N, None) == UNSUP


@pytest.mark.parametrize("T,N,K", [(1, 1 << 30, 1 << 30), (64, MOST, 1 << 16), (1 << 24, 1 << 19, 1 << 19), (1 << 30, 1 << 17, 1 << 17)])
def test_wgrad_tiles(lib, T, N, K):
    """ceil(N / 32) * ceil(K / 128) has to be below 2^31, and that times ceil(T / 64) below 2^36."""
    assert lib.s2_wgrad8(A[0], N, A[1], up16(K), A[2], T, N, K, A[3], BF16, K, 0, None) == UNSUP


def test_rows_too_far_apart(lib):
    """First to last row: at most 2^48 elements, of any matrix."""
    far = 1 << 34
    rows = (1 << 14) + 2
    assert lib.s2_unpack8(A[0], 16, A[1], ROWS, rows, 8, A[2], F32, far, None) == UNSUP
    assert lib.s2_unpack8(A[0], far, A[1], ROWS, rows, 8, A[2], F32, 8, None) == UNSUP
    assert lib.s2_pack8(A[0], F32, rows, 8, far, ROWS, A[1], 16, A[2], None, 0, None, None) == UNSUP
    assert lib.s2_pack8(A[0], F32, 8, rows, rows, TILES, A[1], up16(rows), A[2], A[3], far, A[4], None) == UNSUP
    assert lib.s2_matmul8(A[0], far, A[1], A[2], 128, A[3], TILES, rows, 8, 8, A[4], F32, 8, None) == UNSUP
    assert lib.s2_matmul8(A[0], 16, A[1], A[2], far, A[3], TILES, 8, rows, 8, A[4], F32, rows, None) == UNSUP
    assert lib.s2_wgrad8(A[0], far, A[1], 16, A[2], rows, 8, 8, A[3], F32, 8, 0, None) == UNSUP
