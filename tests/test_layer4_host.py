"""The 4-bit layer without a GPU: the plain implementation that the GPU tests compare with, and the
refusals of the entry points (no call here reaches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _layer4 as ref

VP, U64, I32, SZ = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_size_t
OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
A = 0x10000000  # fake, aligned device addresses; never dereferenced
G = 1 << 32     # far apart
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from sketch_compressed_sparse_gb300 import build

    return ctypes.CDLL(build.build())


def _fn(lib, name, args):
    f = getattr(lib, name)
    f.argtypes, f.restype = args, I32
    return f


def test_code_values():
    for c, v in enumerate(ref.VALUES):
        sign, ex, man = c >> 3, c >> 1 & 3, c & 1
        assert v == (-1) ** sign * (man * 0.5 if ex == 0 else (1 + man / 2) * 2.0 ** (ex - 1))


@pytest.mark.parametrize("v,c", [(0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499999, 1), (1.25, 2), (1.75, 4), (2.5, 4),
                                 (2.5000002, 5), (3.5, 6), (5.0, 6), (5.0000005, 7), (6.0, 7), (-0.25, 8), (-5.0, 14), (-0.0, 8)])
def test_nearest_code(v, c):
    assert ref.nearest_code(np.array([v]))[0] == c


@pytest.mark.parametrize("amax,e", [(6.0, 0), (6.1, 1), (1.0, -2), (1.5, -2), (1.5000001, -1), (0.0, -125), (1e-40, -125),
                                    (2.0 ** 127, 125), (1.5 * 2.0 ** 127, 125), (3.4028234e38, 126), (12.0, 1)])
def test_scale_rule(amax, e):
    x = np.zeros((1, 5))
    x[0, 3] = -np.float32(amax)
    assert int(ref.scale_bytes(x)[0, 0]) - 127 == e


def test_tile_places_are_all_different():
    at = ref.tile_place(np.arange(300)[:, None], np.arange(12)[None], 380)
    assert len(np.unique(at)) == at.size and at.max() < 3 * 3 * 512 and at.min() == 0
    # the first tile: rows 0, 32, 64, 96 and then 1, 33, ... of four blocks each
    assert [int(at[r, 0]) for r in (0, 32, 64, 96, 1)] == [0, 4, 8, 12, 16] and int(at[128, 0]) == 3 * 512


def test_scales_size(lib):
    f = _fn(lib, "s2_pack4_scales_size", [U64, U64, ctypes.POINTER(SZ)])
    b = SZ()
    for rows, cols, want in [(0, 10, 0), (10, 0, 0), (1, 1, 512), (128, 128, 512), (129, 128, 1024), (267735, 1024, 2092 * 8 * 512)]:
        assert f(rows, cols, ctypes.byref(b)) == OK and b.value == want
    assert f(1, 1, None) == INVALID and f(1 << 31, 1, ctypes.byref(b)) == UNSUP and f(1, 1 << 31, ctypes.byref(b)) == UNSUP


def test_pack_refusals(lib):
    f = _fn(lib, "s2_pack4", [VP, I32, U64, U64, U64, VP, U64, VP, VP])

    def call(x=A, dt=BF16, rows=100, cols=201, ldx=201, c=A + G, ldc=112, s=A + 2 * G):
        return f(x, dt, rows, cols, ldx, c, ldc, s, None)

    assert call(dt=2) == INVALID and call(dt=-1) == INVALID
    assert call(ldx=200) == INVALID
    assert call(x=None) == INVALID and call(c=None) == INVALID and call(s=None) == INVALID
    assert call(ldc=96) == INVALID           # rows would overlap
    assert call(ldc=104) == ALIGN            # not a multiple of 16
    assert call(c=A + G + 8) == ALIGN and call(s=A + 2 * G + 8) == ALIGN
    assert call(x=A + 1) == ALIGN and call(dt=F32, x=A + 2) == ALIGN
    assert call(c=A) == INVALID              # over the input
    assert call(s=A + G + 16) == INVALID     # scales inside the codes
    assert call(s=A + 32) == INVALID
    assert call(rows=1 << 31) == UNSUP and call(cols=1 << 31, ldx=1 << 31) == UNSUP and call(ldx=1 << 35) == UNSUP
    assert call(rows=1 << 30, cols=1 << 17, ldx=1 << 17, ldc=1 << 16) == UNSUP  # 2^33 tiles
    assert call(rows=0) == OK and call(cols=0) == OK and call(x=None, c=None, s=None, rows=0) == OK


def test_unpack_refusals(lib):
    f = _fn(lib, "s2_unpack4", [VP, U64, VP, U64, U64, VP, I32, U64, VP])

    def call(c=A, ldc=112, s=A + G, rows=100, cols=201, o=A + 2 * G, dt=F32, ldo=201):
        return f(c, ldc, s, rows, cols, o, dt, ldo, None)

    assert call(dt=9) == INVALID and call(ldo=200) == INVALID and call(ldc=96) == INVALID
    assert call(c=None) == INVALID and call(s=None) == INVALID and call(o=None) == INVALID
    assert call(c=A + 1) == ALIGN and call(ldc=105) == ALIGN and call(o=A + 2 * G + 2) == ALIGN and call(s=A + G + 4) == ALIGN
    assert call(o=A + 1600) == INVALID and call(o=A + G + 100) == INVALID
    assert call(rows=1 << 31) == UNSUP
    assert call(rows=0) == OK and call(cols=0) == OK


def test_matmul_refusals(lib):
    f = _fn(lib, "s2_matmul4", [VP, U64, VP, VP, U64, VP, U64, U64, U64, VP, I32, U64, VP])

    def call(x=A, ldx=128, xs=A + G, w=A + 2 * G, ldw=128, ws=A + 3 * G, M=10, N=30, K=251, y=A + 4 * G, dt=F32, ldy=30):
        return f(x, ldx, xs, w, ldw, ws, M, N, K, y, dt, ldy, None)

    assert call(dt=2) == INVALID
    assert call(ldx=112) == INVALID and call(ldw=112) == INVALID and call(ldy=29) == INVALID
    assert call(x=None) == INVALID and call(w=None) == INVALID and call(y=None) == INVALID
    assert call(xs=None) == INVALID and call(ws=None) == INVALID
    assert call(x=A + 8) == ALIGN and call(w=A + 2 * G + 1) == ALIGN and call(xs=A + G + 8) == ALIGN and call(ws=A + 3 * G + 4) == ALIGN
    assert call(ldx=136) == ALIGN and call(ldw=130) == ALIGN and call(y=A + 4 * G + 2) == ALIGN
    assert call(dt=BF16, y=A + 4 * G + 1) == ALIGN
    assert call(y=A + 16) == INVALID and call(y=A + 2 * G + 128) == INVALID and call(y=A + G + 4) == INVALID and call(y=A + 3 * G) == INVALID
    assert call(M=1 << 31) == UNSUP and call(N=1 << 31, ldy=1 << 31) == UNSUP and call(K=1 << 31, ldx=1 << 30, ldw=1 << 30) == UNSUP
    assert call(M=(1 << 31) - 1, N=4096, ldy=4096) == UNSUP  # tiles
    assert call(M=0) == OK and call(N=0) == OK
    assert call(M=0, y=None, x=None) == OK


def test_binding_allocates_rows_on_16_bytes():
    import sketch_compressed_sparse_gb300 as s2

    for rows, cols in [(1, 1), (3, 31), (3, 33), (130, 257), (0, 4)]:
        codes, scales = s2.alloc_pack4(rows, cols, device="cpu")
        assert codes.shape == (rows, (cols + 1) // 2) and (rows <= 1 or codes.stride(0) % 16 == 0)
        assert scales.numel() == s2.s2_pack4_scales_size(rows, cols)


def test_binding_refuses_host_tensors():
    import sketch_compressed_sparse_gb300 as s2

    codes, scales = s2.alloc_pack4(2, 4, device="cpu")
    with pytest.raises(ValueError):
        s2.s2_pack4(torch.zeros(2, 4), codes, scales)
    with pytest.raises(ValueError):
        s2.s2_unpack4(codes, scales, torch.zeros(2, 4))
    with pytest.raises(ValueError):
        s2.s2_matmul4(codes, scales, codes, scales, torch.zeros(2, 2))
