"""The 8-bit layer without a GPU: the plain implementation that the GPU tests
compare with, against hand-computed values and torch's own e4m3 type, and the
refusals of the entry points (no call here reaches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _layer8 as ref

VP, U64, I32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int
OK, INVALID, ALIGN, UNSUP = 0, 1, 2, 3
A = 0x10000000  # fake, aligned device addresses; never dereferenced
G = 1 << 32     # far apart
F32, BF16, ROWS, TILES = 0, 1, 0, 1


@pytest.fixture(scope="module")
def lib():
    from sketch_compressed_sparse_gb300 import build

    return ctypes.CDLL(build.build())


def test_code_values_match_torch():
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.VALUES, want)


def test_nearest_code_matches_torch():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.uniform(-4, 2.6, size=4000), ref.VALUES[:127],
                        (ref.VALUES[:126] + ref.VALUES[1:127]) / 2, -(ref.VALUES[:126] + ref.VALUES[1:127]) / 2])
    v = v[np.abs(v) <= 448].astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.nearest_code(v.astype(np.float64)), want)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.1, 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (0.0, -117),
                                    (1e-40, -117), (2.0 ** 127, 119), (3.4028234e38, 120), (896.0, 1)])
def test_scale_rule(amax, e):
    x = np.zeros((1, 5))
    x[0, 3] = -np.float32(amax)
    assert int(ref.scale_bytes(x, False)[0, 0]) - 127 == e


def _fn(lib, name, args):
    f = getattr(lib, name)
    f.argtypes, f.restype = args, I32
    return f


def test_pack_refusals(lib):
    f = _fn(lib, "s2_pack8", [VP, I32, U64, U64, U64, I32, VP, U64, VP, VP, U64, VP, VP])

    def call(x=A, dt=BF16, rows=100, cols=200, ldx=200, lay=TILES, c=A + G, ldc=208, s=A + 2 * G, ct=A + 3 * G,
             ldct=112, st=A + 4 * G):
        return f(x, dt, rows, cols, ldx, lay, c, ldc, s, ct, ldct, st, None)

    assert call(dt=2) == INVALID
    assert call(lay=2) == INVALID
    assert call(ldx=199) == INVALID
    assert call(st=None) == INVALID          # one of the transposed pair
    assert call(ct=None) == INVALID
    assert call(lay=ROWS) == INVALID         # no transpose of row scales
    assert call(x=None) == INVALID and call(c=None) == INVALID and call(s=None) == INVALID
    assert call(ldc=199) == INVALID          # rows would overlap
    assert call(ldc=200) == ALIGN            # not a multiple of 16
    assert call(c=A + G + 8) == ALIGN
    assert call(ldct=100) == ALIGN
    assert call(ct=A + 3 * G + 4) == ALIGN
    assert call(x=A + 1) == ALIGN
    assert call(dt=F32, x=A + 2) == ALIGN
    assert call(c=A) == INVALID              # over the input
    assert call(s=A + G + 16) == INVALID     # scales inside the codes
    assert call(st=A + 2 * G) == INVALID
    assert call(rows=1 << 31) == UNSUP
    assert call(cols=1 << 31, ldx=1 << 31) == UNSUP
    assert call(rows=1 << 30, cols=1024, ldx=1024, lay=ROWS, ct=None, st=None) == UNSUP  # 2^33 blocks
    assert call(rows=0) == OK and call(cols=0) == OK
    assert call(x=None, rows=0) == OK


def test_unpack_refusals(lib):
    f = _fn(lib, "s2_unpack8", [VP, U64, VP, I32, U64, U64, VP, I32, U64, VP])

    def call(c=A, ldc=208, s=A + G, lay=ROWS, rows=100, cols=200, o=A + 2 * G, dt=F32, ldo=200):
        return f(c, ldc, s, lay, rows, cols, o, dt, ldo, None)

    assert call(lay=-1) == INVALID and call(dt=9) == INVALID
    assert call(ldo=150) == INVALID
    assert call(c=None) == INVALID and call(s=None) == INVALID and call(o=None) == INVALID
    assert call(c=A + 1) == ALIGN and call(ldc=201) == ALIGN and call(o=A + 2 * G + 2) == ALIGN
    assert call(o=A + 1600) == INVALID
    assert call(o=A + G + 100) == INVALID
    assert call(rows=1 << 31) == UNSUP
    assert call(rows=0) == OK


def test_matmul_refusals(lib):
    f = _fn(lib, "s2_matmul8", [VP, U64, VP, VP, U64, VP, I32, U64, U64, U64, VP, I32, U64, VP])

    def call(x=A, ldx=256, xs=A + G, w=A + 2 * G, ldw=256, ws=A + 3 * G, lay=TILES, M=10, N=30, K=250, y=A + 4 * G,
             dt=F32, ldy=30):
        return f(x, ldx, xs, w, ldw, ws, lay, M, N, K, y, dt, ldy, None)

    assert call(lay=2) == INVALID and call(dt=2) == INVALID
    assert call(ldx=240) == INVALID and call(ldw=240) == INVALID and call(ldy=29) == INVALID
    assert call(ldx=250) == ALIGN and call(ldw=250) == ALIGN
    assert call(x=A + 8) == ALIGN and call(w=A + 2 * G + 1) == ALIGN and call(y=A + 4 * G + 1) == ALIGN
    for k in ("x", "xs", "w", "ws", "y"):
        assert call(**{k: None}) == INVALID
    assert call(y=A + 256) == INVALID            # over X
    assert call(y=A + 2 * G + 512) == INVALID    # over W
    assert call(y=A + G) == INVALID and call(y=A + 3 * G) == INVALID
    assert call(M=1 << 31) == UNSUP and call(N=1 << 31, ldy=1 << 31) == UNSUP
    assert call(ldw=1 << 35) == UNSUP and call(ldy=1 << 35) == UNSUP
    assert call(M=0) == OK and call(N=0) == OK


def test_wgrad_refusals(lib):
    f = _fn(lib, "s2_wgrad8", [VP, U64, VP, U64, VP, U64, U64, U64, VP, I32, U64, I32, VP])

    def call(dy=A, lddy=30, x=A + G, ldx=256, xs=A + 2 * G, T=10, N=30, K=250, dw=A + 3 * G, dt=F32, lddw=250, acc=0):
        return f(dy, lddy, x, ldx, xs, T, N, K, dw, dt, lddw, acc, None)

    assert call(dt=2) == INVALID
    assert call(lddy=29) == INVALID and call(ldx=240) == INVALID and call(lddw=249) == INVALID
    assert call(ldx=250) == ALIGN and call(x=A + G + 4) == ALIGN
    assert call(dy=A + 1) == ALIGN and call(dw=A + 3 * G + 2) == ALIGN
    for k in ("dy", "x", "xs", "dw"):
        assert call(**{k: None}) == INVALID
    assert call(dw=A + 100) == INVALID           # over dY
    assert call(dw=A + G) == INVALID and call(dw=A + 2 * G) == INVALID
    assert call(T=1 << 31) == UNSUP and call(K=1 << 31, ldx=1 << 31, lddw=1 << 31) == UNSUP
    assert call(N=0) == OK and call(K=0) == OK
    assert call(T=0, acc=1) == OK                # adds nothing


def test_binding_checks():
    import sketch_compressed_sparse_gb300 as s2

    cpu = torch.zeros((4, 16), dtype=torch.uint8)
    with pytest.raises(ValueError):  # host tensors
        s2.s2_pack8(torch.zeros((4, 16)), cpu, cpu)
    with pytest.raises(ValueError):
        s2.s2_matmul8(cpu, cpu, cpu, cpu, torch.zeros((4, 4)))
    f = _fn(ctypes.CDLL(s2.lib_path()), "s2_wait_faults", [VP])
    assert f(None) == INVALID


def test_calls_without_ctypes():
    """The extension's calls are the library's: the statuses that ctypes gets, None as a null
    pointer, and errors for what is no argument list."""
    import os

    import sketch_compressed_sparse_gb300 as s2
    from sketch_compressed_sparse_gb300 import build

    if not os.path.exists(build.CALLS):
        pytest.skip("built without Python's headers")
    lib = ctypes.CDLL(s2.lib_path())
    cases = {
        "s2_pack8": [(None, 0, 0, 5, 5, 0, None, 16, None, None, 0, None, None),
                     (None, 0, 3, 5, 5, 0, None, 16, None, None, 0, None, None),
                     (16, 7, 3, 5, 5, 0, 32, 16, 64, None, 0, None, None),
                     (16, 0, 3, 5, 4, 0, 32, 16, 64, None, 0, None, None)],
        "s2_unpack8": [(None, 16, None, 0, 0, 5, None, 0, 5, None), (None, 16, None, 0, 3, 5, None, 0, 5, None),
                       (16, 16, 64, 9, 3, 5, 128, 0, 5, None)],
        "s2_matmul8": [(None, 16, None, None, 16, None, 1, 0, 4, 5, None, 0, 4, None),
                       (16, 16, 32, 64, 16, 96, 1, 2, 4, 5, 130, 0, 4, None),
                       (16, 16, 32, 64, 16, 96, 1, 2, 4, 5, None, 0, 4, 2 ** 63)],
        "s2_wgrad8": [(None, 4, None, 16, None, 2, 0, 5, None, 0, 5, 0, None),
                      (16, 4, 32, 16, 64, 2, 4, 5, None, 0, 5, 1, None),
                      (17, 4, 32, 16, 64, 2, 4, 5, 128, 0, 5, 1, None)],
    }
    for name, calls in cases.items():
        f = _fn(lib, name, s2._SIGS[name][0])
        for args in calls:
            assert s2._f(name)(*args) == f(*args), (name, args)
        n = len(s2._SIGS[name][0])
        with pytest.raises(TypeError):
            s2._f(name)(*(0,) * (n - 1))
        with pytest.raises(TypeError):
            s2._f(name)(*("x",) * n)
        with pytest.raises(OverflowError):
            s2._f(name)(*(2 ** 64,) * n)
