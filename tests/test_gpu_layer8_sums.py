"""GPU tests of the 8-bit layer's long sums, in every form that its planners choose: sums split over
a cluster, tiles of one block, pairs of blocks, aligned and misaligned rows.

The tensor cores cut off what they add, on average half a unit, at most 2^-24 of a chunk's own sum,
for each of the chunk's additions: always towards zero, so that a bfloat16 result's own rounding
(2^-9 of the value in the mean square, of either sign) hides it in one output and not in the mean of many. With
n outputs the mean of sign(exact) (y - exact) over the mean of |exact| is therefore at most
    additions of a chunk * 2^-24 + 6 * 2^-9 / sqrt(n)
in magnitude, with six standard deviations (each below 2^-9 on average) for the roundings, whose sizes grow with
the outputs as |exact| does (their mean square over their squared mean is below 2: n is halved).

A float32 and a bfloat16 result are the same sums, rounded once more, only where both are one chunk
(up to 704 tokens in a block, up to 4096 of K); beyond, their chunks differ.
"""
import pytest
import torch

from tests import _layer8 as ref
from tests.test_gpu_layer8 import DEV

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2


def packed_here(rows, cols, seed, lay="rows"):
    """A packed normal matrix, on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes, scales = s2.alloc_pack8(rows, cols, lay)
    s2.s2_pack8(torch.randn((rows, cols), generator=g, device=DEV), codes, scales, lay)
    return codes, scales


def values(codes, scales, lay="rows"):
    """The values of a packed matrix in float64."""
    rows, cols = codes.shape
    s = torch.exp2(scales.double() - 127).repeat_interleave(128, 1)[:, :cols]
    if lay == "tiles":
        s = s.repeat_interleave(128, 0)[:rows]
    return torch.from_numpy(ref.VALUES).to(DEV)[codes.int()] * s


def normal(rows, cols, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((rows, cols), generator=g, device=DEV).to(dtype)


def drift(got, want):
    return abs(float(((got.double() - want) * want.sign()).mean() / want.abs().mean()))


def drift_bound(additions, n):
    return additions * 2.0 ** -24 + 6 * 2.0 ** -9 / (n / 2) ** 0.5


# split over a cluster, one block a tile, pairs; aligned and misaligned rows (on 152 SMs)
@pytest.mark.parametrize("T,N,K", [(1600000, 264, 260), (1600000, 263, 260), (60000, 9600, 256), (60000, 9601, 256),
                                   (48000, 4096, 1024), (48000, 4097, 1024)])
def test_wgrad_bfloat16_does_not_drift(T, N, K):
    """A bfloat16 result's chunks are 2048 tokens at most, 128 additions of 16."""
    xc, xs = packed_here(T, K, 1)
    dy = normal(T, N, 2, torch.bfloat16)
    dw = torch.empty((N, K), dtype=torch.bfloat16, device=DEV)
    s2.s2_wgrad8(dy, xc, xs, dw)
    want = dy.double().T @ values(xc, xs)
    assert drift(dw, want) <= drift_bound(128, N * K)
    assert float((dw.double() - want).norm() / want.norm()) <= 128 * 2.0 ** -24 + 2.0 ** -9
    assert s2.s2_wait_faults() == 0


# one block a tile, pairs (on 152 SMs)
@pytest.mark.parametrize("M,N,K", [(64, 20000, 131072), (2048, 1024, 267735)])
def test_matmul_bfloat16_does_not_drift(M, N, K):
    """Beyond 65536 of K a bfloat16 result's chunks are 4096 at most, 128 additions of 32."""
    xc, xs = packed_here(M, K, 1)
    wc, ws = packed_here(N, K, 2, "tiles")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    s2.s2_matmul8(xc, xs, wc, ws, y)
    want = torch.zeros((M, N), dtype=torch.float64, device=DEV)
    for k in range(0, K, 16384):
        b = slice(k // 128, (k + 16384) // 128)
        want += values(xc[:, k:k + 16384], xs[:, b]) @ values(wc[:, k:k + 16384], ws[:, b], "tiles").T
    assert drift(y, want) <= drift_bound(128, M * N)
    assert float((y.double() - want).norm() / want.norm()) <= 128 * 2.0 ** -24 + 2.0 ** -9
    assert s2.s2_wait_faults() == 0


# clusters of two to eight, one block a tile, pairs; aligned and misaligned rows (on 152 SMs)
@pytest.mark.parametrize("T,N,K", [(6000, 264, 260), (6000, 301, 260), (2100, 130, 130), (4500, 128, 130), (2000, 640, 520),
                                   (2000, 641, 520), (3000, 1496, 700), (3000, 1497, 700), (3000, 1200, 1100), (3000, 1201, 1100),
                                   (2000, 2504, 4000), (2000, 2501, 4000), (6000, 4096, 1024), (6000, 4097, 1024)])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_sums(T, N, K, accumulate, dtype):
    """44 additions of 16 in a chunk of a float32 result, 128 of a bfloat16 one; T/704 + 1 chunks, eight
    parts and what was there before at most, each added with a rounding; the last one 2^-9 in
    the mean square in bfloat16.
    A token that is left out or taken twice is off by about 1 / sqrt(T), 4000 times the float32 bound."""
    xc, xs = packed_here(T, K, 1)
    dy = normal(T, N, 2, torch.bfloat16)
    dw = normal(N, K, 3, dtype)
    want = dy.double().T @ values(xc, xs)
    size = want.norm()
    if accumulate:
        want += dw.double()
        size = size + dw.double().norm()
    s2.s2_wgrad8(dy, xc, xs, dw, accumulate)
    additions = 44 if dtype == torch.float32 else 128
    bound = (additions + (T / 704 + 1 + 8 + 1) ** 0.5) * 2.0 ** -24 + (2.0 ** -9 if dtype == torch.bfloat16 else 0)
    assert float((dw.double() - want).norm() / size) <= bound
    assert s2.s2_wait_faults() == 0
