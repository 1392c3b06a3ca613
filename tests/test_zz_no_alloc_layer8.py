"""The 8-bit layer's calls allocate nothing on the device: one shape for each form that a call can
take, made once (which loads its kernel) and then again, with the free memory unchanged."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def packed(rows, cols, lay="rows"):
    import sketch_compressed_sparse_gb300 as s2

    codes, scales = s2.alloc_pack8(rows, cols, lay)
    s2.s2_pack8(torch.randn((rows, cols), device=DEV), codes, scales, lay)
    return codes, scales


def check(call):
    call()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()) == before


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lay", ["rows", "tiles"])
@pytest.mark.parametrize("rows,cols", [(1, 1024), (300, 700), (300, 701)])
def test_pack_and_unpack(rows, cols, lay, dtype):
    import sketch_compressed_sparse_gb300 as s2

    x = torch.randn((rows, cols), device=DEV).to(dtype)
    codes, scales = s2.alloc_pack8(rows, cols, lay)
    t = s2.alloc_pack8(cols, rows, lay) if lay == "tiles" else ()
    check(lambda: s2.s2_pack8(x, codes, scales, lay, *t))
    check(lambda: s2.s2_unpack8(codes, scales, x, lay))


# every width of token tile, split and not; pairs; sums in chunks; an empty sum
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (24, 20000, 1024), (64, 20000, 512), (100, 20000, 512), (300, 2000, 256),
                                   (2000, 4000, 512), (1, 256, 66048), (64, 20000, 8192), (300, 1000, 66048), (1100, 1100, 66048),
                                   (30, 50, 0)])
def test_matmul(M, N, K, dtype):
    import sketch_compressed_sparse_gb300 as s2

    (x, xs), (w, ws) = packed(M, K), packed(N, K, "tiles")
    y = torch.empty((M, N), dtype=dtype, device=DEV)
    check(lambda: s2.s2_matmul8(x, xs, w, ws, y))


# split over clusters, one block a tile, pairs; aligned and misaligned rows; no tokens
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,N,K", [(6000, 264, 260), (6000, 263, 260), (3000, 1200, 1100), (3000, 1201, 1100), (3000, 4096, 1024),
                                   (3000, 4097, 1024), (0, 30, 40)])
def test_wgrad(T, N, K, dtype, accumulate):
    import sketch_compressed_sparse_gb300 as s2

    x, xs = packed(T, K)
    dy = torch.randn((T, N), device=DEV).to(BF16)
    dw = torch.zeros((N, K), dtype=dtype, device=DEV)
    check(lambda: s2.s2_wgrad8(dy, x, xs, dw, accumulate))
