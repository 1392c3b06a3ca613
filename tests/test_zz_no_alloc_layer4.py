"""The 4-bit layer's calls allocate nothing on the device: one shape for each form that a call can
take, made once (which loads its kernel) and then again, with the free memory unchanged."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def packed(rows, cols):
    import sketch_compressed_sparse_gb300 as s2

    codes, scales = s2.alloc_pack4(rows, cols)
    s2.s2_pack4(torch.randn((rows, cols), device=DEV), codes, scales)
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
@pytest.mark.parametrize("rows,cols", [(1, 1024), (300, 700), (300, 704)])
def test_pack_and_unpack(rows, cols, dtype):
    import sketch_compressed_sparse_gb300 as s2

    x = torch.randn((rows, cols), device=DEV).to(dtype)
    codes, scales = s2.alloc_pack4(rows, cols)
    check(lambda: s2.s2_pack4(x, codes, scales))
    check(lambda: s2.s2_unpack4(codes, scales, x))


# every width of token tile, split and not; pairs; sums in chunks; an empty sum
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (24, 20000, 1024), (64, 20000, 512), (100, 20000, 512), (300, 2000, 256),
                                   (2000, 4000, 512), (1, 256, 132096), (64, 20000, 16384), (1100, 1100, 132096), (30, 50, 0)])
def test_matmul(M, N, K, dtype):
    import sketch_compressed_sparse_gb300 as s2

    (x, xs), (w, ws) = packed(M, K), packed(N, K)
    y = torch.empty((M, N), dtype=dtype, device=DEV)
    check(lambda: s2.s2_matmul4(x, xs, w, ws, y))
