"""GPU tests of the 4-bit layer: packing, unpacking and the product of packed
matrices, against the plain float64 implementation in tests/_layer4.py.

Codes and scale bytes are compared bit for bit, unpacked values exactly.

Products: with x_k, w_k the exact values, the products x_k w_k are exact in
the tensor core (two 2-bit significands) and are added to float32
accumulators. Let A = sum |x_k w_k|. A step adds 64 products and the
accumulator; each of its terms may lose less than one unit in the last place
of float32 at the step's largest term, so a step loses less than
65 * 2^-23 * A. Splitting K among up to eight blocks, and chunks of 8192 k, add
a rounding each. So
    |y - exact| <= (65 * ceil(K/64) + 8 + K/8192) * 2^-23 * A          (float32)
A bfloat16 result of K <= 8192 is the float32 result rounded once to nearest,
and is compared with that bit for bit.
"""
import numpy as np
import pytest
import torch

from tests import _layer4 as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SENTINEL = 0xA5


def make(rows, cols, tag, dtype="f32", kind="normal"):
    rng = np.random.default_rng(tag)
    x = rng.normal(size=(rows, cols))
    if kind == "wide":  # magnitudes over the whole float range, zero blocks, signed zeros
        x *= 10.0 ** rng.uniform(-44, 37, size=x.shape)
        x[rng.random(x.shape) < 0.1] = -0.0
        x[::3] = 0.0
    if kind == "grid":  # halfway between codes, and codes
        x = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 4.0, -0.0, 0.125], size=x.shape)
        x *= rng.choice([-1.0, 1.0], size=x.shape) * 2.0 ** rng.integers(-20, 20, size=(rows, 1))
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def padded(rows, cols, extra=16, dtype=torch.uint8, fill=SENTINEL):
    """A matrix inside a larger one, filled, so that writes outside it show."""
    ld = -(-cols // 16) * 16 + extra
    whole = torch.full((rows + 1, ld), fill, dtype=dtype, device=DEV)
    return whole, whole[:rows, :cols]


def untouched(whole, rows, cols, fill=SENTINEL):
    w = whole.clone()
    w[:rows, :cols] = fill
    return bool((w == fill).all())


SIZES = [(1, 1), (1, 1024), (2, 8), (3, 127), (5, 128), (2, 129), (64, 7), (127, 300), (128, 128), (130, 257), (1000, 72),
         (257, 1031)]


def check_pack(x):
    rows, cols = x.shape
    codes_want, scales_want, values = ref.pack(x.double().cpu().numpy())
    whole, codes = padded(rows, (cols + 1) // 2)
    scales = torch.full((scales_want.size + 16,), SENTINEL, dtype=torch.uint8, device=DEV)
    s2.s2_pack4(x, codes, scales)
    np.testing.assert_array_equal(codes.cpu().numpy(), codes_want)
    np.testing.assert_array_equal(scales[:scales_want.size].cpu().numpy(), scales_want)
    assert untouched(whole, rows, (cols + 1) // 2) and bool((scales[scales_want.size:] == SENTINEL).all())
    return codes, scales, values


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack_and_unpack(rows, cols, dtype):
    for kind in ("normal", "wide", "grid"):
        x = make(rows, cols, rows * 7 + cols, dtype, kind)
        codes, scales, values = check_pack(x.to(DEV))
        # and back, exactly, in both types (a code times its scale has 2 significant bits)
        for out_t in (torch.float32, torch.bfloat16):
            wo, out = padded(rows, cols, extra=3, dtype=out_t, fill=7.0)
            s2.s2_unpack4(codes, scales, out)
            np.testing.assert_array_equal(out.double().cpu().numpy(), values)
            assert untouched(wo, rows, cols, 7.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ld,off", [(300, 0), (301, 0), (304, 1), (304, 8), (333, 3)])
def test_pack_strides_and_offsets(dtype, ld, off):
    """Rows of a larger matrix, at any offset and row length."""
    rows, cols = 70, 290
    big = make(rows, ld + off, ld, dtype).to(DEV)
    x = big.reshape(-1)[off:off + rows * ld].reshape(rows, ld)[:, :cols]
    codes, scales, values = check_pack(x)
    flat = torch.zeros(off + rows * ld, device=DEV, dtype=DT[dtype])
    out = flat[off:].reshape(rows, ld)[:, :cols]
    s2.s2_unpack4(codes, scales, out)
    np.testing.assert_array_equal(out.double().cpu().numpy(), values)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pack_not_finite(dtype):
    """A block with a NaN or an infinity is NaN as a whole; the others are as without them."""
    x = make(130, 260, 5, dtype)
    x[3, 5], x[4, 200], x[129, 259], x[7, 130] = float("nan"), float("inf"), float("-inf"), float("nan")
    x[7, 128] = float("inf")
    codes, scales, values = check_pack(x.to(DEV))
    out = torch.empty((130, 260), device=DEV)
    s2.s2_unpack4(codes, scales, out)
    bad = np.zeros((130, 260), bool)
    bad[3, :32] = bad[4, 192:224] = bad[129, 256:] = bad[7, 128:160] = True
    np.testing.assert_array_equal(np.isnan(out.cpu().numpy()), bad)
    np.testing.assert_array_equal(out.double().cpu().numpy(), values)


def test_unpack_every_code_and_byte():
    """All 16 codes under every scale byte: rows 0..127 of two rows of tiles are the bytes 0..255."""
    codes = torch.from_numpy(np.tile(ref.pairs(np.arange(16, dtype=np.uint8)[None]), (256, 2))).contiguous().to(DEV)
    sb = np.arange(256, dtype=np.uint8)
    scales = torch.from_numpy(ref.tiled(sb[:, None], 32)).to(DEV)
    out = torch.empty((256, 32), device=DEV)
    s2.s2_unpack4(codes, scales, out)
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.tile(ref.VALUES, 2)[None] * np.exp2(sb.astype(np.float64) - 127)[:, None]
        want[255] = np.nan
        np.testing.assert_array_equal(out.cpu().numpy(), want.astype(np.float32))


def packed(x):
    codes, scales = s2.alloc_pack4(*x.shape)
    c, s, values = ref.pack(x.double().numpy())
    codes.copy_(torch.from_numpy(c))
    scales.copy_(torch.from_numpy(s))
    return codes, scales, values


def bound(K, A):
    return (65 * -(-K // 64) + 8 + K / 8192) * 2.0 ** -23 * A + 2.0 ** -149


def check_matmul(M, N, K, dtype, kind="normal", ldy_extra=0):
    x, w = make(M, K, M + 3 * K), make(N, K, N + 5 * K + 1)
    if kind == "mixed":  # block scales that differ by row and by block of K
        rng = np.random.default_rng(K)
        x = x * torch.from_numpy(2.0 ** rng.integers(-12, 12, size=(M, ref.blocks(K))).repeat(32, 1)[:, :K]).float()
        w = w * torch.from_numpy(2.0 ** rng.integers(-12, 12, size=(N, ref.blocks(K))).repeat(32, 1)[:, :K]).float()
        x[::4] = 0
    xc, xs, xv = packed(x)
    wc, ws, wv = packed(w)
    flat = torch.full((M * (N + ldy_extra) + 5,), 3.0, dtype=DT[dtype], device=DEV)
    y = flat[1:1 + M * (N + ldy_extra)].reshape(M, N + ldy_extra)[:, :N]
    s2.s2_matmul4(xc, xs, wc, ws, y)
    y32 = y
    if dtype == "bf16":
        y32 = torch.empty((M, N), device=DEV)
        s2.s2_matmul4(xc, xs, wc, ws, y32)
        assert torch.equal(y, y32.to(torch.bfloat16))
    got = y32.double().cpu().numpy()
    want, A = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    err = np.abs(got - want)
    tol = bound(K, A)
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-300))} of the bound"
    y.fill_(3.0)
    assert bool((flat == 3.0).all()), "wrote outside y"
    assert s2.s2_wait_faults() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 192, 225, 300, 385])
def test_matmul_tokens(M, dtype):
    """Every choice of the token tile, one token among them."""
    check_matmul(M, 300, 650, dtype, "mixed")


@pytest.mark.parametrize("N,K", [(1, 1), (1, 128), (7, 31), (128, 127), (129, 129), (64, 16), (130, 512), (1000, 513),
                                 (333, 1024), (2000, 2056), (50, 5000)])
@pytest.mark.parametrize("M", [1, 40, 260])
def test_matmul_sizes(M, N, K):
    check_matmul(M, N, K, "f32", ldy_extra=N % 3)


def test_matmul_many_tiles():
    """More tiles than SMs: every block takes several, in both tile orders."""
    check_matmul(3, 40000, 200, "bf16", "mixed")
    check_matmul(2000, 2100, 300, "f32", "mixed")
    check_matmul(5000, 700, 256, "bf16", "mixed")
    check_matmul(20000, 250, 384, "f32", "mixed")
    check_matmul(230, 40001, 650, "bf16", "mixed")
    check_matmul(9001, 1030, 700, "f32", "mixed")


@pytest.mark.parametrize("M,N,K", [(1, 256, 66000), (40, 700, 33001), (64, 20000, 16400), (300, 1000, 140000), (1100, 1100, 132000)])
def test_matmul_long_sums(M, N, K):
    """A long float32 sum loses no more than one of 8192 products: each of its 128 additions of 64 drops
    at most 2^-23 of the sum so far, which is at most the chunk's own on average; the chunks and a
    split sum's parts are added with rounding (2^-24 each, of random sign). A bfloat16 result may be
    one sum: 2^-23 for each of its additions, and its own rounding, half of 2^-8. Every result is the
    same on every run."""
    codes, scales, values = [], [], []
    for rows, step in ((M, 1 + M // 40), (N, 1 + N // 40)):
        g = torch.Generator(device=DEV).manual_seed(rows + K)
        c, b = s2.alloc_pack4(rows, K)
        s2.s2_pack4(torch.randn((rows, K), device=DEV, generator=g), c, b)
        v = torch.empty((rows, K), device=DEV)
        s2.s2_unpack4(c, b, v)
        codes.append(c)
        scales.append(b)
        values.append((torch.arange(0, rows, step), v[::step].double().cpu().numpy()))
        del v
    (i, xv), (j, wv) = values
    want = xv @ wv.T
    for dtype, tol in (("f32", (128 + (K / 8192 + 9) ** 0.5) * 2.0 ** -23), ("bf16", min(K, 131072) / 64 * 2.0 ** -23 + 2.0 ** -9)):
        y = torch.full((M, N + 1), 3.0, dtype=DT[dtype], device=DEV)
        s2.s2_matmul4(codes[0], scales[0], codes[1], scales[1], y[:, :N])
        got = y.double().cpu().numpy()
        assert (got[:, N] == 3.0).all()
        err = np.linalg.norm(got[np.ix_(i.numpy(), j.numpy())] - want) / np.linalg.norm(want)
        assert err <= tol, (dtype, err)
        again = torch.empty((M, N), dtype=DT[dtype], device=DEV)
        for _ in range(3):
            s2.s2_matmul4(codes[0], scales[0], codes[1], scales[1], again)
            assert torch.equal(again, y[:, :N])
    assert s2.s2_wait_faults() == 0


def test_matmul_empty():
    codes = torch.zeros((4, 16), dtype=torch.uint8, device=DEV)
    none = codes[:, :0]
    y = torch.full((4, 6), 5.0, device=DEV)[:, :4]
    nos = torch.zeros(0, dtype=torch.uint8, device=DEV)
    s2.s2_matmul4(none, nos, none, nos, y)  # K = 0: an empty sum
    assert bool((y == 0).all())
    s2.s2_matmul4(codes[:0], nos, codes, torch.zeros(512, dtype=torch.uint8, device=DEV), y[:0])


@pytest.mark.parametrize("M", [3, 40, 300])
def test_matmul_not_finite(M):
    """A NaN block reaches the outputs of its row and no other."""
    x, w = make(M, 300, 1), make(250, 300, 2)
    x[2, 290], w[11, 3], w[129, 299] = float("nan"), float("inf"), float("nan")
    xc, xs, _ = packed(x)
    wc, ws, _ = packed(w)
    y = torch.empty((M, 250), device=DEV)
    s2.s2_matmul4(xc, xs, wc, ws, y)
    want = torch.zeros((M, 250), dtype=torch.bool)
    want[2] = True
    want[:, [11, 129]] = True
    assert torch.equal(torch.isnan(y).cpu(), want)


def test_matmul_of_what_pack_wrote():
    """Codes and scales straight from s2_pack4, into memory that held NaN scales and codes before."""
    M, N, K = 70, 1000, 333
    x, w = make(M, K, 3), make(N, K, 4)
    got = []
    for t in (x, w):
        codes, scales = s2.alloc_pack4(*t.shape)
        codes.fill_(0xff)
        scales.fill_(0xff)
        s2.s2_pack4(t.to(DEV), codes, scales)
        got += [codes, scales]
    y = torch.empty((M, N), device=DEV)
    s2.s2_matmul4(*got, y)
    xv, wv = ref.pack(x.double().numpy())[2], ref.pack(w.double().numpy())[2]
    assert (np.abs(y.double().cpu().numpy() - xv @ wv.T) <= bound(K, np.abs(xv) @ np.abs(wv).T)).all()


@pytest.mark.parametrize("rows,width", [(1, 512), (200, 640)])
def test_stream_order(rows, width):
    """Every kernel reads what the one before it wrote and overwrites what an earlier one read, 40 times
    without a wait, also as a graph and between other kernels: the bits of the same calls with a wait
    after each."""
    wc, ws, _ = packed(make(width, width, 1) / width ** 0.5)
    start = make(rows, width, 2, "bf16").to(DEV)
    x = torch.zeros((rows, width), dtype=torch.bfloat16, device=DEV)
    codes, scales = s2.alloc_pack4(rows, width)
    back = torch.zeros((rows, width), device=DEV)

    def chain(between):
        x.copy_(start)
        for i in range(40):
            s2.s2_pack4(x, codes, scales)
            between()
            s2.s2_matmul4(codes, scales, wc, ws, x)
            between()
            s2.s2_unpack4(codes, scales, back)
            between()
            if i % 4 == 3:  # another library's kernels on both sides
                x.add_(back.to(torch.bfloat16))
                between()

    chain(torch.cuda.synchronize)
    want = [t.clone() for t in (x, back, codes, scales)]
    for _ in range(5):
        chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(want, (x, back, codes, scales)))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (x, back, codes, scales)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros((rows, width), dtype=torch.bfloat16, device=DEV)
    s2.s2_pack4(start, codes, scales)
    torch.cuda.synchronize()
    s2.s2_matmul4(codes, scales, wc, ws, y, stream=side)
    side.synchronize()
    z = torch.zeros_like(y)
    s2.s2_matmul4(codes, scales, wc, ws, z)
    assert torch.equal(y, z) and s2.s2_wait_faults() == 0


def test_offsets_past_32_bits():
    """Rows so far apart that every array's last offset passes 2^32 elements or bytes."""
    far = (1 << 31) + 16
    M, N, K = 3, 150, 200
    x, w = make(M, K, 1), make(N, K, 2)
    wide = torch.empty((M - 1) * far + K, dtype=torch.float32, device=DEV).as_strided((M, K), (far, 1))
    wide.copy_(x)
    codes = torch.empty((M - 1) * far + K, dtype=torch.uint8, device=DEV).as_strided((M, K // 2), (far, 1))
    scales = torch.empty(1024, dtype=torch.uint8, device=DEV)
    s2.s2_pack4(wide, codes, scales)
    want, want_s, xv = ref.pack(x.double().numpy())
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    s2.s2_unpack4(codes, scales, wide)
    np.testing.assert_array_equal(wide.double().cpu().numpy(), xv)
    del wide
    wc, ws, wv = packed(w)
    y = torch.empty((M - 1) * far + N, dtype=torch.bfloat16, device=DEV).as_strided((M, N), (far, 1))
    y32 = torch.empty((M, N), device=DEV)
    s2.s2_matmul4(codes, scales, wc, ws, y)
    s2.s2_matmul4(codes, scales, wc, ws, y32)
    assert torch.equal(y, y32.to(torch.bfloat16))
    assert (np.abs(y32.double().cpu().numpy() - xv @ wv.T) <= bound(K, np.abs(xv) @ np.abs(wv).T)).all()


def test_large_matrix():
    """More elements than 32 bits count: rows at the start, past 2^31 and at the end."""
    rows, cols = (1 << 32) // 4096 + 7, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    some = [0, 5, rows // 2 + 3, rows - 130, rows - 1]
    part = make(len(some), cols, 1, "bf16")
    x[some] = part.to(DEV)
    codes, scales = s2.alloc_pack4(rows, cols)
    s2.s2_pack4(x, codes, scales)
    x.fill_(3.0)
    s2.s2_unpack4(codes, scales, x)
    np.testing.assert_array_equal(x[some].double().cpu().numpy(), ref.pack(part.double().numpy())[2])
    assert int(torch.count_nonzero(x.view(torch.int16).any(dim=1))) == len(some)


def test_binding_refusals():
    codes, scales = s2.alloc_pack4(8, 64)
    x = torch.zeros((8, 64), device=DEV)
    with pytest.raises(TypeError):
        s2.s2_pack4(x.half(), codes, scales)
    with pytest.raises(ValueError):
        s2.s2_pack4(x.t(), codes, scales)
    with pytest.raises(ValueError):
        s2.s2_pack4(x[:7], codes, scales)
    with pytest.raises(ValueError):
        s2.s2_pack4(x, codes, scales[:400])
    with pytest.raises(ValueError):
        s2.s2_pack4(x[:, :62], codes, scales)
    with pytest.raises(s2.S2Error) as e:
        s2.s2_pack4(x[:, :40], codes.reshape(-1)[:8 * 20].reshape(8, 20), scales)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        s2.s2_matmul4(codes, scales, codes[:, :30], scales, x)
    with pytest.raises(ValueError):
        s2.s2_matmul4(codes, scales, codes, scales, x)
