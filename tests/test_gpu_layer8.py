"""GPU tests of the 8-bit layer: packing, unpacking and the product of packed
matrices, against the plain float64 implementation in tests/_layer8.py.

Codes and scale bytes are compared bit for bit, unpacked values exactly.

Products: with x_k, w_k the exact values, the products x_k w_k are exact in
the tensor core (two 4-bit significands) and are added to float32
accumulators. Let A = sum |x_k w_k|. A step adds 32 products and the
accumulator; each of its terms may lose less than one unit in the last place
of float32 at the step's largest term, so a step loses less than
33 * 2^-23 * (largest partial magnitude <= A). That would give a bound of
33 * K/32 * 2^-23 * A; terms lost from below the accumulator's last place are
of random sign, but no use is made of that. Splitting K among up to eight
blocks adds eight float32 roundings. So
    |y - exact| <= (K + 33 + 8) * 2^-23 * A          (float32)
A bfloat16 result is the float32 result rounded once to nearest, and is
compared with that bit for bit.

Weight gradients: the products dy x (8 and 4 significant bits) are exact, a
step adds 16 of them and the accumulator, so likewise
    |dw - exact| <= (17/16 T + 17 + 8 + 2) * 2^-23 * (A + |what was there|),
the last two for the addition to what was there.
"""
import numpy as np
import pytest
import torch

from tests import _layer8 as ref

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
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    return t


def padded(rows, cols, extra=16, dtype=torch.uint8, fill=SENTINEL):
    """A matrix inside a larger one, filled, so that writes outside it show."""
    ld = -(-cols // 16) * 16 + extra
    whole = torch.full((rows + 1, ld), fill, dtype=dtype, device=DEV)
    return whole, whole[:rows, :cols]


def untouched(whole, rows, cols, fill=SENTINEL):
    w = whole.clone()
    w[:rows, :cols] = fill
    return bool((w == fill).all())


SIZES = [(1, 1), (1, 1024), (3, 127), (5, 128), (2, 129), (64, 7), (127, 300), (128, 128), (130, 257), (1000, 72),
         (257, 1031)]


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack_and_unpack(rows, cols, dtype, tiles):
    lay = "tiles" if tiles else "rows"
    for kind in ("normal", "wide"):
        x = make(rows, cols, rows * 7 + cols, dtype, kind)
        want, want_s = ref.pack(x.double().numpy(), tiles)
        whole, codes = padded(rows, cols)
        scales = torch.full((want_s.size + 3,), SENTINEL, dtype=torch.uint8, device=DEV)
        extra = {}
        if tiles:
            whole_t, codes_t = padded(cols, rows)
            scales_t = torch.full((want_s.size + 3,), SENTINEL, dtype=torch.uint8, device=DEV)
            extra = {"codes_t": codes_t, "scales_t": scales_t}
        s2.s2_pack8(x.to(DEV), codes, scales, lay, **extra)
        np.testing.assert_array_equal(codes.cpu().numpy(), want)
        np.testing.assert_array_equal(scales[:want_s.size].cpu().numpy(), want_s.reshape(-1))
        assert untouched(whole, rows, cols) and bool((scales[want_s.size:] == SENTINEL).all())
        if tiles:
            np.testing.assert_array_equal(codes_t.cpu().numpy(), want.T)
            np.testing.assert_array_equal(scales_t[:want_s.size].cpu().numpy(), want_s.T.reshape(-1))
            assert untouched(whole_t, cols, rows) and bool((scales_t[want_s.size:] == SENTINEL).all())
        # and back, exactly, in both types (a code times its scale has 4 significant bits)
        for out_t in (torch.float32, torch.bfloat16):
            wo, out = padded(rows, cols, extra=3, dtype=out_t, fill=7.0)
            s2.s2_unpack8(codes, scales, out, lay)
            np.testing.assert_array_equal(out.double().cpu().numpy(), ref.unpack(want, want_s, tiles))
            assert untouched(wo, rows, cols, 7.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ld,off", [(300, 0), (301, 0), (304, 1), (304, 8), (333, 3)])
def test_pack_strides_and_offsets(dtype, ld, off):
    """Rows of a larger matrix, at any offset and row length."""
    rows, cols = 70, 290
    big = make(rows, ld + off, ld, dtype).to(DEV)
    x = big.reshape(-1)[off:off + rows * ld].reshape(rows, ld)[:, :cols]
    for lay in ("rows", "tiles"):
        codes, scales = s2.alloc_pack8(rows, cols, lay)
        s2.s2_pack8(x, codes, scales, lay)
        want, want_s = ref.pack(x.double().cpu().numpy(), lay == "tiles")
        np.testing.assert_array_equal(codes.cpu().numpy(), want)
        np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
        flat = torch.zeros(off + rows * ld, device=DEV, dtype=DT[dtype])
        out = flat[off:].reshape(rows, ld)[:, :cols]
        s2.s2_unpack8(codes, scales, out, lay)
        np.testing.assert_array_equal(out.double().cpu().numpy(), ref.unpack(want, want_s, lay == "tiles"))


@pytest.mark.parametrize("tiles", [False, True])
def test_pack_not_finite(tiles):
    """NaN and infinities become NaN codes; the rest of their block is as without them."""
    x = make(130, 260, 5)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[3, 5] = bad[4, 200] = bad[129, 259] = bad[7, 128:256] = True
    y = x.clone()
    y[bad] = torch.tensor([float("nan"), float("inf"), float("-inf")]).repeat(100)[:int(bad.sum())]
    y[7, 128:256] = float("inf")  # a row's block with nothing finite
    codes, scales = s2.alloc_pack8(130, 260, "tiles" if tiles else "rows")
    s2.s2_pack8(y.to(DEV), codes, scales, "tiles" if tiles else "rows")
    want, want_s = ref.pack(y.double().numpy(), tiles)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    out = torch.empty((130, 260), device=DEV)
    s2.s2_unpack8(codes, scales, out, "tiles" if tiles else "rows")
    assert torch.equal(torch.isnan(out).cpu(), bad)


def test_unpack_every_code_and_byte():
    """All 256 codes under every scale byte whose values float32 holds exactly (2^-9 * 2^(b-127) normal), and byte 255."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).reshape(1, 256).repeat(246, 1).contiguous().to(DEV)
    sb = torch.arange(10, 256, dtype=torch.int32).to(torch.uint8)
    scales = sb.reshape(-1, 1).repeat(1, 2).contiguous().to(DEV)
    out = torch.empty((246, 256), device=DEV)
    s2.s2_unpack8(codes, scales, out)
    want = ref.VALUES[None, :] * np.exp2(sb.numpy().astype(np.float64) - 127)[:, None]
    want[-1] = np.nan
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(out.cpu().numpy(), want.astype(np.float32))


def packed(x, lay):
    codes, scales = s2.alloc_pack8(*x.shape, lay)
    c, s = ref.pack(x.double().numpy(), lay == "tiles")
    codes.copy_(torch.from_numpy(c))
    scales.copy_(torch.from_numpy(s))
    return codes, scales, ref.unpack(c, s, lay == "tiles")


def bound(K, A):
    return (K + 41) * 2.0 ** -23 * A + 2.0 ** -149


def check_matmul(M, N, K, dtype, w_lay, kind="normal", ldy_extra=0):
    x, w = make(M, K, M + 3 * K), make(N, K, N + 5 * K + 1)
    if kind == "mixed":  # block scales that differ by row and by block of K
        rng = np.random.default_rng(K)
        x = x * torch.from_numpy(2.0 ** rng.integers(-12, 12, size=(M, ref.blocks(K))).repeat(128, 1)[:, :K]).float()
        w = w * torch.from_numpy(2.0 ** rng.integers(-12, 12, size=(N, ref.blocks(K))).repeat(128, 1)[:, :K]).float()
        x[::4] = 0
    xc, xs, xv = packed(x, "rows")
    wc, ws, wv = packed(w, w_lay)
    flat = torch.full((M * (N + ldy_extra) + 5,), 3.0, dtype=DT[dtype], device=DEV)
    y = flat[1:1 + M * (N + ldy_extra)].reshape(M, N + ldy_extra)[:, :N]
    s2.s2_matmul8(xc, xs, wc, ws, y, w_lay)
    y32 = y
    if dtype == "bf16":
        y32 = torch.empty((M, N), device=DEV)
        s2.s2_matmul8(xc, xs, wc, ws, y32, w_lay)
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
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 225, 300])
def test_matmul_tokens(M, dtype):
    """Every choice of the token tile, one token among them."""
    check_matmul(M, 300, 650, dtype, "tiles")


@pytest.mark.parametrize("N,K", [(1, 1), (1, 128), (7, 31), (128, 127), (129, 129), (64, 16), (130, 512), (1000, 513),
                                 (333, 1024), (2000, 2056), (50, 5000)])
@pytest.mark.parametrize("M", [1, 40, 260])
def test_matmul_sizes(M, N, K):
    check_matmul(M, N, K, "f32", "tiles", ldy_extra=N % 3)


@pytest.mark.parametrize("w_lay", ["rows", "tiles"])
@pytest.mark.parametrize("M,N,K", [(1, 256, 2048), (20, 500, 1100), (250, 400, 900)])
def test_matmul_scales(M, N, K, w_lay):
    """Scales that differ from row to row and block to block, and zero rows."""
    check_matmul(M, N, K, "f32", w_lay, kind="mixed")


def test_matmul_many_tiles():
    """More tiles than SMs: every block takes several, in both tile orders."""
    check_matmul(3, 40000, 200, "bf16", "tiles")
    check_matmul(2000, 2100, 300, "f32", "tiles")
    check_matmul(5000, 700, 256, "bf16", "tiles")
    check_matmul(20000, 250, 384, "f32", "rows", kind="mixed")
    check_matmul(230, 40001, 650, "bf16", "tiles", kind="mixed")
    check_matmul(9001, 1030, 700, "f32", "rows", kind="mixed")


@pytest.mark.parametrize("M,N,K", [(1, 256, 66000), (40, 700, 33001), (64, 20000, 8200), (300, 1000, 65536),
                                   (1100, 1100, 65536), (700, 1601, 65000)])
def test_matmul_long_sums(M, N, K):
    """A long float32 sum loses no more than one of 4096 products: each of its 128 additions of 32
    products drops on average half a unit, at most 2^-24 of the sum so far, which is at most the
    chunk's own on average; the chunks and a split sum's parts are added with rounding (another 2^-24
    each, of random sign). A bfloat16 result is one sum: 2^-24 for each of its additions, and its own
    rounding, half of 2^-8."""
    codes, scales, values = [], [], []
    for rows, lay, step in ((M, "rows", 1 + M // 40), (N, "tiles", 1 + N // 40)):
        g = torch.Generator(device=DEV).manual_seed(rows + K)
        c, b = s2.alloc_pack8(rows, K, lay)
        s2.s2_pack8(torch.randn((rows, K), device=DEV, generator=g), c, b, lay)
        some = torch.arange(0, rows, step)
        codes.append(c)
        scales.append(b)
        of = some // 128 if lay == "tiles" else some
        v = ref.VALUES[c[some].cpu().numpy()] * ref.spread(b[of].cpu().numpy(), len(some), K, False)
        values.append((some, v))
    (i, xv), (j, wv) = values
    want = xv @ wv.T
    for dtype, tol in (("f32", (128 + (K / 4096 + 9) ** 0.5) * 2.0 ** -24), ("bf16", K / 32 * 2.0 ** -24 + 2.0 ** -9)):
        y = torch.full((M, N + 1), 3.0, dtype=DT[dtype], device=DEV)
        s2.s2_matmul8(codes[0], scales[0], codes[1], scales[1], y[:, :N])
        got = y.double().cpu().numpy()
        assert (got[:, N] == 3.0).all()
        err = np.linalg.norm(got[np.ix_(i.numpy(), j.numpy())] - want) / np.linalg.norm(want)
        assert err <= tol, (dtype, err)
        again = torch.empty((M, N), dtype=DT[dtype], device=DEV)
        for _ in range(5):
            s2.s2_matmul8(codes[0], scales[0], codes[1], scales[1], again)
            assert torch.equal(again, y[:, :N])
    assert s2.s2_wait_faults() == 0


def test_matmul_empty():
    codes = torch.zeros((4, 16), dtype=torch.uint8, device=DEV)
    none = codes[:, :0]
    y = torch.full((4, 6), 5.0, device=DEV)[:, :4]
    nos = torch.zeros(0, dtype=torch.uint8, device=DEV)
    s2.s2_matmul8(none, nos, none, nos, y)  # K = 0: an empty sum
    assert bool((y == 0).all())
    s2.s2_matmul8(codes[:0], nos, codes, torch.zeros((1, 1), dtype=torch.uint8, device=DEV), y[:0])


def test_matmul_not_finite():
    """A NaN code reaches the outputs of its row and no other."""
    xc, xs, _ = packed(make(40, 300, 1), "rows")
    wc, ws, _ = packed(make(50, 300, 2), "tiles")
    xc[7, 290] = 0x7f
    wc[11, 3] = 0xff
    y = torch.empty((40, 50), device=DEV)
    s2.s2_matmul8(xc, xs, wc, ws, y)
    bad = torch.isnan(y).cpu()
    want = torch.zeros((40, 50), dtype=torch.bool)
    want[7] = True
    want[:, 11] = True
    assert torch.equal(bad, want)


def test_matmul_repeats_and_streams():
    """The same bits on every run, and on a side stream."""
    xc, xs, _ = packed(make(9, 4096, 1), "rows")
    wc, ws, _ = packed(make(1024, 4096, 2), "tiles")
    outs = []
    for i in range(4):
        y = torch.empty((9, 1024), device=DEV)
        st = torch.cuda.Stream() if i % 2 else torch.cuda.current_stream()
        st.wait_stream(torch.cuda.current_stream())
        s2.s2_matmul8(xc, xs, wc, ws, y, stream=st)
        torch.cuda.synchronize()
        outs.append(y)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_input_gradient_from_transposed_weight():
    """dX = dY W from the transposed codes that packing a weight by tiles also writes."""
    T, N, K = 70, 300, 200
    w = make(N, K, 3)
    codes, scales = s2.alloc_pack8(N, K, "tiles")
    codes_t, scales_t = s2.alloc_pack8(K, N, "tiles")
    s2.s2_pack8(w.to(DEV), codes, scales, "tiles", codes_t, scales_t)
    gc, gs, gv = packed(make(T, N, 4), "rows")
    dx = torch.empty((T, K), device=DEV)
    s2.s2_matmul8(gc, gs, codes_t, scales_t, dx)
    wv = ref.unpack(*ref.pack(w.double().numpy(), True), True)
    want, A = gv @ wv, np.abs(gv) @ np.abs(wv)
    assert (np.abs(dx.double().cpu().numpy() - want) <= bound(N, A)).all()


def check_wgrad(T, N, K, dtype="f32", dy_off=0, dy_extra=0, dw_extra=0, accumulate=False, kind="normal"):
    xc, xs, xv = packed(make(T, K, T + K, kind=kind), "rows")
    ld = N + dy_extra
    flat = torch.full((dy_off + T * ld,), float("nan"), dtype=torch.bfloat16, device=DEV)
    dy = flat[dy_off:].reshape(T, ld)[:, :N]
    dy.copy_(make(T, N, T + N + 1, "bf16"))
    out = torch.full((N * (K + dw_extra) + 5,), 3.0, dtype=DT[dtype], device=DEV)
    dw = out[1:1 + N * (K + dw_extra)].reshape(N, K + dw_extra)[:, :K]
    prior = np.zeros((N, K))
    if accumulate:
        dw.copy_(make(N, K, 9, dtype))
        prior = dw.double().cpu().numpy()
    dw32 = dw.float() if dtype == "bf16" else dw
    s2.s2_wgrad8(dy, xc, xs, dw, accumulate)
    if dtype == "bf16":
        s2.s2_wgrad8(dy, xc, xs, dw32, accumulate)
        assert torch.equal(dw, dw32.to(torch.bfloat16))
    yv = dy.double().cpu().numpy()
    want, A = yv.T @ xv + prior, np.abs(yv).T @ np.abs(xv) + np.abs(prior)
    err = np.abs(dw32.double().cpu().numpy() - want)
    tol = (17 / 16 * T + 27) * 2.0 ** -23 * A + 2.0 ** -149
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-300))} of the bound"
    dw.fill_(3.0)
    assert bool((out == 3.0).all()), "wrote outside dw"
    assert s2.s2_wait_faults() == 0


@pytest.mark.parametrize("T", [1, 2, 15, 16, 63, 64, 65, 130, 511, 1000])
@pytest.mark.parametrize("N,K", [(1, 1), (8, 16), (64, 128), (65, 129), (7, 300), (200, 96), (333, 257)])
def test_wgrad_sizes(T, N, K):
    check_wgrad(T, N, K, dw_extra=N % 2)


@pytest.mark.parametrize("off,extra", [(0, 0), (0, 1), (1, 0), (3, 2), (5, 3), (7, 7), (8, 4), (2, 8), (0, 8)])
@pytest.mark.parametrize("N", [300, 328])
def test_wgrad_strides(N, off, extra):
    """dY at every kind of misalignment; what lies between its rows is NaN and must not matter."""
    check_wgrad(150, N, 200, dy_off=off, dy_extra=extra)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N", [104, 333])
def test_wgrad_types(N, accumulate, dtype):
    check_wgrad(300, N, 250, dtype, accumulate=accumulate)


@pytest.mark.parametrize("T", [1, 3, 7, 8, 9, 70, 600])
@pytest.mark.parametrize("N", [129, 20001])
def test_wgrad_few_tokens_unaligned(T, N):
    """Fewer tokens than residues, and first rows that are not finite where no token follows."""
    check_wgrad(T, N, 100)
    xc, xs, _ = packed(make(T, 100, 1), "rows")
    dy = make(T, N, 2, "bf16").to(DEV)
    dy[0, 5] = float("inf")
    dw = torch.empty((N, 100), device=DEV)
    s2.s2_wgrad8(dy, xc, xs, dw)
    bad = ~torch.isfinite(dw)
    assert bool(bad[5].any()) and int(bad.any(1).sum()) == 1


@pytest.mark.parametrize("T", [513, 1100, 2100, 4500])
@pytest.mark.parametrize("N,extra", [(128, 0), (130, 1)])
def test_wgrad_split_tokens(T, N, extra):
    """Few tiles and many tokens: every size of cluster."""
    check_wgrad(T, N, 130, dy_extra=extra)
    check_wgrad(T, N, 130, "bf16", dy_extra=extra, accumulate=True)


@pytest.mark.parametrize("N,extra", [(2500, 0), (2501, 0), (2049, 3)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_many_tiles(N, extra, accumulate):
    """More tiles than SMs, in aligned and unaligned rows."""
    check_wgrad(200, N, 4000, dy_extra=extra, accumulate=accumulate)
    check_wgrad(70, 40 * N, 128, "bf16", dy_extra=extra, accumulate=accumulate)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 131, 259), (5, 16, 128), (40, 4500, 1001), (300, 2001, 2500), (900, 100, 70)])
def test_wgrad_accumulate(T, N, K, dtype):
    """dw += over single blocks, pairs and split tokens, with columns and rows past the last tile."""
    check_wgrad(T, N, K, dtype, dy_extra=-N % 8, dw_extra=3, accumulate=True)
    check_wgrad(T, N, K, dtype, dw_extra=1, accumulate=True)


@pytest.mark.parametrize("T,N,K", [(2, 40, 200), (500, 64, 128), (300, 2001, 2500)])
def test_wgrad_accumulate_keeps_subnormals(T, N, K):
    """Adding zeros leaves every number as it is, those below the least normal one too."""
    xc, xs, _ = packed(make(T, K, 1), "rows")
    dy = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    for dtype, bits in ((torch.float32, torch.int32), (torch.bfloat16, torch.int16)):
        dw = torch.arange(1, N * K + 1, dtype=torch.int32, device=DEV).remainder(127).to(bits).reshape(N, K).contiguous()
        want = dw.clone()
        s2.s2_wgrad8(dy, xc, xs, dw.view(dtype), accumulate=True)
        assert torch.equal(dw, want)


@pytest.mark.parametrize("N", [264, 301])
def test_wgrad_long_sums(N):
    """A long float32 sum loses no more than one of 704 tokens: each of its 44 additions of 16
    tokens drops on average half a unit, at most 2^-24 of the sum so far, which is at most the
    chunk's own on average; the chunks are added with rounding (another 2^-24 each, of random sign)."""
    T, K = 6000, 260
    xc, xs, xv = packed(make(T, K, 1), "rows")
    dy = make(T, N, 2, "bf16")
    dw = torch.empty((N, K), device=DEV)
    s2.s2_wgrad8(dy.to(DEV), xc, xs, dw)
    want = dy.double().numpy().T @ xv
    err = np.linalg.norm(dw.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= (44 + 9 ** 0.5) * 2.0 ** -24


def test_wgrad_empty():
    dw = torch.full((5, 7), 2.0, device=DEV)[:, :6]
    dy = torch.zeros((0, 5), dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((0, 6), dtype=torch.uint8, device=DEV)
    nos = torch.zeros(0, dtype=torch.uint8, device=DEV)
    s2.s2_wgrad8(dy, x, nos, dw, True)
    assert bool((dw == 2).all())
    s2.s2_wgrad8(dy, x, nos, dw)
    assert bool((dw == 0).all())


def test_wgrad_masked_tokens():
    """Tokens without gradient, among them whole blocks of 64, and without activation."""
    T, N, K = 400, 130, 140
    x = make(T, K, 1)
    x[5:9] = 0
    dy = make(T, N, 2, "bf16")
    dy[64:200] = 0
    xc, xs, xv = packed(x, "rows")
    dw = torch.empty((N, K), device=DEV)
    s2.s2_wgrad8(dy.to(DEV), xc, xs, dw)
    yv = dy.double().numpy()
    tol = (17 / 16 * T + 27) * 2.0 ** -23 * (np.abs(yv).T @ np.abs(xv))
    assert (np.abs(dw.double().cpu().numpy() - yv.T @ xv) <= tol + 2.0 ** -149).all()
    s2.s2_wgrad8(torch.zeros_like(dy).to(DEV), xc, xs, dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("N", [128, 129])
def test_wgrad_not_finite(N):
    """A NaN activation reaches its column of dW, a NaN gradient its row, and nothing else."""
    xc, xs, _ = packed(make(100, 200, 1), "rows")
    xc[33, 150] = 0x7f
    dy = make(100, N, 2, "bf16").to(DEV)
    dy[70, 11] = float("nan")
    dw = torch.empty((N, 200), device=DEV)
    s2.s2_wgrad8(dy, xc, xs, dw)
    want = torch.zeros((N, 200), dtype=torch.bool)
    want[:, 150] = True
    want[11] = True
    assert torch.equal(torch.isnan(dw).cpu(), want)


def test_wgrad_scale_range():
    """Activations over the whole range of the scales: 2^-117 and 2^120 are exact in bfloat16."""
    x = torch.zeros((2, 256))
    x[0, :128], x[0, 128:] = 3.0e38, 1.0e-38
    x[1, :128], x[1, 128:] = 1.0, 2.0 ** -126
    codes, scales = s2.alloc_pack8(2, 256)
    s2.s2_pack8(x.to(DEV), codes, scales)
    assert scales.cpu().tolist() == [[247, 10], [119, 10]]
    v = torch.empty((2, 256), device=DEV)
    s2.s2_unpack8(codes, scales, v)
    dw = torch.empty((2, 256), device=DEV)
    s2.s2_wgrad8(torch.eye(2, dtype=torch.bfloat16, device=DEV), codes, scales, dw)
    assert torch.equal(dw, v)


@pytest.mark.parametrize("extra", [0, 1])
def test_wgrad_every_code_and_byte(extra):
    """dY = 1: dW holds X's values exactly, for every code (NaN aside) under every byte that packing writes."""
    n = 238
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(n, 1)
    codes[:, [0x7f, 0xff]] = 0
    scales = torch.arange(10, 248, dtype=torch.int32).to(torch.uint8).reshape(-1, 1).repeat(1, 2).contiguous()
    want = ref.unpack(codes.numpy(), scales.numpy(), False)
    with np.errstate(over="ignore"):
        want = np.where(np.abs(want) >= 2.0 ** 128, 0.0, want)  # past float32: left out
    codes = torch.where(torch.from_numpy(want == 0), torch.zeros_like(codes), codes)
    dy = torch.zeros((n, 20000 + extra), dtype=torch.bfloat16, device=DEV)  # wide enough for every form
    dy[:, :n] = torch.eye(n)
    for N in (n + extra, 20000 + extra):
        dw = torch.empty((N, 256), device=DEV)
        s2.s2_wgrad8(dy[:, :N] if extra else dy[:, :N].contiguous(), codes.to(DEV), scales.to(DEV), dw)
        np.testing.assert_array_equal(dw[:n].double().cpu().numpy(), want)
        assert bool((dw[n:] == 0).all())


@pytest.mark.parametrize("N", [512, 515])
def test_wgrad_repeats_and_streams(N):
    xc, xs, _ = packed(make(1000, 500, 1), "rows")
    dy = make(1000, N, 2, "bf16").to(DEV)
    outs = []
    for i in range(4):
        dw = torch.empty((N, 500), device=DEV)
        st = torch.cuda.Stream() if i % 2 else torch.cuda.current_stream()
        st.wait_stream(torch.cuda.current_stream())
        s2.s2_wgrad8(dy, xc, xs, dw, stream=st)
        torch.cuda.synchronize()
        outs.append(dw)
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("T,N,K", [(600, 20001, 100), (640, 20000, 100), (2000, 20001, 128), (700, 9001, 520)])
def test_wgrad_same_bits_from_cold_caches(T, N, K):
    """Copies that come late and early, in every order, give the same bits: L2 flushed before every other run."""
    xc, xs, xv = packed(make(T, K, 1), "rows")
    dy = make(T, N, 2, "bf16").to(DEV)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    first, dw = torch.empty((N, K), device=DEV), torch.empty((N, K), device=DEV)
    s2.s2_wgrad8(dy, xc, xs, first)
    yv = dy.double().cpu().numpy()
    tol = (17 / 16 * T + 27) * 2.0 ** -23 * (np.abs(yv).T @ np.abs(xv)) + 2.0 ** -149
    assert (np.abs(first.double().cpu().numpy() - yv.T @ xv) <= tol).all()
    for i in range(100):
        if i % 2:
            flush.fill_(i)
        dw.fill_(7.0)
        s2.s2_wgrad8(dy, xc, xs, dw)
        assert torch.equal(dw, first), f"run {i}"


@pytest.mark.parametrize("M,N,K", [(24, 20001, 1024), (100, 20000, 700), (500, 9001, 2048)])
def test_matmul_same_bits_from_cold_caches(M, N, K):
    xc, xs, _ = packed(make(M, K, 1), "rows")
    wc, ws, _ = packed(make(N, K, 2), "tiles")
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    first, y = torch.empty((M, N), device=DEV), torch.empty((M, N), device=DEV)
    s2.s2_matmul8(xc, xs, wc, ws, first)
    for i in range(100):
        if i % 2:
            flush.fill_(i)
        y.fill_(7.0)
        s2.s2_matmul8(xc, xs, wc, ws, y)
        assert torch.equal(y, first), f"run {i}"


@pytest.mark.parametrize("rows,width", [(1, 512), (200, 700), (2500, 1536)])
def test_stream_order(rows, width):
    """Every kernel reads what the one before it wrote and overwrites what an earlier one read, 40
    times without a wait, also as a graph and between other kernels: the bits of the same calls
    with a wait after each."""
    wc, ws, _ = packed(make(width, width, 1) / width ** 0.5, "tiles")
    start = make(rows, width, 2, "bf16").to(DEV)
    pad = -(-width // 8) * 8
    x = torch.zeros((rows, pad), dtype=torch.bfloat16, device=DEV)[:, :width]
    codes, scales = s2.alloc_pack8(rows, width)
    back, dw = torch.zeros((rows, width), device=DEV), torch.zeros((width, width), device=DEV)

    def chain(between):
        x.copy_(start)
        dw.zero_()
        for i in range(40):
            s2.s2_pack8(x, codes, scales)
            between()
            s2.s2_matmul8(codes, scales, wc, ws, x)
            between()
            s2.s2_wgrad8(x, codes, scales, dw, accumulate=True)
            between()
            s2.s2_unpack8(codes, scales, back)
            between()
            if i % 4 == 3:  # another library's kernels on both sides
                x.add_(back.to(torch.bfloat16))
                between()

    chain(torch.cuda.synchronize)
    want = [t.clone() for t in (x, back, dw, codes, scales)]
    for _ in range(5):
        chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(want, (x, back, dw, codes, scales)))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain(lambda: None)
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (x, back, dw, codes, scales)))
    assert s2.s2_wait_faults() == 0


def test_waits_for_other_streams():
    """A call after a wait for another stream's event reads what that stream wrote, although the
    kernel before it in its own stream lets it start early; also over the legacy default stream."""
    rows, width = 300, 640
    wc, ws, _ = packed(make(512, width, 1), "tiles")
    busy = torch.randn((4096, 4096), device=DEV)
    inputs = [make(rows, width, 10 + i).to(DEV) for i in range(8)]
    want = []
    for v in inputs:
        c, b = s2.alloc_pack8(rows, width)
        s2.s2_pack8(v, c, b)
        y = torch.empty((rows, 512), device=DEV)
        s2.s2_matmul8(c, b, wc, ws, y)
        want.append((c.clone(), y))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for own in (torch.cuda.current_stream(), torch.cuda.Stream()):
        x = torch.zeros((rows, width), device=DEV)
        c, b = s2.alloc_pack8(rows, width)
        other = s2.alloc_pack8(rows, width)
        y = torch.empty((rows, 512), device=DEV)
        torch.cuda.synchronize()
        for v, (codes, out) in zip(inputs, want):
            with torch.cuda.stream(side):
                side.wait_stream(own)
                for _ in range(3):
                    busy.mm(busy)
                x.copy_(v)
            with torch.cuda.stream(own):
                s2.s2_pack8(inputs[0], *other, stream=own)
                own.wait_stream(side)
                s2.s2_pack8(x, c, b, stream=own)
                s2.s2_matmul8(c, b, wc, ws, y, stream=own)
                own.synchronize()
            assert torch.equal(c, codes) and torch.equal(y, out)


def test_wgrad_against_differences():
    """L(W) = sum(G * (X W^T)) is linear in W: its central difference along a direction D of packed
    weights is <dL/dW, D>. Both sides in float64 from the operators' float32 outputs:
    each y is off by at most (K + 41) 2^-23 A_y and each dw by (17/16 T + 27) 2^-23 A_w."""
    T, N, K = 90, 70, 200
    xc, xs, xv = packed(make(T, K, 1), "rows")
    g = make(T, N, 2, "bf16")
    w, d = make(N, K, 3), make(N, K, 4)
    gv = g.double().numpy()
    dw = torch.empty((N, K), device=DEV)
    s2.s2_wgrad8(g.to(DEV), xc, xs, dw)
    loss, wv, room = [], [], 0.0
    for sign in (1, -1):
        wc, ws, v = packed(w + sign * d, "tiles")
        y = torch.empty((T, N), device=DEV)
        s2.s2_matmul8(xc, xs, wc, ws, y)
        loss.append((gv * y.double().cpu().numpy()).sum())
        wv.append(v)
        room += (np.abs(gv) * bound(K, np.abs(xv) @ np.abs(v).T)).sum()
    step = wv[0] - wv[1]
    room += (np.abs(step) * (17 / 16 * T + 27) * 2.0 ** -23 * (np.abs(gv).T @ np.abs(xv))).sum()
    assert abs((loss[0] - loss[1]) - (dw.double().cpu().numpy() * step).sum()) <= room


@pytest.mark.parametrize("off", [0, 1, 3, 8])
@pytest.mark.parametrize("T", [1, 2, 9])
def test_wgrad_one_row_anywhere(T, off):
    check_wgrad(T, 77, 140, dy_off=off)


def test_offsets_past_32_bits():
    """Rows so far apart that every array's last offset passes 2^32 elements or bytes."""
    far = (1 << 31) + 16
    T, N, K = 3, 150, 200
    x, w, g = make(T, K, 1), make(N, K, 2), make(T, N, 3, "bf16")
    wide = torch.empty((T - 1) * far + K, dtype=torch.float32, device=DEV).as_strided((T, K), (far, 1))
    wide.copy_(x)
    codes = torch.empty((T - 1) * far + K, dtype=torch.uint8, device=DEV).as_strided((T, K), (far, 1))
    scales = torch.empty((T, 2), dtype=torch.uint8, device=DEV)
    s2.s2_pack8(wide, codes, scales)
    want, want_s = ref.pack(x.double().numpy(), False)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    xv = ref.unpack(want, want_s, False)
    s2.s2_unpack8(codes, scales, wide)
    np.testing.assert_array_equal(wide.double().cpu().numpy(), xv)
    del wide
    wc, ws, wv = packed(w, "tiles")
    y = torch.empty((T - 1) * far + N, dtype=torch.bfloat16, device=DEV).as_strided((T, N), (far, 1))
    y32 = torch.empty((T, N), device=DEV)
    s2.s2_matmul8(codes, scales, wc, ws, y)
    s2.s2_matmul8(codes, scales, wc, ws, y32)
    assert torch.equal(y, y32.to(torch.bfloat16))
    assert (np.abs(y32.double().cpu().numpy() - xv @ wv.T) <= bound(K, np.abs(xv) @ np.abs(wv).T)).all()
    y.copy_(g)
    dw = torch.empty((N, K), device=DEV)
    for dy in (y, torch.empty((T - 1) * (far + 1) + N, dtype=torch.bfloat16, device=DEV).as_strided((T, N), (far + 1, 1))):
        dy.copy_(g)
        s2.s2_wgrad8(dy, codes, scales, dw)
        yv = g.double().numpy()
        tol = (17 / 16 * T + 27) * 2.0 ** -23 * (np.abs(yv).T @ np.abs(xv)) + 2.0 ** -149
        assert (np.abs(dw.double().cpu().numpy() - yv.T @ xv) <= tol).all()
        del dy
    far_dw = torch.empty((N - 1) * (1 << 25) + K, device=DEV).as_strided((N, K), (1 << 25, 1))
    s2.s2_wgrad8(g.to(DEV), codes, scales, far_dw)
    assert torch.equal(far_dw, dw)


def test_binding_refusals():
    codes, scales = s2.alloc_pack8(8, 64)
    x = torch.zeros((8, 64), device=DEV)
    with pytest.raises(TypeError):
        s2.s2_pack8(x.half(), codes, scales)
    with pytest.raises(ValueError):
        s2.s2_pack8(x.t(), codes, scales)
    with pytest.raises(ValueError):
        s2.s2_pack8(x[:7], codes, scales)
    with pytest.raises(ValueError):
        s2.s2_pack8(x, codes, scales[:4])
    with pytest.raises(s2.S2Error) as e:
        s2.s2_pack8(x[:, :40], codes.reshape(-1)[:8 * 40].reshape(8, 40), scales)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        s2.s2_matmul8(codes, scales, codes[:, :48], scales, x)
