"""GPU tests of s2_distill against the plain float64 implementation in tests/_distill.py.

Rounding: an exponential exp2(d * c), d = z - max, is off by at most 2^-22 of itself by its own
evaluation, and |d c| ln 2 times 2^-24 for each of d, c and their product; where |d c| passes 126 it may
be taken for 0. A thread adds up to V/512 + 16 of them, and 16 joins follow. So with X the largest |z -
max| / temperature that counts (at most 90) a probability is off by at most
    E = (4 + 3 X + V/512 + 32 + 4) * 2^-24
of itself, and a gradient by E times the sum of the magnitudes that make it up, and its own rounding, half
a step of its type. The loss is a sum of terms like q (log q - log p), each off by E times (|log q| + |log
p| + 1) q; the sum over K entries adds K/512 + 24 roundings, which E covers for the K taken here.
"""
import numpy as np
import pytest
import torch

from tests import _distill as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def np64(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def rows_at(T, V, dtype, ld=None, off=0, fill=5.0):
    """A matrix inside a larger buffer, `off` elements from an aligned address."""
    ld = V if ld is None else ld
    flat = torch.full((off + T * ld + 9,), fill, dtype=dtype, device=DEV)
    return flat, flat[off:off + T * ld].reshape(T, ld)[:, :V]


def make(T, V, K, tag=0, spread=3.0, repeat=False, missing=False, masked=False):
    rng = np.random.default_rng([T, V, K, tag])
    z = rng.normal(size=(T, V)) * spread
    if masked:
        z[rng.random((T, V)) < 0.3] = -np.inf
    idx = np.stack([rng.permutation(V)[:K] if V < 100000 else rng.integers(0, V, K) for _ in range(T)]) if K else np.zeros((T, 0), int)
    if repeat and K > 1:
        idx[:, rng.integers(0, K, 1 + K // 3)] = idx[:, :1]
    if missing and K:
        idx[rng.random((T, K)) < 0.3] = rng.choice([-1, V, -2 ** 31, 2 ** 31 - 1])
    t = rng.normal(size=(T, K)) * 3
    y = rng.integers(0, V, T)
    if missing:
        y[::3] = -1
    dev = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(d).to(DEV)  # noqa: E731
    return dev(z, torch.float32), dev(idx, torch.int32), dev(t, torch.float32), dev(y, torch.int32), dev(rng.random(T) + 0.5, torch.float32)


def check(z, idx, t, y, w, dtype="f32", ddtype="f32", temperature=1.0, soft=1.0, hard=0.0, scale=1.0, ld=None, off=0, ldd=None, offd=0):
    T, V = z.shape
    _, logits = rows_at(T, V, DT[dtype], ld, off)
    logits.copy_(z)
    z64 = np64(logits)
    loss = torch.full((T + 1,), 7.0, device=DEV)
    args = dict(targets=y, row_weight=w, temperature=temperature, soft=soft, hard=hard, scale=scale)
    want, dwant, room, droom = ref.distill(z64, np64(idx), np64(t), np64(y), np64(w), temperature, soft, hard, scale)
    with np.errstate(invalid="ignore"):
        x = np.where(np.isfinite(z64), z64.max(axis=1, keepdims=True) - z64, 0.0) / min(1.0, temperature)
    E = (4 + 3 * min(90.0, float(np.nanmax(x)) if x.size else 0.0) + V / 512 + 36) * 2.0 ** -24
    want = np.where(np.abs(want) > np.finfo(np.float32).max, np.copysign(np.inf, want), want)
    flat = None
    for grad in (True, False):
        d = None
        if grad:
            flat, d = rows_at(T, V, DT[ddtype], ldd, offd)
        s2.s2_distill(logits, idx, t, loss, d, **args)
        got = loss.double().cpu().numpy()
        assert got[T] == 7.0
        same = np.isfinite(want)
        np.testing.assert_array_equal(np.isfinite(got[:T]), same)
        np.testing.assert_array_equal(got[:T][~same], want[~same])  # infinities and NaN
        assert (np.abs(got[:T] - want)[same] <= (E * room + 2.0 ** -24 * np.abs(want))[same] + 1e-37).all(), np.max(np.abs(got[:T] - want)[same] / (E * room[same] + 1e-37))
        if grad:
            dgot = d.double().cpu().numpy()
            fine = np.isfinite(dwant)
            np.testing.assert_array_equal(np.isnan(dgot), np.isnan(dwant))
            tol = E * droom + STEP[ddtype] * np.abs(dwant) * 1.01 + 1e-37
            assert (np.abs(dgot - dwant)[fine] <= tol[fine]).all(), np.max((np.abs(dgot - dwant) / tol)[fine])
            d.fill_(5.0)
            assert bool((flat == 5.0).all()), "wrote outside dlogits"
    return want


@pytest.mark.parametrize("dtype,ddtype", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 7, 2), (5, 8, 8), (4, 9, 3), (2, 1000, 1), (300, 333, 5), (40, 4099, 64), (7, 33278, 100),
                                   (2, 267735, 64), (400, 2500, 17)])
def test_sizes_and_types(T, V, K, dtype, ddtype):
    z, idx, t, y, w = make(T, V, K)
    check(z, idx, t, y, w, dtype, ddtype, temperature=2.0, soft=4.0, hard=0.3, scale=1.0 / T)
    check(z, idx, t, y, None, dtype, ddtype, temperature=1.0, soft=1.0, hard=0.5)
    check(z, idx, t, None, None, dtype, ddtype, temperature=0.5, soft=1.0)


@pytest.mark.parametrize("dtype,ddtype", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("ld,off,ldd,offd", [(333, 0, 333, 0), (333, 3, 333, 3), (340, 1, 333, 0), (336, 8, 344, 0), (333, 0, 333, 5), (400, 7, 401, 2)])
def test_alignments(ld, off, ldd, offd, dtype, ddtype):
    """Rows that start anywhere, in both arrays."""
    z, idx, t, y, w = make(20, 333, 9)
    check(z, idx, t, y, w, dtype, ddtype, temperature=2.0, hard=0.3, ld=ld, off=off, ldd=ldd, offd=offd)


@pytest.mark.parametrize("V,K", [(50, 40), (700, 128), (900, 256), (5000, 257), (5000, 300), (70000, 1000)])
def test_repeated_and_missing_entries(V, K):
    """An index twice counts twice; one outside the row not at all; targets among the entries and not."""
    for kw in (dict(repeat=True), dict(missing=True), dict(repeat=True, missing=True)):
        z, idx, t, y, w = make(6, V, K, **kw)
        idx[2] = -1          # no teacher
        idx[4, :] = idx[4, 0] if int(idx[4, 0]) >= 0 else 3  # one word only
        y[1] = 3
        idx[1, K // 2] = 3   # the target is an entry
        check(z, idx, t, y, w, temperature=2.0, soft=2.0, hard=0.4)
        check(z, idx, t, y, w, "bf16", "bf16", temperature=1.0, hard=0.4)


def test_many_entries():
    z, idx, t, y, w = make(2, 20000, 8192, repeat=True)
    check(z, idx, t, y, w, temperature=2.0, hard=0.5)
    with pytest.raises(s2.S2Error):
        check(z, torch.zeros((2, 8193), dtype=torch.int32, device=DEV), torch.zeros((2, 8193), device=DEV), y, w)


@pytest.mark.parametrize("V", [40, 3000, 100003])
def test_masked_logits(V):
    """-infinity has no probability; entries there make the loss infinite; the type's lowest value is a number."""
    z, idx, t, y, w = make(8, V, 6, masked=True)
    z[0] = float("-inf")                    # nothing left
    z[1] = float("-inf")
    z[1, int(idx[1, 0])] = 0.5              # one word left
    z[2] = torch.finfo(torch.float32).min   # all the same, lowest
    z[3, ::2] = torch.finfo(torch.float32).min
    z[5, idx[5].long()] = 1.0               # every entry has probability
    z[6] = 3.0
    t[6] = float("-inf")                    # a teacher without weight
    t[5, 2] = float("-inf")
    y[6] = -1
    y[5] = idx[5, 1]
    for hard in (0.0, 0.5):
        want = check(z, idx, t, y, None, temperature=2.0, hard=hard)
        assert np.isinf(want[0]) and np.isfinite(want[[2, 5, 6]]).all() and want[6] == 0
    y[0] = -1
    idx[0] = -1
    assert check(z, idx, t, y, None, hard=0.5)[0] == 0


@pytest.mark.parametrize("V", [40, 3000])
def test_not_finite(V):
    """NaN and +infinity among the logits make a row NaN, a teacher's NaN the loss and its entries, and no
    other row; a weight of 0 leaves them out."""
    z, idx, t, y, _ = make(6, V, 6)
    z[1, 5], z[2, V - 1] = float("nan"), float("inf")
    t[3, 2] = float("nan")
    w = torch.ones(6, device=DEV)
    loss, d = torch.empty(6, device=DEV), torch.empty((6, V), device=DEV)
    s2.s2_distill(z, idx, t, loss, d, targets=y, row_weight=w, hard=0.5)
    bad = torch.tensor([False, True, True, True, False, False])
    assert torch.equal(torch.isnan(loss).cpu(), bad)
    assert torch.equal(torch.isnan(d).any(1).cpu(), bad) and bool(torch.isnan(d[1:3]).all())
    assert torch.equal(torch.isnan(d[3]).nonzero()[:, 0], idx[3].long().unique())
    w[1:4] = 0
    s2.s2_distill(z, idx, t, loss, d, targets=y, row_weight=w, hard=0.5)
    assert not bool(loss[1:4].any()) and not bool(d[1:4].any()) and bool((loss[[0, 4, 5]] > 0).all())
    z[1:4], t[3, 2] = z[:3].clone(), 0.5
    z[1, 5] = 1.0
    check(z, idx, t, y, w, hard=0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_is_left_from_rows_before(dtype):
    """Rows whose ends lie inside a group, in few and many blocks, right after rows of NaN in every block."""
    bad = torch.full((2000, 30001), float("nan"), dtype=DT[dtype], device=DEV)
    bi = torch.arange(100, dtype=torch.int32, device=DEV).repeat(2000, 1)
    bt, bl, bd = torch.full((2000, 100), float("nan"), device=DEV), torch.empty(2000, device=DEV), torch.empty_like(bad)
    for T, V, K in [(6, 50, 40), (9, 333, 0), (30, 5003, 20), (3, 100001, 9), (700, 3001, 5)]:
        z, idx, t, y, w = make(T, V, K, repeat=True, missing=True)
        w[::4] = 0
        for hard in (0.0, 0.4):
            s2.s2_distill(bad, bi, bt, bl, bd, targets=bi[:, 0].contiguous(), hard=0.5, temperature=2.0)
            check(z, idx, t, y, w, dtype, dtype, temperature=1.5, hard=hard)


def test_no_teacher_and_nothing():
    """Cross entropy alone, and rows without any term."""
    z, _, _, y, w = make(9, 777, 3, missing=True)
    check(z, None, None, y, w, hard=1.0)
    check(z, None, None, y, w, "bf16", "bf16", hard=1.0, temperature=3.0)
    check(z, None, None, None, None)
    empty = torch.empty((4, 0), device=DEV)
    loss = torch.full((4,), 3.0, device=DEV)
    s2.s2_distill(empty, None, None, loss, empty)
    assert not bool(loss.any())
    s2.s2_distill(z[:0], None, None, loss[:0], z[:0])


@pytest.mark.parametrize("dtype,V", [("f32", 1000003), ("bf16", 1800001)])
def test_rows_larger_than_shared_memory(dtype, V):
    """Rows that a cluster cannot keep are read again."""
    z, idx, t, y, w = make(2, V, 10)
    check(z, idx, t, y, w, dtype, dtype, temperature=2.0, hard=0.3)


def test_extreme_temperatures_and_scales():
    z, idx, t, y, w = make(5, 300, 6)
    for temp in (1e-3, 0.05, 30.0, 1e6):
        check(z, idx, t, y, w, temperature=temp, soft=min(temp * temp, 1e6), hard=0.2)
    check(z * 1e4, idx, t * 1e4, y, w, temperature=1.0)
    check(z, idx, t, y, -w, hard=0.2, scale=-1e-20)


def test_gradient_matches_differences():
    """Along a direction D of entries in [-1, 1]: the central difference with step h is off by h^2/6 times the
    third derivative, a third central moment of D under p, at most 8 (its range is 2), for each softmax;
    and by the rounding of two losses over 2 h."""
    T, V, K, h, temp, soft, hard = 4, 500, 12, 2.0 ** -6, 2.0, 4.0, 0.5
    z, idx, t, y, w = make(T, V, K, repeat=True)
    rng = np.random.default_rng(5)
    D = torch.from_numpy(rng.uniform(-1, 1, size=(T, V))).float().to(DEV)
    D = (D * 256).round() / 256
    z = (z * 256).round() / 256      # z + h D is exact
    loss, d = torch.empty(T, device=DEV), torch.empty((T, V), device=DEV)
    args = dict(targets=y, row_weight=w, temperature=temp, soft=soft, hard=hard)
    s2.s2_distill(z, idx, t, loss, d, **args)
    slope = (d.double() * D.double()).sum(1).cpu().numpy()
    up, down = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    s2.s2_distill(z + h * D, idx, t, up, **args)
    s2.s2_distill(z - h * D, idx, t, down, **args)
    diff = ((up.double() - down.double()) / (2 * h)).cpu().numpy()
    _, _, room, droom = ref.distill(np64(z), np64(idx), np64(t), np64(y), np64(w), temp, soft, hard, 1.0)
    E = (4 + 3 * 30 + V / 512 + 36) * 2.0 ** -24
    tol = 8 * h * h / 6 * (soft / temp ** 3 + hard) * 1.5 + E * room / h * 1.1 + E * droom.sum(1) * 1.1
    assert (np.abs(diff - slope) <= tol).all()


def test_offsets_past_32_bits():
    far = (1 << 31) + 8
    T, V, K = 3, 700, 5
    z, idx, t, y, w = make(T, V, K)
    wide = torch.empty((T - 1) * far + V, dtype=torch.bfloat16, device=DEV).as_strided((T, V), (far, 1))
    out = torch.empty((T - 1) * far + V, dtype=torch.bfloat16, device=DEV).as_strided((T, V), (far, 1))
    wide.copy_(z)
    loss, l2 = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    near = torch.empty((T, V), dtype=torch.bfloat16, device=DEV)
    s2.s2_distill(wide, idx, t, loss, out, targets=y, hard=0.5)
    s2.s2_distill(wide.contiguous(), idx, t, l2, near, targets=y, hard=0.5)
    assert torch.equal(out.contiguous(), near) and torch.equal(loss, l2)


def test_streams_graphs_and_repeats():
    """The same bits on every run, on a side stream, in two graphs at once, and after the inputs changed."""
    T, V, K = 30, 30011, 20
    z, idx, t, y, w = make(T, V, K, repeat=True)
    z = z.to(torch.bfloat16)
    args = dict(targets=y, row_weight=w, temperature=2.0, hard=0.5)

    def fresh():
        return torch.empty(T, device=DEV), torch.empty((T, V), dtype=torch.bfloat16, device=DEV)

    want = fresh()
    s2.s2_distill(z, idx, t, *want, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fresh()
    s2.s2_distill(z, idx, t, *got, **args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        g, o = torch.cuda.CUDAGraph(), fresh()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for _ in range(3):
                s2.s2_distill(z, idx, t, *o, **args)
        graphs.append(g)
        outs.append(o)
    for _ in range(4):
        for o in outs:
            o[0].zero_(), o[1].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, o))
    # the next kernel starts early: it has to wait for the one before it
    for i in range(10):
        z2 = torch.empty_like(z)
        z2.copy_(z)
        z2 *= 1 + i
        s2.s2_distill(z2, idx, t, *got, **args)
        s2.s2_distill(got[1], idx, t, *outs[0], **args)
    torch.cuda.synchronize()
    check_loss, check_d = fresh()
    s2.s2_distill(z2, idx, t, check_loss, check_d, **args)
    torch.cuda.synchronize()
    again = fresh()
    s2.s2_distill(check_d, idx, t, *again, **args)
    assert all(torch.equal(a, b) for a, b in zip(again, outs[0]))


def test_allocates_nothing():
    z, idx, t, y, w = make(50, 5000, 20)
    loss, d = torch.empty(50, device=DEV), torch.empty_like(z)
    for grad in (d, None):
        call = lambda: s2.s2_distill(z, idx, t, loss, grad, targets=y, hard=0.5, temperature=2.0)  # noqa: E731,B023
        call()
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
        for _ in range(3):
            call()
        torch.cuda.synchronize()
        assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()) == before


def test_binding_refusals():
    z, idx, t, y, w = make(4, 50, 3)
    loss = torch.empty(4, device=DEV)
    for bad in (dict(teacher_idx=idx, teacher=None), dict(teacher_idx=idx[:, :2], teacher=t), dict(teacher_idx=idx[:3], teacher=t[:3])):
        with pytest.raises(ValueError):
            s2.s2_distill(z, loss=loss, **bad)
    with pytest.raises(ValueError):
        s2.s2_distill(z, idx, t, loss[:3])
    with pytest.raises(ValueError):
        s2.s2_distill(z, idx, t, loss, z.new_empty(4, 49))
    with pytest.raises(TypeError):
        s2.s2_distill(z, idx.long(), t, loss)
    with pytest.raises(TypeError):
        s2.s2_distill(z, idx, t.half(), loss)
    with pytest.raises(ValueError):
        s2.s2_distill(z.t(), idx, t, loss)
    with pytest.raises(ValueError):
        s2.s2_distill(z, idx.t().contiguous().t(), t, loss)
    with pytest.raises(s2.S2Error) as e:
        s2.s2_distill(z, idx, t, loss, z)  # in place
    assert e.value.status == 1
