"""GPU tests of s2_sample against the plain float64 implementation in tests/_sample.py.

A weight is right to 2^-35 of itself and rounded to 2^-44 of the largest, so a sum of V weights is off by at
most 2^-35 of itself and V 2^-44 of the largest: below 2^-33 together for V up to 2^10, and as the errors
have either sign, by a hundredth of that where V is large. Rows in which a border lies within 2^-32 (of the
sums) of what decides are not compared; there must be hardly any. The rows here have at most 4 10^5
borders, so one is that near with a chance of 4 10^5 * 2 * 2^-32 = 2 10^-4 for each of two sums.
"""
import numpy as np
import pytest
import torch

from tests._sample import sample

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def settings(T, tag):
    rng = np.random.default_rng(tag)
    return dict(temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5, 4.0], T).astype(np.float32),
                top_k=rng.choice([0, 0, -1, 1, 2, 20, 50, 700, 5000, 10 ** 9], T).astype(np.int32),
                top_p=rng.choice([1.0, 1.0, 0.999, 0.95, 0.8, 0.4, 0.01, 2.0, 0.0], T).astype(np.float32),
                min_p=rng.choice([0.0, 0.0, 0.0, 0.01, 0.1, 0.7, 1.0, -1.0], T).astype(np.float32))


def place(z, dtype, ld=None, off=0):
    T, V = z.shape
    ld = V if ld is None else ld
    flat = torch.full((off + T * ld + 9,), 99.0, dtype=DT[dtype], device=DEV)  # larger than any logit: must not be seen
    view = flat[off:off + T * ld].reshape(T, ld)[:, :V]
    view.copy_(z if isinstance(z, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(z, dtype=np.float32)))
    return view


def check(z, u, dtype="f32", ld=None, off=0, cleared=0.02, **kw):
    logits = place(z, dtype, ld, off)
    T = logits.shape[0]
    u = np.asarray(u, np.float32)
    dev = {k: torch.from_numpy(np.asarray(v)).to(DEV) for k, v in kw.items() if v is not None}
    out = torch.full((T + 1,), -7, dtype=torch.int32, device=DEV)
    s2.s2_sample(logits, torch.from_numpy(u).to(DEV), out, **dev)
    got = out.cpu().numpy()
    assert got[T] == -7
    l = logits.float().cpu().numpy()
    unclear = 0
    for i in range(T):
        want, clear = sample(l[i], u[i], **{k: v[i] for k, v in kw.items() if v is not None})
        if clear:
            assert got[i] == want, (i, got[i], want, {k: v[i] for k, v in kw.items() if v is not None}, u[i])
        unclear += not clear
    assert unclear <= cleared * T + 1
    return got[:T]


def normal(T, V, tag, sigma=2.0):
    return np.random.default_rng([T, V, tag]).normal(size=(T, V)) * sigma


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(3, 1), (9, 2), (30, 7), (30, 8), (30, 9), (60, 255), (200, 1000), (60, 4099), (40, 33278), (1, 33278)])
def test_sizes(T, V, dtype):
    z, u = normal(T, V, 0), np.random.default_rng(V).random(T)
    check(z, u, dtype, **settings(T, V))
    check(z, u, dtype)
    check(z, u, dtype, temperature=np.full(T, 0.8, np.float32), top_p=np.full(T, 0.92, np.float32))
    check(z, u, dtype, top_k=np.full(T, 40, np.int32))
    check(z * 4, u, dtype, min_p=np.full(T, 0.05, np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [100003, 267735, 1000003, 1800001])
def test_large_vocabularies(V, dtype):
    """Rows in the shared memory of many blocks, and rows that they cannot keep."""
    T = 6
    z, u = normal(T, V, 1), np.random.default_rng(V).random(T)
    check(z, u, dtype, **settings(T, V))
    check(z, u, dtype)
    check(z, u, dtype, top_p=np.float32([0.1, 0.5, 0.9, 0.99, 0.9999, 1.0]))
    check(z, u, dtype, top_k=np.int32([2, 30, 1000, 30000, V - 1, V]), top_p=np.float32([0.9] * T))


@pytest.mark.parametrize("ld,off", [(1003, 0), (1003, 3), (1008, 1), (1016, 8), (1101, 7)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_alignments(ld, off, dtype):
    z, u = normal(50, 1003, 2), np.random.default_rng(ld).random(50)
    check(z, u, dtype, ld=ld, off=off, **settings(50, ld))


@pytest.mark.parametrize("V", [50, 3000, 70001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits(V, dtype):
    """Ties go by index: all logits the same, few values, a border among equal ones. Sums are exact here."""
    T = 24
    rng = np.random.default_rng(V)
    u = np.concatenate([[0.0, 0.5, 0.25, 1 - 2.0 ** -24], rng.random(T - 4)]).astype(np.float32)
    for z in (np.full((T, V), 3.25), np.full((T, V), -0.0) * rng.choice([1.0, -1.0], size=(T, V))):
        got = check(z, u, dtype)
        np.testing.assert_array_equal(got, np.floor(u.astype(np.float64) * V).astype(int))
        check(z, u, dtype, top_k=np.int32(rng.integers(1, V + 1, T)), top_p=np.float32(rng.choice([0.5, 0.25, 0.75, 1.0], T)))
    z = rng.choice([2.0, 1.0, 0.0, -1.0], size=(T, V), p=[0.05, 0.25, 0.3, 0.4])
    check(z, u, dtype, **settings(T, V + 1))
    check(z, u, dtype, top_k=np.int32(rng.integers(1, V + 1, T)), cleared=0.3)
    check(z, u, dtype, top_p=np.float32(rng.random(T)), cleared=0.3)


@pytest.mark.parametrize("V", [40, 5000, 100003])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masks_and_special_numbers(V, dtype):
    """-infinity and NaN are never drawn, the type's lowest value only where nothing else is; +infinity takes all."""
    T = 20
    rng = np.random.default_rng(V)
    z, u = normal(T, V, 3), rng.random(T).astype(np.float32)
    z[rng.random((T, V)) < 0.5] = -np.inf
    z[0] = -np.inf
    z[1] = np.nan
    z[2] = -np.inf
    z[2, V // 2] = -50.0
    z[3, ::3] = np.nan
    z[4, 1::2] = -3e38
    z[5] = -3e38
    z[6, 5] = z[6, V - 1] = np.inf
    z[7] = np.inf
    z[8, :] = -np.inf
    z[8, [3, 9]] = [0.0, -3e38]
    z[9] = rng.choice([-3e38, 3e38, 0.0], V)
    z[10] = -1e4 + rng.random(V) * 1e-3
    z[11] = rng.normal(size=V) * 1e-42
    got = check(z, u, dtype)
    assert got[0] == got[1] == -1 and got[2] == V // 2 and got[6] in (5, V - 1)
    check(z, u, dtype, top_k=np.full(T, V // 3, np.int32), top_p=np.full(T, 0.9, np.float32), cleared=0.3)
    check(z, u, dtype, top_k=np.full(T, 3, np.int32))
    check(z, u, dtype, top_p=np.full(T, 0.6, np.float32), cleared=0.3)
    check(z, u, dtype, min_p=np.full(T, 0.3, np.float32), cleared=0.3)
    check(z, u, dtype, **settings(T, 11), cleared=0.3)


def test_extreme_settings():
    T, V = 30, 2500
    z, rng = normal(T, V, 4), np.random.default_rng(9)
    u = rng.random(T).astype(np.float32)
    odd = np.float32([np.nan, np.inf, -np.inf, -1.0, 0.0, 1e-45, 2.0 ** -126, 1e-30, 1e-3, 1e30, 3e38, 1.0])
    some = lambda: odd[rng.integers(0, len(odd), T)]  # noqa: E731
    for _ in range(6):
        kw = dict(temperature=some(), top_p=some(), min_p=some(), top_k=rng.choice([0, 1, 2 ** 31 - 1, -2 ** 31, 7], T).astype(np.int32))
        with np.errstate(over="ignore"):
            check(z, u, cleared=0.5, **kw)
    got = check(z, np.where(np.arange(T) % 2, 1.0, -1.0), temperature=np.full(T, 1e30, np.float32))
    assert (got == np.where(np.arange(T) % 2, V - 1, 0)).all()
    check(z, some())
    check(z * 1e5, u, temperature=np.full(T, 3.0, np.float32), top_p=np.full(T, 0.9, np.float32), cleared=0.3)
    check(z * 1e-4, u, top_p=np.full(T, 0.9, np.float32), top_k=np.full(T, 900, np.int32))


@pytest.mark.parametrize("T,V,base,temperature", [(40, 4099, 1e6, 1.0), (40, 4099, -1e6, 0.3), (150, 140001, 1e6, 1.0),
                                                  (150, 140001, -3e6, 2.0), (40, 33278, 2e5, 0.05)])
def test_logits_far_from_zero(T, V, base, temperature):
    """Logits whose floats lie as far apart as the ranges in which a border is looked for: what a range or a
    part of it holds may not be judged by a rounded edge."""
    rng = np.random.default_rng([T, V, 5])
    z = base + rng.normal(size=(T, V)) * 2
    kw = dict(temperature=np.full(T, temperature, np.float32), top_k=rng.choice([0, 3, 40, 200, 999, 3000, V // 20], T).astype(np.int32),
              top_p=rng.choice([1.0, 0.97, 0.9, 0.6, 0.2], T).astype(np.float32))
    check(z, rng.random(T), "f32", **kw)


def test_every_token_can_be_drawn():
    """Over an even grid of u each of the kept tokens comes as often as its probability says."""
    V, T = 300, 20000
    l = normal(1, V, 5)[0].astype(np.float32)
    u = (np.arange(T) + 0.5) / T
    out = torch.empty(T, dtype=torch.int32, device=DEV)
    rows = torch.from_numpy(l).to(DEV).repeat(T, 1)
    s2.s2_sample(rows, torch.from_numpy(u).float().to(DEV), out, top_k=torch.full((T,), 100, dtype=torch.int32, device=DEV))
    p = np.exp(l.astype(np.float64))
    p[np.argsort(-l, kind="stable")[100:]] = 0
    p /= p.sum()
    got = np.bincount(out.cpu().numpy(), minlength=V) / T
    assert np.abs(got - p).max() <= 2 / T and (got[p == 0] == 0).all()


def test_offsets_past_32_bits():
    far = (1 << 31) + 8
    z = normal(3, 700, 6)
    wide = torch.empty(2 * far + 700, dtype=torch.bfloat16, device=DEV).as_strided((3, 700), (far, 1))
    wide.copy_(torch.from_numpy(z))
    u = torch.tensor([0.2, 0.5, 0.9], device=DEV)
    a, b = (torch.empty(3, dtype=torch.int32, device=DEV) for _ in range(2))
    p = torch.full((3,), 0.9, device=DEV)
    s2.s2_sample(wide, u, a, top_p=p)
    s2.s2_sample(wide.contiguous(), u, b, top_p=p)
    assert torch.equal(a, b)


def test_streams_graphs_and_repeats():
    """The same tokens on every run, on a side stream, in two graphs at once; and a call that reads what the
    kernel before it wrote."""
    T, V = 50, 30011
    kw = {k: torch.from_numpy(v).to(DEV) for k, v in settings(T, 3).items()}
    z = torch.from_numpy(normal(T, V, 7)).float().to(DEV)
    u = torch.rand(T, device=DEV)
    want = torch.empty(T, dtype=torch.int32, device=DEV)
    s2.s2_sample(z, u, want, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(want)
    s2.s2_sample(z, u, got, **kw, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    outs, graphs, streams = [torch.empty_like(want) for _ in range(2)], [], [torch.cuda.Stream() for _ in range(2)]
    for o in outs:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for _ in range(3):
                s2.s2_sample(z, u, o, **kw)
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want, o) for o in outs)
    # logits written by the product before it, without a wait between
    x, w = torch.randn((T, 256), device=DEV), torch.randn((V, 256), device=DEV) / 16
    xc, wc = s2.alloc_pack4(T, 256), s2.alloc_pack4(V, 256)
    s2.s2_pack4(w, *wc)

    def chain(between):
        for i in range(10):
            s2.s2_pack4(x * (1 + i), *xc)
            between()
            s2.s2_matmul4(*xc, *wc, z)
            between()
            s2.s2_sample(z, u, got, **kw)
            between()
        return got.clone()

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(chain(lambda: None), want)


def test_allocates_nothing():
    T, V = 20, 40000
    z = torch.from_numpy(normal(T, V, 8)).float().to(DEV)
    kw = {k: torch.from_numpy(v).to(DEV) for k, v in settings(T, 4).items()}
    u, out = torch.rand(T, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV)
    s2.s2_sample(z, u, out, **kw)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    for _ in range(3):
        s2.s2_sample(z, u, out, **kw)
    torch.cuda.synchronize()
    assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()) == before


def test_empty_and_refusals():
    z, u, out = torch.zeros((4, 50), device=DEV), torch.rand(4, device=DEV), torch.full((4,), 5, dtype=torch.int32, device=DEV)
    s2.s2_sample(z[:, :0], u, out)
    assert bool((out == -1).all())
    s2.s2_sample(z[:0], u[:0], out[:0])
    for bad in (dict(u=u[:3]), dict(tokens=out[:3]), dict(top_p=u[:2]), dict(top_p=u[:, None]), dict(logits=z.t())):
        with pytest.raises(ValueError):
            s2.s2_sample(**{**dict(logits=z, u=u, tokens=out), **bad})
    for bad in (dict(tokens=out.long()), dict(top_k=u), dict(temperature=u.double()), dict(logits=z.half())):
        with pytest.raises(TypeError):
            s2.s2_sample(**{**dict(logits=z, u=u, tokens=out), **bad})
