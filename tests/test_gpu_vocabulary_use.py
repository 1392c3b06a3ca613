"""The 4-bit product, the distillation loss and the sampling call as a program uses them: one after the
other in a graph whose inputs change, from several threads at once, captured before anything else of the
process ran, and on the first rows and columns of larger buffers."""
import subprocess
import sys
import threading
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


class Layer:
    """A softmax layer in 4 bits with a teacher's lists and settings, and one step
    over them: logits, loss and gradient, next tokens."""

    def __init__(self, T, V, H, K, seed, gap=0):
        import sketch_compressed_sparse_gb300 as s2

        self.s2 = s2
        g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, device=DEV, generator=g)  # noqa: E731
        self.x, w = rand(T, H).to(torch.bfloat16), rand(V, H) / H ** 0.5
        self.w, self.xc = s2.alloc_pack4(V, H), s2.alloc_pack4(T, H)
        s2.s2_pack4(w, *self.w)
        self.idx = torch.randint(0, V, (T, K), dtype=torch.int32, device=DEV, generator=g)
        self.teacher = rand(T, K)
        self.y = torch.randint(0, V, (T,), dtype=torch.int32, device=DEV, generator=g)
        self.u = torch.rand(T, device=DEV, generator=g)
        self.set = dict(temperature=0.5 + torch.rand(T, device=DEV, generator=g),
                        top_k=torch.randint(0, 200, (T,), dtype=torch.int32, device=DEV, generator=g),
                        top_p=0.5 + torch.rand(T, device=DEV, generator=g))
        self.whole = [torch.full((T + gap, V + gap), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        self.z, self.d = [t[:T, :V] for t in self.whole]
        self.losses, self.all_tokens = torch.full((T + gap,), 7.0, device=DEV), torch.full((T + gap,), 7, dtype=torch.int32, device=DEV)
        self.loss, self.tokens = self.losses[:T], self.all_tokens[:T]

    def step(self, between=lambda: None):
        s2 = self.s2
        s2.s2_pack4(self.x, *self.xc)
        between()
        s2.s2_matmul4(*self.xc, *self.w, self.z)
        between()
        s2.s2_distill(self.z, self.idx, self.teacher, self.loss, self.d, targets=self.y, temperature=2.0, hard=0.5)
        between()
        s2.s2_sample(self.z, self.u, self.tokens, **self.set)
        between()

    def out(self):
        return [t.clone() for t in (self.z, self.loss, self.d, self.tokens)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,V", [(1, 30011), (37, 5003), (300, 33278)])
def test_graph_with_new_inputs(T, V):
    """A captured step, replayed after its inputs and settings changed in place: what the calls give with a
    wait after each. Two graphs that share every buffer but run one after the other."""
    a = Layer(T, V, 256, 20, 1)
    a.step()
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[-1]):
            a.step()
    for i in range(6):
        a.x.mul_(1.1)
        a.u.copy_((a.u + 0.37) % 1.0)
        a.teacher.neg_()
        a.set["top_k"].add_(1)
        graphs[i % 2].replay()
        got = a.out()
        torch.cuda.synchronize()
        a.step(torch.cuda.synchronize)
        assert same(got, a.out())
    assert a.s2.s2_wait_faults() == 0


def test_rows_behind_the_last():
    """Outputs that are parts of larger buffers: nothing around them is written. Logits and tokens are those of
    a call on buffers of its own, bit for bit. The loss and its gradient are so up to the order of the two
    float32 sums over a row, whose parts begin at multiples of eight elements of the address, and these rows
    begin elsewhere. A sum of positive numbers in another order is off by the additions that a number goes
    through, at most 64 (ten groups of four pairs, lanes, warps, blocks) of 2^-24 on each side: 2^-17. The
    logarithms of both sums enter the loss with weights of 1 and 0.5, next to roundings of the loss itself. An
    element without an entry is a probability of that error, rounded to bfloat16 on each side: 2^-7 + 2^-15 of
    itself; at an entry or a target it is off by 2^-15 at most besides (weights of 0.5 and 0.5, halved by no
    scale, of numbers up to 1)."""
    a, b = Layer(29, 5003, 256, 20, 2, gap=3), Layer(29, 5003, 256, 20, 2)
    a.step()
    b.step()
    (az, al, ad, at), (bz, bl, bd, bt) = a.out(), b.out()
    assert torch.equal(az, bz) and torch.equal(at, bt)
    assert bool(((al - bl).abs() <= 2.0 ** -16 * (1 + bl.abs())).all())
    listed = torch.zeros((29, 5003), device=DEV).scatter_(1, torch.cat([a.idx, a.y[:, None]], 1).long(), 1.0)
    ad, bd = ad.float(), bd.float()
    assert bool(((ad - bd).abs() <= (2.0 ** -7 + 2.0 ** -15) * bd.abs() + 2.0 ** -15 * listed).all())
    for t in a.whole:
        assert bool((t[29:] == 7).all()) and bool((t[:, 5003:] == 7).all())
    assert bool((a.losses[29:] == 7).all()) and bool((a.all_tokens[29:] == 7).all())


def test_threads_at_once():
    """Four host threads, each with a stream and sizes of its own, whose kernels share the GPU."""
    layers = [Layer(T, V, 256, K, s) for s, (T, V, K) in enumerate([(3, 30011, 20), (40, 12007, 64), (100, 5003, 300), (250, 2048, 1)])]
    wants = []
    for a in layers:
        a.step(torch.cuda.synchronize)
        wants.append(a.out())
    torch.cuda.synchronize()
    failed = []

    def work(a, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    a.step()
                    if not same(a.out(), want):
                        failed.append("other bits")
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=z) for z in zip(layers, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and layers[0].s2.s2_wait_faults() == 0


FIRST = """
import torch
import sketch_compressed_sparse_gb300 as s2
z = torch.randn((9, 30011), device="cuda")
u, tokens = torch.rand(9, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
codes, scales = s2.alloc_pack4(9, 30011)
back = torch.zeros_like(z)
p = torch.full((9,), 0.9, device="cuda")
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    s2.s2_pack4(z, codes, scales)
    s2.s2_unpack4(codes, scales, back)
    s2.s2_sample(back, u, tokens, top_p=p)
g.replay()
got = [t.clone() for t in (codes, scales, back, tokens)]
s2.s2_pack4(z, codes, scales)
s2.s2_unpack4(codes, scales, back)
s2.s2_sample(back, u, tokens, top_p=p)
assert all(torch.equal(a, b) for a, b in zip(got, (codes, scales, back, tokens)))
print("same")
"""


def test_captured_before_any_call():
    """Packing, unpacking and sampling look nothing up on the device: their first call may be a captured one."""
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=Path(__file__).parents[1], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
