"""Calls that come first inside a stream capture: of a process (where s2.h does not ask for one before), and of a form and
a shape that only calls of other forms came before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SETUP = """
import torch
import sketch_compressed_sparse_gb300 as s2

def make(T, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((T, V), generator=g, device="cuda").to(dtype)
    i = torch.randint(V, (T, 9), generator=g, device="cuda", dtype=torch.int32)
    return z, i, torch.randn((T, 9), generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")

def captured(call, outs):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        call()
    for _ in range(2):
        for o in outs:
            o.fill_(3)
        g.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, outs))
"""

SAMPLE = """
z, i, t, u = make(7, 40009, torch.bfloat16)
tokens, p = torch.empty(7, dtype=torch.int32, device="cuda"), torch.full((7,), 0.9, device="cuda")
captured(lambda: s2.s2_sample(z, u, tokens, top_p=p), [tokens])
"""

PACK = """
z, i, t, u = make(70, 1000, torch.float32)
codes, scales = s2.alloc_pack4(70, 1000)
codes.fill_(1), scales.fill_(1)
captured(lambda: s2.s2_pack4(z, codes, scales), [scales])
captured(lambda: s2.s2_unpack4(codes, scales, z), [z])
"""

FORMS = """
small = make(3, 1000, torch.float32)
s2.s2_distill(*small[:3], torch.empty(3, device="cuda"))
a, b = s2.alloc_pack4(3, 1000), s2.alloc_pack4(5, 1000)
for m, k in ((3, a), (5, b)):
    s2.s2_pack4(torch.randn((m, 1000), device="cuda"), *k)
s2.s2_matmul4(*a, *b, torch.empty((3, 5), device="cuda"))
for T, V, dtype, temperature in ((7, 40009, torch.bfloat16, 3.0), (500, 2003, torch.float32, 2.0)):
    z, i, t, u = make(T, V, dtype)
    loss, d, y = torch.empty(T, device="cuda"), torch.empty((T, V), dtype=torch.bfloat16, device="cuda"), i[:, 0].contiguous()
    captured(lambda: s2.s2_distill(z, i, t, loss, d, targets=y, temperature=temperature, hard=0.5), [loss, d])
    many, tm = i.repeat(1, 40), t.repeat(1, 40)
    captured(lambda: s2.s2_distill(z, many, tm, loss, d, targets=y, temperature=temperature, hard=0.5), [loss, d])
    x, w = s2.alloc_pack4(T, 700), s2.alloc_pack4(400, 700)
    s2.s2_pack4(torch.randn((T, 700), device="cuda"), *x)
    s2.s2_pack4(torch.randn((400, 700), device="cuda"), *w)
    out = torch.empty((T, 400), dtype=torch.bfloat16, device="cuda")
    captured(lambda: s2.s2_matmul4(*x, *w, out), [out])
"""


@pytest.mark.parametrize("code", [SAMPLE, PACK, FORMS], ids=["sample", "pack4", "other forms"])
def test_first_call_is_captured(code):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SETUP + code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
