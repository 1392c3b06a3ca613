"""s2_distill at temperatures where its two sums have nothing to do with one another, and where logits hardly differ."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sketch_compressed_sparse_gb300 as s2

DEV = "cuda"


def test_time_does_not_depend_on_the_temperature():
    """The log-sum of a row at temperature 8 lies far above the one at 1: each sum rests on its own of the row
    before, so neither is taken again. (A third more time is allowed; where every row is gone over three times it is
    more than 1.4 times. The least of several times, in turn.)"""
    T, V, K = 512, 267735, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn((T, V), generator=g, device=DEV).mul_(1.2)
    z -= 1.1 * torch.log(1.0 + torch.randperm(V, generator=g, device=DEV))
    z = z.to(torch.bfloat16)
    idx = torch.randint(V, (T, K), generator=g, device=DEV, dtype=torch.int32)
    t, y = torch.randn((T, K), generator=g, device=DEV), idx[:, 0].contiguous()
    loss, d = torch.empty(T, device=DEV), torch.empty_like(z)

    def ms(temperature):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            s2.s2_distill(z, idx, t, loss, d, targets=y, temperature=temperature, soft=3.0, hard=0.25)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b)

    times = [(ms(3.0), ms(8.0)) for _ in range(8)][2:]
    near, far = (min(x) for x in zip(*times))
    assert far <= near * 4 / 3, (near, far)


@pytest.mark.parametrize("V", [1003, 2000003])
@pytest.mark.parametrize("temperature", [1e30, 8e36, 1e37, 3e38])
def test_huge_temperatures(temperature, V):
    """Every finite distance is next to nothing: a row is uniform, its loss log V, each probability 1 / V. (A sum of V
    ones, V / 1000 in each of a thread's, and the twenty that join them: off by 2^-24 (V / 1000 + 20) of itself at most;
    the exponent of the sum, log2 V, is off by 2^-22 of itself.)"""
    z = torch.randn((40, V), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    idx, t = torch.full((40, 1), 7, dtype=torch.int32, device=DEV), torch.zeros((40, 1), device=DEV)
    loss, d = torch.empty(40, device=DEV), torch.empty((40, V), device=DEV)
    s2.s2_distill(z, idx, t, loss, d, temperature=temperature, soft=1e30)
    off = 2.0 ** -24 * (V / 1000 + 20 + 4 * math.log2(V))
    assert (loss.double() / 1e30 - math.log(V)).abs().max().item() <= off * 2
    d = d.double() * (temperature / 1e30 * V)
    d[:, 7] += V
    assert (d - 1).abs().max(dim=0)[0][torch.arange(V, device=DEV) != 7].max().item() <= off * 2
    assert (d[:, 7] - 1).abs().max().item() <= off * 2 + V * 2.0 ** -23


@pytest.mark.parametrize("temperature", [1.0, 1e30, 8e36, 1e37, 3e38])
def test_infinite_logit_behind_what_is_kept(temperature):
    """+infinity makes a row NaN also where it lies behind what a cluster keeps of the row."""
    V = 2000003
    z = torch.randn((2, V), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    z[0, V - 5] = float("inf")
    idx, t = torch.full((2, 1), 7, dtype=torch.int32, device=DEV), torch.zeros((2, 1), device=DEV)
    loss, d = torch.empty(2, device=DEV), torch.empty((2, V), device=DEV)
    s2.s2_distill(z, idx, t, loss, d, temperature=temperature)
    assert bool(torch.isnan(loss[0])) and bool(torch.isnan(d[0]).all())
    assert bool(torch.isfinite(loss[1])) and bool(torch.isfinite(d[1]).all())
