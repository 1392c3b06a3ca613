"""s2_distill with a teacher and targets, at temperatures where its two sums have nothing to do with one another."""
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
