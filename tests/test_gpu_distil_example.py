"""The distilled softmax layer of examples/: teacher, student, exchange and serving run together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import _distill, _layer4, _layer8
from tests._sample import sample

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("distil_softmax_layer", os.path.join(ROOT, "examples", "distil_softmax_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_runs(example):
    losses, served = example.train(steps=3)
    assert len(losses) == 3 and all(np.isfinite(losses))
    assert served.shape == (24,) and bool(((served >= 0) & (served < 1003)).all())


def test_a_step_from_the_teacher_to_the_weight_gradient(example):
    """Every operator of a step on what the one before it wrote, in float64 beside it. Products: bounds of
    tests/test_gpu_layer4.py and test_gpu_layer8.py; loss and gradient: the bound of tests/test_gpu_distill.py."""
    V, H, T, W, K = 333, 200, 96, 2, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    teacher = example.ReadLayer(torch.randn((V, H), generator=g, device="cuda"), T)
    layer = example.DistilledLayer(V, H, T, W)
    (hidden, tops, targets, weight), = example.batches(teacher, W, T, K, 1)
    _, _, tw = _layer4.pack(torch.randn((V, H), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").double().cpu().numpy())
    dhidden = torch.empty((W, T, H), device="cuda")
    for k in range(W):
        h = hidden[k].double().cpu().numpy()
        _, _, hv = _layer4.pack(h)
        y = teacher.forward(hidden[k]).double().cpu().numpy()
        assert (np.abs(y - hv @ tw.T) <= (65 * 4 + 8) * 2.0 ** -23 * (np.abs(hv) @ np.abs(tw).T)).all()
        idx, top = tops[k]
        np.testing.assert_array_equal(top.double().cpu().numpy(), np.take_along_axis(y, idx.cpu().numpy(), 1))
        d = layer.distil(k, hidden[k], idx, top, targets[k], weight[k])
        z = layer.logits.double().cpu().numpy()
        loss, grad, room, groom = _distill.distill(z, idx.cpu().numpy(), top.double().cpu().numpy(), targets[k].cpu().numpy(),
                                                   weight[k].double().cpu().numpy(), 2.0, 4.0, 0.25, 1 / (T * W))
        E = (4 + 3 * min(90.0, np.ptp(z, axis=1).max()) + V / 512 + 36) * 2.0 ** -24
        assert (np.abs(layer.loss[k].double().cpu().numpy() - loss) <= E * room + 2.0 ** -24 * np.abs(loss) + 1e-37).all()
        dv = d.double().cpu().numpy()
        assert (np.abs(dv - grad) <= E * groom + 2.0 ** -8 * 1.01 * np.abs(grad) + 1e-37).all()
        assert not dv[weight[k].cpu().numpy() == 0].any()
        layer.backward(k, d, dhidden[k])
        xc, xs = _layer8.pack(h, False)
        xv = _layer8.unpack(xc, xs, False)
        got = layer.grad[k].view(V, H).double().cpu().numpy()
        assert (np.abs(got - dv.T @ xv) <= (17 / 16 * T + 41) * 2.0 ** -23 * (np.abs(dv).T @ np.abs(xv))).all()



def test_served_words(example):
    """The words that serving draws are those of its own logits, by the plain rule."""
    V, H, B = 1003, 128, 24
    layer = example.DistilledLayer(V, H, 32, 1)
    hidden = torch.randn((B, H), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").to(torch.bfloat16)
    tokens = example.serve(layer, hidden).cpu().numpy()
    logits = example.ReadLayer(layer.weight, B).forward(hidden).cpu().numpy()
    u = torch.rand(B, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").cpu().numpy()
    of = lambda *v: np.resize(np.asarray(v, np.float32), B)  # noqa: E731
    t, k, p, m = of(0.0, 0.7, 1.0, 1.3), of(0, 50, 0).astype(np.int32), of(1.0, 0.9, 0.95, 1.0, 0.8), of(0.0, 0.0, 0.02)
    for i in range(B):
        want, clear = sample(logits[i], u[i], t[i], k[i], p[i], m[i])
        assert not clear or tokens[i] == want
