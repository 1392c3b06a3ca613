"""The 8-bit softmax layer of examples/ run together with the compressed exchange."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import _layer8 as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("softmax_layer_8bit", os.path.join(ROOT, "examples", "softmax_layer_8bit.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loss_falls(example):
    """log(1003) = 6.9 at random; the words are learned through Top-K, sketch and 8 bits."""
    losses = example.train(steps=12)
    assert all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]


def test_gradients_of_a_step(example):
    """grad[k] and dhidden are the layer's gradients at the packed values: each float32 sum of
    exact products is off by at most (number of terms + 41) * 2^-23 * sum of magnitudes."""
    V, H, T, W = 333, 200, 96, 2
    layer = example.SoftmaxLayer(V, H, T, W)
    (hidden, targets), = example.batches(V, H, T, W, 1)
    dhidden = torch.empty((W, T, H), device="cuda")
    wv = ref.unpack(layer.codes.cpu().numpy(), layer.scales.cpu().numpy(), True)
    np.testing.assert_array_equal(layer.codes_t.cpu().numpy(), layer.codes.t().cpu().numpy())
    for k in range(W):
        logits = layer.forward(k, hidden[k])
        xc, xs = ref.pack(hidden[k].double().cpu().numpy(), False)
        xv = ref.unpack(xc, xs, False)
        y = logits.double().cpu().numpy()
        assert (np.abs(y - xv @ wv.T) <= (H + 41) * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T)).all()
        d = torch.softmax(logits, dim=1).to(torch.bfloat16)
        layer.backward(k, d, dhidden[k])
        dv = d.double().cpu().numpy()
        got = layer.grad[k].view(V, H).double().cpu().numpy()
        assert (np.abs(got - dv.T @ xv) <= (17 / 16 * T + 41) * 2.0 ** -23 * (np.abs(dv).T @ np.abs(xv))).all()
        gc, gs = ref.pack(dv, False)
        gv = ref.unpack(gc, gs, False)
        got = dhidden[k].double().cpu().numpy()
        assert (np.abs(got - gv @ wv) <= (V + 41) * 2.0 ** -23 * (np.abs(gv) @ np.abs(wv))).all()


def test_waits_that_ran_out_end_the_training(example, monkeypatch):
    """The count is asked before and after the steps; one that rises is an error and no list of losses."""
    counts = iter([3, 3])
    monkeypatch.setattr(example.s2, "s2_wait_faults", lambda: next(counts))
    assert len(example.train(steps=1)) == 1
    counts = iter([3, 4])
    with pytest.raises(RuntimeError):
        example.train(steps=1)
