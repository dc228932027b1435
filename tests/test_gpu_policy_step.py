"""The losses, the K-FAC step and the clipping together, as they are used."""
import math
import os
import sys

import pytest
import torch

from second_order_optimisation_gb300 import kfac, workloads
from second_order_optimisation_gb300.step import KfacStep

pytestmark = pytest.mark.gpu
DEV = "cuda"
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_example_learns(loss):
    import policy_step
    r = policy_step.train(loss, rounds=12)
    assert all(math.isfinite(x) for x in r)
    assert abs(r[0] - 0.5) < 0.05          # the first round's policy knows nothing
    assert min(r[-3:]) > r[0] + 0.05, r


def _layers():
    return [workloads.Layer("a", 64, 64, 3, 1, 1, 8, 8), workloads.Layer("fc", 96, 40, 1, 1, 0, 1, 1, True)]


def _inputs(layers, batch):
    xs, gs, grads = zip(*[[t.to(DEV) for t in workloads.layer_inputs(L, batch, "clip-step")] for L in layers])
    return xs, gs, [_pitched(g) for g in grads]


def _pitched(g):
    """Rows on 128-byte boundaries (the 16-bit preconditioner wants a multiple of 8)."""
    v = torch.zeros(g.shape[0], (g.shape[1] + 63) // 64 * 64, dtype=g.dtype, device=g.device)[:, :g.shape[1]]
    return v.copy_(g)


@pytest.mark.parametrize("metric", [True, False])
@pytest.mark.parametrize("share", [0.25, 10.0])
def test_bounded_step(metric, share):
    """With max_norm the weights move by eta * scale * P, P as without it."""
    layers, batch, eta = _layers(), 4, 0.5
    xs, gs, grads = _inputs(layers, batch)
    plain = KfacStep(layers, batch)
    plain.run(xs, gs, grads)
    P = [s.out.double() for s in plain.state]
    other = [g.double() for g in grads] if metric else P
    length = math.sqrt(sum(float((p * o).sum()) for p, o in zip(P, other)))
    w0 = [torch.randn(L.d_g, L.d_a, device=DEV) for L in layers]
    w = [t.clone() for t in w0]
    step = KfacStep(layers, batch, weights=w, eta=eta, max_norm=share * length, metric=metric)
    step.run(xs, gs, grads)
    scale = min(1.0, share)
    assert abs(float(step.norm) - length) < 1e-5 * length
    assert abs(float(step.scale) - scale) < 1e-5
    for a, b, p, s in zip(w, w0, P, step.state):
        assert torch.equal(s.out.double(), p)
        want = b.double() - eta * scale * p
        assert float((a.double() - want).abs().max()) <= 1e-6 * float(want.abs().max()) + 1e-5 * float((eta * p).abs().max())


def test_bounded_gradients_without_weights():
    layers, batch = _layers(), 4
    xs, gs, grads = _inputs(layers, batch)
    plain = KfacStep(layers, batch)
    plain.run(xs, gs, grads)
    step = KfacStep(layers, batch, max_norm=1e-3, metric=False)
    step.run(xs, gs, grads)
    total = math.sqrt(sum(float((s.out.double() ** 2).sum()) for s in step.state))
    assert abs(total - 1e-3) < 1e-8
    for a, b in zip(step.state, plain.state):
        assert torch.allclose(a.out.double(), b.out.double() * float(step.scale), rtol=1e-6, atol=0)
