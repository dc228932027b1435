"""Verification of drafts, the policy loss, checkpoints, factors and the step together, as they
are used."""
import math
import os
import sys

import numpy as np
import pytest
import torch

from tests import checkpoint_ref as ref
from second_order_optimisation_gb300 import kfac, workloads
from second_order_optimisation_gb300.step import KfacStep

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("loss,drafts,checkpoints", [("policy", 3, True), ("policy", 4, False), ("preference", 0, True)])
def test_example_runs(loss, drafts, checkpoints):
    import policy_step
    r = policy_step.train(loss, rounds=4, drafts=drafts, checkpoints=checkpoints)
    assert len(r) == 4 and all(math.isfinite(x) for x in r)


def _keep(t, one=False):
    c = kfac.Checkpoint.empty(*t.shape, one)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(t, c, one)])
    return c


def _values(c, cols):
    """A checkpoint's values in 64 bits, by its bytes."""
    q = c.q.cpu().numpy()[:, :c.width]
    s = c.scales.cpu().numpy().astype(np.int64)
    t, k = np.arange(-(-c.rows // 32))[:, None], np.arange(c.width)[None]
    return ref.values(q, s[ref.place(c.rows, t, k)] - 127)


def test_from_drafts_to_the_step():
    """Drafts are verified; the loss takes the tokens and their log-probabilities; its output gradients and the
    features are kept in 8 bits; weight gradient, factors and step are made from them."""
    rows, din, vocab, k = 300, 130, 200, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    a, w, w_old = rand(rows, din).bfloat16(), rand(vocab, din) * 0.1, rand(vocab, din) * 0.1
    logits, draft = a @ w.bfloat16().t(), a @ (0.8 * w + 0.2 * w_old).bfloat16().t()
    gumbel = -torch.empty(rows, vocab, device="cuda").exponential_(generator=g).log()
    tokens = (draft.float() + gumbel).argmax(1)
    offsets = torch.arange(0, rows + 1, k + 1, dtype=torch.int32, device="cuda")
    accepted, logp = torch.empty(len(offsets) - 1, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    out = torch.empty_like(tokens)
    ws = kfac.kfac_verify_draft(kfac.VerifyDraft(
        logits, tokens, offsets, accepted, out, logp, draft=draft, uniform=torch.rand(rows, device="cuda", generator=g),
        noise=torch.empty(len(offsets) - 1, vocab, device="cuda").exponential_(generator=g)))
    assert int(ws.view(torch.int32)[0]) == 0
    n = accepted.cpu().numpy()
    live = np.concatenate([np.arange(k + 1) <= m for m in n])
    assert 0 < n.mean() < k and np.array_equal(out.cpu().numpy() >= 0, live)

    # the loss: ratio 1 at every live row, nothing clipped, ignored rows without gradient
    adv = rand(rows)
    stats, lp, dlogits = torch.empty(5, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(logits)
    kfac.kfac_policy_loss(kfac.PolicyLoss(logits, out, adv, logp, stats, lp, dlogits, grad_scale=float(rows)))
    assert (lp - logp).abs().max() < 2e-6 and float(stats[4]) == 0
    assert abs(float(stats[0]) + float(adv[torch.from_numpy(live).cuda()].mean())) < 1e-4
    assert int(torch.count_nonzero(dlogits[~torch.from_numpy(live).cuda()])) == 0

    # kept in 8 bits: within the format's bound of what they are, products exact
    ca, cg = _keep(a, one=True), _keep(dlogits)
    va, vg = _values(ca, din + 1), _values(cg, vocab)
    top = np.abs(np.concatenate([dlogits.double().cpu().numpy(), np.zeros((-rows % 32, vocab))])).reshape(-1, 32, vocab).max(1)
    step = np.repeat(np.maximum(top * 2.0 ** -17.8, 0), 32, 0)[:rows]  # 2^(e - 10), 448 2^(e - 1) < top
    d = dlogits.double().cpu().numpy()
    assert (np.abs(vg - d) <= np.maximum(2.0 ** -4 * np.abs(d), step)).all()
    layer = workloads.Layer("head", din, vocab, 1, 1, 0, 1, 1, True)
    kf = KfacStep([layer], rows, xi=0.5, gamma=1e-2, weights=[torch.zeros(vocab, din + 1, device="cuda")], eta=0.1)
    kf.run([ca], [cg])
    grad = kf._grads[0].double().cpu().numpy()
    want, tol = ref.weight_grad(vg, va, float(np.float32(1.0 / rows)))
    assert (np.abs(grad - want) <= tol + ref.ROUND["bf16"] * np.abs(want) + 1e-37).all()
    A = np.triu(kf.state[0].A.double().cpu().numpy())
    wantA, tolA = ref.weight_grad(va, va, 0.5 / rows, 0.5, np.eye(din + 1))
    assert (np.abs(A - np.triu(wantA)) <= tolA + 4 * ref.E * np.abs(np.triu(wantA)) + 1e-30).all()
    assert kf.info.cpu().tolist() == [0, 0]

    # the same step from the values that the checkpoints stand for
    plain = KfacStep([layer], rows, xi=0.5, gamma=1e-2)
    x = torch.empty(rows, din, dtype=torch.bfloat16, device="cuda")
    gr = torch.empty_like(dlogits)
    kfac.kfac_checkpoint_load([kfac.CheckpointItem(x, ca, True), kfac.CheckpointItem(gr, cg)])
    plain.run([x], [gr], [kf._grads[0]])
    P, Q = kf.state[0].out.double(), plain.state[0].out.double()
    assert float((P - Q).norm() / Q.norm()) < 2e-2
    moved = kf.weights[0].double()
    assert float((moved + 0.1 * P).norm() / (0.1 * P).norm()) < 1e-5


def test_step_refuses():
    layer = workloads.Layer("head", 64, 32, 1, 1, 0, 1, 1, True)
    kf = KfacStep([layer], 8)
    x, g = torch.zeros(8, 64, device="cuda"), torch.zeros(8, 32, device="cuda")
    with pytest.raises(ValueError):  # without its column of ones
        kf.run([_keep(x)], [_keep(g)], [torch.zeros(32, 65, dtype=torch.bfloat16, device="cuda")])
    with pytest.raises(TypeError):
        kf.run([x], [_keep(g)])


def test_two_streams_and_a_captured_step():
    """Calls on two streams at once, each with its workspace, and the same captured with an eager call
    beside it, give what one stream gives."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = [torch.randn(2000, 300, device="cuda", generator=g) for _ in range(2)]
    y = [torch.randn(2000, 200, device="cuda", generator=g) for _ in range(2)]

    def all_of(i, out, F, ck=None, ws=None, stream=None):
        ca, cg = ck or (kfac.Checkpoint.empty(2000, 300), kfac.Checkpoint.empty(2000, 200))
        kfac.kfac_checkpoint_store([kfac.CheckpointItem(x[i], ca), kfac.CheckpointItem(y[i], cg)], stream)
        w1, w2 = ws or (None, None)
        kfac.kfac_weight_grad([kfac.WeightGrad(ca, cg, out)], w1, stream)
        kfac.kfac_factor_update([kfac.FactorSource(ca, F, alpha=0.1)], w2, stream)

    want = [(torch.empty(200, 300, device="cuda"), torch.zeros(300, 300, device="cuda")) for _ in range(2)]
    for i in range(2):
        all_of(i, *want[i])
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [(torch.empty(200, 300, device="cuda"), torch.zeros(300, 300, device="cuda")) for _ in range(2)]
    cks = [(kfac.Checkpoint.empty(2000, 300), kfac.Checkpoint.empty(2000, 200)) for _ in range(2)]
    wss = [tuple(torch.empty(1 << 27, dtype=torch.uint8, device="cuda") for _ in range(2)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            all_of(i, *got[i], cks[i], wss[i], sides[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sides[0]):
        all_of(0, *got[0], cks[0], wss[0])
    got[0][0].zero_()
    got[1][0].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        all_of(1, *got[1], cks[1], wss[1], sides[1])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
