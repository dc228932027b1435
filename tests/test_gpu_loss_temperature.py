"""Losses on logits at temperatures far from 1: logits of a size that the
temperature brings to order 1, some of them -inf (p = 0 whatever the temperature
is).  Bounds as in loss_ref.py."""
import numpy as np
import pytest
import torch

from second_order_optimisation_gb300 import kfac
from tests import loss_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SHAPES = [(8, 18), (9, 1500), (300, 600), (7, 33000)]  # small kernels (8 and 32 lanes), warps, ring or stream
#        temperature, the logits' size, what is added to all of them
RANGES = [("f32", 1e-10, 1e-10, 0.0), ("bf16", 1e-10, 1e-10, 0.0), ("f32", 1e-30, 1e-30, 0.0), ("f32", 1e-36, 1e-36, 0.0),
          ("f16", 1e-3, 1e-3, 0.0), ("f16", 1e-10, 0.0, 0.0), ("f16", 300.0, 300.0, -20000.0), ("f16", 4e3, 4e3, 0.0),
          ("f16", 1e4, 8e3, 0.0), ("f16", 1e9, 8e3, 0.0), ("bf16", 1e27, 1e27, 0.0), ("f32", 1e29, 1e29, 0.0),
          ("bf16", 1e33, 1e33, 0.0), ("f32", 1e-9, 1e-9, 1e-9)]


def _logits(dtype, rows, vocab, size, base, seed):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(rows, vocab, generator=g, dtype=torch.float64) * size + base)
    off = torch.rand(rows, vocab, generator=g) < 0.3
    t = torch.randint(0, vocab, (rows,), generator=g)
    off[torch.arange(rows), t] = False
    z[off] = -float("inf")
    z = z.to(TYPES[dtype])
    return z, z.double().numpy(), t.numpy()


def vec(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.float32, device=DEV)


def nums(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype,tau,size,base", RANGES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_logprob_entropy_and_gradients(dtype, tau, size, base, rows, vocab):
    z, zn, t = _logits(dtype, rows, vocab, size, base, rows + vocab)
    tau = float(np.float32(tau))
    zd, td, live = z.to(DEV), torch.from_numpy(t).to(DEV), np.ones(rows, bool)
    logp, lse, h = (torch.full((rows,), 7.0, device=DEV) for _ in range(3))
    saved = torch.empty(rows, 2, device=DEV)
    kfac.kfac_token_logprob(kfac.TokenLogprob(zd, td, logp, lse, h, tau, saved))
    r = ref.rows_of(zn, t, tau, live)
    ref.close(nums(logp), r["logp"], r["tol"], "logp")
    ref.close(nums(h), r["h"], r["hol"], "entropy")
    only = torch.empty(rows, device=DEV)
    kfac.kfac_token_logprob(kfac.TokenLogprob(zd, td, only, temperature=tau))
    ref.close(nums(only), r["logp"], r["tol"], "logp alone")
    rng = np.random.default_rng(vocab)
    g, gh = ((rng.normal(size=rows) * tau).astype(np.float32) for _ in range(2))  # the gradients are of order 1
    for with_h in (True, False):
        d = torch.full_like(zd, 7.0)
        kfac.kfac_token_logprob_grad(kfac.TokenLogprobGrad(zd, td, saved, vec(g), d, h if with_h else None,
                                                          vec(gh) if with_h else None, tau))
        want, tol = ref.dlogits(r, t, live, g.astype(float), gh.astype(float) if with_h else None, 1.0, tau)
        ref.close(nums(d), want, tol + ref.ROUND[dtype] * np.abs(want) + ref.TINY[dtype], "dlogits")
        assert bool((d[torch.isinf(zd)] == 0).all())


@pytest.mark.parametrize("dtype,tau,size,base", RANGES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("gradient", [True, False])
def test_policy_with_entropy(dtype, tau, size, base, rows, vocab, gradient):
    z, zn, t = _logits(dtype, rows, vocab, size, base, rows + vocab)
    tau = float(np.float32(tau))
    zd, live, ent = z.to(DEV), np.ones(rows, bool), 0.02
    lp = ref.rows_of(zn, t, tau, live)["logp"]
    rng = np.random.default_rng(vocab)
    old = (lp - np.log(np.array([0.5, 0.9, 1.1, 1.6])[rng.integers(0, 4, rows)])).astype(np.float32)
    adv, w = rng.normal(size=rows).astype(np.float32), np.full(rows, 1 / rows)
    d = torch.full_like(zd, 7.0) if gradient else None
    stats, logp, h = torch.empty(5, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ws = kfac.kfac_policy_loss(kfac.PolicyLoss(
        zd, torch.from_numpy(t).to(DEV), vec(adv), vec(old), stats, logp, d, entropy=h, entropy_coef=ent, temperature=tau, grad_scale=tau))
    want = ref.policy(zn, t, live, adv.astype(float), old.astype(float), None, w, 0.2, 0.2, 0.0, ent, tau, tau)
    ref.close(nums(logp), want["r"]["logp"], want["r"]["tol"], "logp")
    ref.close(nums(h), want["r"]["h"], want["r"]["hol"], "entropy")
    ref.close(nums(stats), want["stats"], want["stol"], "stats")
    assert int(ws[:4].view(torch.int32).item()) == 0
    if gradient:
        ref.close(nums(d), want["d"], want["tol"] + ref.ROUND[dtype] * np.abs(want["d"]) + ref.TINY[dtype], "dlogits")
