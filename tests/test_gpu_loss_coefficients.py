"""A gradient coefficient that is not finite once grad_scale and the temperature are
in it is named in the error word, whichever kernel made it."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHAPES = [(9, 31), (200, 3001), (7, 33000), (2, 1_500_003)]


def word(ws):
    torch.cuda.synchronize()
    return int(ws[:4].view(torch.int32).item())


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("scale,tau,expect", [(1.0, 1.0, 0), (3e38, 0.01, 1), (3e38, 1.0, 1), (1e30, 1.0, 0)])
def test_policy(rows, vocab, scale, tau, expect):
    z = torch.randn(rows, vocab, device=DEV)
    t = torch.arange(rows, device=DEV)
    logp, stats = torch.empty(rows, device=DEV), torch.empty(5, device=DEV)
    kfac.kfac_token_logprob(kfac.TokenLogprob(z, t, logp, temperature=tau))
    adv = torch.full((rows,), 1e3, device=DEV)  # (r = 1: a coefficient of 1e3 / rows before the scale)
    for d in (torch.empty_like(z), None):
        ws = kfac.kfac_policy_loss(kfac.PolicyLoss(z, t, adv, logp, stats, dlogits=d, temperature=tau, grad_scale=scale))
        assert word(ws) == (kfac.ERRW_NONFINITE if expect and d is not None else 0)
        if d is not None:
            assert bool(torch.isfinite(d).all()) == (not expect)
        assert bool(torch.isfinite(stats).all())


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("scale,tau,expect", [(1.0, 1.0, 0), (3e38, 0.01, 1), (3e38, 1.0, 1), (1e30, 1.0, 0)])
def test_preference(rows, vocab, scale, tau, expect):
    z = torch.randn(rows, vocab, device=DEV)
    t = torch.arange(rows, device=DEV)
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=DEV)
    loss = torch.empty(1, device=DEV)
    for d in (torch.empty_like(z), None):
        ws = kfac.kfac_preference_loss(kfac.PreferenceLoss(z, t, off, loss, dlogits=d, kind="ipo", beta=0.005,  # slopes of 200
                                                           temperature=tau, grad_scale=scale))
        assert word(ws) == (kfac.ERRW_NONFINITE if expect and d is not None else 0)
        if d is not None:
            assert bool(torch.isfinite(d).all()) == (not expect)
        assert bool(torch.isfinite(loss).all())
