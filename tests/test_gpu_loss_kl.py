"""The KL term of the policy loss where policy and reference nearly agree.

d = ref - logp is formed exactly here (two fp32 numbers close to each other, or far
enough apart that the test takes the rounded difference), so only the term's own
arithmetic is compared.  Below |d| = 1/4 it is a product of d^2 and a polynomial: 8
roundings at most.  Above, expm1f (1 ulp = 2 e) less d: 3 e |e^d - 1| and one
rounding of the difference."""
import numpy as np
import pytest
import torch

from second_order_optimisation_gb300 import kfac
from tests import loss_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = np.array([0.0, 1e-6, -1e-6, 1e-4, -1e-4, 3e-4, -3e-4, 1e-3, -1e-3, 4e-3, -1e-2, 0.03, -0.1, 0.2, -0.2499, 0.2499, 0.26,
              -0.26, 0.7, -1.5, 3.0, -8.0, 20.0])


@pytest.mark.parametrize("rows,vocab", [(46, 18), (46, 1000), (230, 3000), (46, 33000)])
@pytest.mark.parametrize("gradient", [True, False])
def test_small_differences(rows, vocab, gradient):
    g = torch.Generator().manual_seed(vocab)
    z = torch.randn(rows, vocab, generator=g) * 2
    t = torch.randint(0, vocab, (rows,), generator=g)
    zd, td = z.to(DEV), t.to(DEV)
    new = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    logp, kl, stats, none = new(rows), new(rows), new(5), torch.zeros(rows, device=DEV)
    d = torch.empty_like(zd) if gradient else None
    run = lambda r: kfac.kfac_policy_loss(kfac.PolicyLoss(  # noqa: E731
        zd, td, none, none, stats, logp, d, r, kl=kl, kl_coef=0.5))
    run(none)
    rf = logp + torch.from_numpy(np.resize(D, rows)).float().to(DEV)
    run(rf)
    lp = logp.double().cpu().numpy()
    diff = (rf - logp).double().cpu().numpy()
    em = np.expm1(diff)
    want = em - diff
    tol = ref.E * np.where(np.abs(diff) < 0.25, 8 * want, 3 * np.abs(em) + 2 * want)
    got = kl.double().cpu().numpy()
    assert (got >= 0).all()
    ref.close(got, want, tol, "kl")
    st = stats.double().cpu().numpy()
    ref.close(st[2], want.mean(), tol.mean() + 4 * ref.E * want.mean(), "mean kl")
    ref.close(st[0], 0.5 * want.mean(), 0.5 * tol.mean() + 4 * ref.E * want.mean(), "loss")
    assert np.abs(lp).max() < 50
    if not gradient:
        return
    live = np.ones(rows, bool)
    zn, tn = z.double().numpy(), t.numpy()
    r = ref.rows_of(zn, tn, 1.0, live)
    g = -0.5 * em / rows
    want_d, tol_d = ref.dlogits(r, tn, live, g, None, 1.0, 1.0, 8 * ref.E * np.abs(g))
    ref.close(d.double().cpu().numpy(), want_d, tol_d + ref.E * np.abs(want_d) + 1e-37, "dlogits")
