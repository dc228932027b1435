"""Temperatures that the losses on logits refuse, without a GPU."""
import ctypes

import pytest

from second_order_optimisation_gb300 import kfac

BIG = (1 << 24) + 1  # a vocabulary that is refused as UNSUPPORTED once the arguments are found valid


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kfac.load()


def _calls(lib, tau):
    d = dict(dtype=kfac.KFAC_BF16, logits=0x1000, ld=BIG, rows=4, vocab=BIG, target=0x2000, temperature=tau)
    d_out = dict(dlogits=0x9000, ld_d=BIG)
    p = ctypes.byref
    ws = 0x100000, 1 << 30, None
    return [lib.kfac_token_logprob(p(kfac.LogprobDesc(**d, logp=0x3000)), None),
            lib.kfac_token_logprob_grad(p(kfac.LogprobGradDesc(**d, **d_out, saved=0x3000, dlogp=0x4000)), None),
            lib.kfac_policy_loss(p(kfac.PolicyDesc(**d, **d_out, advantage=0x3000, old_logp=0x4000, clip_low=0.2,
                                                   clip_high=0.2, grad_scale=1.0, stats=0x5000)), *ws),
            lib.kfac_preference_loss(p(kfac.PreferenceDesc(**d, **d_out, seq_offsets=0x3000, pairs=1, beta=0.1,
                                                           grad_scale=1.0, loss=0x4000)), *ws)]


@pytest.mark.parametrize("tau", [4e-39, 1e-45])
def test_too_small(lib, tau):
    assert _calls(lib, tau) == [kfac.KFAC_ERR_INVALID] * 4


@pytest.mark.parametrize("tau", [4.3e-39, 1e-38, 1.0, 3.4e38])
def test_valid(lib, tau):
    assert _calls(lib, tau) == [kfac.KFAC_ERR_UNSUPPORTED] * 4
