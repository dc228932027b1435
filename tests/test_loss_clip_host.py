"""Losses on logits and clipping, without a GPU: what the entry points refuse,
and that the 64-bit reference's gradients are the differences of its losses."""
import ctypes

import numpy as np
import pytest
import torch

from tests import loss_ref as ref
from second_order_optimisation_gb300 import kfac

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kfac.load()


# ------------------------------------------------------------ the reference itself

def _differences(loss, z, eps=1e-5):
    d = np.zeros_like(z)
    for i in np.ndindex(*z.shape):
        if not np.isfinite(z[i]):
            continue
        a, b = z.copy(), z.copy()
        a[i] += eps
        b[i] -= eps
        d[i] = (loss(a) - loss(b)) / (2 * eps)
    return d


@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_policy_reference_gradient_is_the_difference(tau):
    rng = np.random.default_rng(5)
    z = rng.normal(size=(7, 6)) * 2
    z[2, 1] = -INF
    t = np.array([0, 5, 3, 2, 0, 1, 4])
    live = np.array([1, 1, 1, 0, 1, 1, 1], bool)
    lp = ref.rows_of(z, t, tau, live)["logp"]
    old = lp - np.log([0.5, 0.9, 1.5, 1, 1.1, 1.3, 0.7])
    adv = np.array([1.0, -2, 0.5, 1, 1, -1, -0.3])
    w = np.where(live, rng.uniform(0.5, 1, 7), 0)

    def run(x):
        return ref.policy(x, t, live, adv, old, lp + 0.3, w, 0.2, 0.25, 0.1, 0.02, 3.0, tau)

    d = _differences(lambda x: 3.0 * run(x)["stats"][0], z)
    assert np.abs(d - run(z)["d"]).max() < 1e-8 * 50


@pytest.mark.parametrize("kind,smooth", [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_reference_gradient_is_the_difference(kind, smooth, average):
    rng = np.random.default_rng(6)
    z = rng.normal(size=(9, 5))
    t = rng.integers(0, 5, 9)
    live = np.array([1, 1, 0, 1, 1, 1, 1, 1, 1], bool)
    off = np.array([0, 3, 5, 5, 8])  # one sequence empty, row 8 of none
    r = rng.normal(size=4) - 3
    pw = np.array([0.4, 0.6])
    inside = live & (np.arange(9) < 8)

    def run(x):
        return ref.preference(x, t, inside, off, r, pw, kind, 0.3, smooth, average, 2.0, 1.0)

    d = _differences(lambda x: 2.0 * run(x)["loss"], z)
    assert np.abs(d - run(z)["d"]).max() < 1e-8 * 50


# ------------------------------------------------------------ refusals

def _lp(**kw):
    d = dict(dtype=kfac.KFAC_BF16, logits=0x1000, ld=100, rows=4, vocab=100, target=0x2000, target_i32=0,
             temperature=1.0, logp=0x3000)
    d.update(kw)
    return kfac.LogprobDesc(**d)


LOGITS_BAD = [dict(logits=None), dict(target=None), dict(rows=-1), dict(vocab=0), dict(ld=99), dict(dtype=7),
              dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=NAN), dict(temperature=INF),
              dict(logits=0x1001)]


@pytest.mark.parametrize("bad", LOGITS_BAD + [dict(logp=None), dict(saved=0x3004)])
def test_logprob_refuses(lib, bad):
    assert lib.kfac_token_logprob(ctypes.byref(_lp(**bad)), None) == kfac.KFAC_ERR_INVALID


def test_logprob_limits_and_nothing_to_do(lib):
    assert lib.kfac_token_logprob(None, None) == kfac.KFAC_ERR_INVALID
    big = (1 << 24) + 1
    assert lib.kfac_token_logprob(ctypes.byref(_lp(vocab=big, ld=big)), None) == kfac.KFAC_ERR_UNSUPPORTED
    assert lib.kfac_token_logprob(ctypes.byref(_lp(rows=1 << 31)), None) == kfac.KFAC_ERR_UNSUPPORTED
    assert lib.kfac_token_logprob(ctypes.byref(_lp(rows=0, logits=None, target=None)), None) == kfac.KFAC_OK
    # pointers that are not device memory
    assert lib.kfac_token_logprob(ctypes.byref(_lp()), None) == kfac.KFAC_ERR_INVALID


def _lg(**kw):
    d = dict(dtype=kfac.KFAC_BF16, logits=0x1000, ld=100, rows=4, vocab=100, target=0x2000, target_i32=0,
             temperature=1.0, saved=0x3000, dlogp=0x4000, dlogits=0x5000, ld_d=100)
    d.update(kw)
    return kfac.LogprobGradDesc(**d)


@pytest.mark.parametrize("bad", LOGITS_BAD + [dict(saved=None), dict(saved=0x3004), dict(dlogp=None), dict(dlogits=None), dict(ld_d=99),
                                              dict(dlogits=0x5001), dict(dentropy=0x6000)])
def test_logprob_grad_refuses(lib, bad):
    assert lib.kfac_token_logprob_grad(ctypes.byref(_lg(**bad)), None) == kfac.KFAC_ERR_INVALID


def _po(**kw):
    d = dict(dtype=kfac.KFAC_BF16, logits=0x1000, ld=100, rows=4, vocab=100, target=0x2000, target_i32=0,
             temperature=1.0, advantage=0x3000, old_logp=0x4000, clip_low=0.2, clip_high=0.2, grad_scale=1.0,
             stats=0x5000, dlogits=0x6000, ld_d=100)
    d.update(kw)
    return kfac.PolicyDesc(**d)


@pytest.mark.parametrize("bad", LOGITS_BAD + [
    dict(advantage=None), dict(old_logp=None), dict(stats=None), dict(ld_d=99), dict(dlogits=0x6001),
    dict(clip_low=-0.1), dict(clip_high=NAN), dict(kl_coef=0.1), dict(kl=0x7000), dict(kl_coef=INF, ref_logp=0x7000),
    dict(entropy_coef=NAN), dict(grad_scale=INF), dict(seq_offsets=0x7000, seqs=0), dict(seq_mean=1),
    dict(seq_mean=1, seq_offsets=0x7000, seqs=2, weight=0x8000)])
def test_policy_refuses(lib, bad):
    d = _po(**bad)
    assert lib.kfac_policy_loss(ctypes.byref(d), 0x100000, 1 << 30, None) == kfac.KFAC_ERR_INVALID
    assert lib.kfac_policy_loss_workspace_size(ctypes.byref(d)) == 0


def _pr(**kw):
    d = dict(dtype=kfac.KFAC_BF16, logits=0x1000, ld=100, rows=4, vocab=100, target=0x2000, target_i32=0,
             temperature=1.0, seq_offsets=0x3000, pairs=1, beta=0.1, grad_scale=1.0, loss=0x4000, dlogits=0x5000, ld_d=100)
    d.update(kw)
    return kfac.PreferenceDesc(**d)


@pytest.mark.parametrize("bad", LOGITS_BAD + [
    dict(seq_offsets=None), dict(loss=None), dict(pairs=0), dict(ld_d=99), dict(dlogits=0x5001), dict(kind=3),
    dict(kind=-1), dict(beta=0.0), dict(beta=NAN), dict(beta=INF), dict(label_smoothing=1.0),
    dict(label_smoothing=-0.1), dict(label_smoothing=0.1, kind=1), dict(grad_scale=NAN)])
def test_preference_refuses(lib, bad):
    d = _pr(**bad)
    assert lib.kfac_preference_loss(ctypes.byref(d), 0x100000, 1 << 30, None) == kfac.KFAC_ERR_INVALID
    assert lib.kfac_preference_loss_workspace_size(ctypes.byref(d)) == 0


@pytest.mark.parametrize("make,run,size", [(_po, "kfac_policy_loss", "kfac_policy_loss_workspace_size"),
                                           (_pr, "kfac_preference_loss", "kfac_preference_loss_workspace_size")])
def test_loss_workspaces(lib, make, run, size):
    d = make()
    need = getattr(lib, size)(ctypes.byref(d))
    assert need > 0
    call = getattr(lib, run)
    assert call(ctypes.byref(d), None, 0, None) == kfac.KFAC_ERR_WORKSPACE
    assert call(ctypes.byref(d), 0x100001, need, None) == kfac.KFAC_ERR_WORKSPACE
    assert call(ctypes.byref(d), 0x100000, need - 256, None) == kfac.KFAC_ERR_WORKSPACE
    assert call(ctypes.byref(d), 0x100000, need, None) == kfac.KFAC_ERR_INVALID  # not device memory
    assert call(None, 0x100000, need, None) == kfac.KFAC_ERR_INVALID


def _cl(**kw):
    d = dict(x=0x1000, ld=10, rows=3, cols=10, dtype=kfac.KFAC_F32, y_dtype=kfac.KFAC_F32, out=0x2000, ld_out=10, out_dtype=kfac.KFAC_F32)
    d.update(kw)
    return (kfac.ClipDesc * 1)(kfac.ClipDesc(**d))


@pytest.mark.parametrize("bad", [dict(x=None), dict(ld=9), dict(rows=-1), dict(cols=-1), dict(dtype=9),
                                 dict(out_dtype=9), dict(ld_out=9), dict(y=0x3000, ld_y=9), dict(w=0x3000, ld_w=9),
                                 dict(x=0x1002), dict(w=0x3002, ld_w=10), dict(y=0x3002, ld_y=10), dict(y=0x3000, ld_y=10, y_dtype=9),
                                 dict(dtype=kfac.KFAC_BF16, y=0x3000, ld_y=10), dict(dtype=kfac.KFAC_F16, y=0x3000, ld_y=10, y_dtype=kfac.KFAC_BF16),
                                 dict(out=0x1000, out_dtype=kfac.KFAC_BF16), dict(out=0x1000, ld_out=11)])
def test_clip_refuses(lib, bad):
    arr = _cl(**bad)
    assert lib.kfac_clip_norm(arr, 1, 1.0, 0.0, None, None, 0x100000, 1 << 20, None) == kfac.KFAC_ERR_INVALID
    assert lib.kfac_clip_norm_workspace_size(arr, 1) == 0


def test_clip_refuses_scalars_and_workspaces(lib):
    arr = _cl()
    for max_norm, eta in ((0.0, 0.0), (-1.0, 0.0), (NAN, 0.0), (1.0, NAN), (1.0, INF)):
        assert lib.kfac_clip_norm(arr, 1, max_norm, eta, None, None, 0x100000, 1 << 20, None) == kfac.KFAC_ERR_INVALID
    need = lib.kfac_clip_norm_workspace_size(arr, 1)
    assert need > 0 and lib.kfac_clip_norm_workspace_size(None, 0) > 0
    assert lib.kfac_clip_norm(arr, 1, 1.0, 0.0, None, None, None, 0, None) == kfac.KFAC_ERR_WORKSPACE
    assert lib.kfac_clip_norm(arr, 1, 1.0, 0.0, None, None, 0x100010, need, None) == kfac.KFAC_ERR_WORKSPACE
    assert lib.kfac_clip_norm(arr, 1, 1.0, 0.0, None, None, 0x100000, need - 256, None) == kfac.KFAC_ERR_WORKSPACE
    assert lib.kfac_clip_norm(arr, 1, 1.0, 0.0, None, None, 0x100000, need, None) == kfac.KFAC_ERR_INVALID
    assert lib.kfac_clip_norm(arr, -1, 1.0, 0.0, None, None, 0x100000, need, None) == kfac.KFAC_ERR_INVALID
    assert lib.kfac_clip_norm(None, 1, 1.0, 0.0, None, None, 0x100000, need, None) == kfac.KFAC_ERR_INVALID


def test_binding_refuses():
    z, t, o = torch.zeros(4, 6), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(TypeError):
        kfac.kfac_token_logprob(kfac.TokenLogprob(z.double(), t, o))
    with pytest.raises(TypeError):
        kfac.kfac_token_logprob(kfac.TokenLogprob(z, t.short(), o))
    with pytest.raises(ValueError):
        kfac.kfac_token_logprob(kfac.TokenLogprob(torch.zeros(6, 4).t(), t, o))
    with pytest.raises(ValueError):
        kfac.kfac_token_logprob(kfac.TokenLogprob(z, t[:3], o))
    with pytest.raises(ValueError):
        kfac.kfac_token_logprob(kfac.TokenLogprob(z, t, torch.zeros(8)[::2]))
    with pytest.raises(TypeError):
        kfac.kfac_token_logprob_grad(kfac.TokenLogprobGrad(z, t, torch.zeros(4, 2), o, z.half()))
    with pytest.raises(ValueError):
        kfac.kfac_preference_loss(kfac.PreferenceLoss(z, t, torch.zeros(4, dtype=torch.int32), o[:1]))
    with pytest.raises(ValueError):
        kfac.kfac_preference_loss(kfac.PreferenceLoss(z, t, torch.zeros(3, dtype=torch.int32), o[:1], kind="other"))
    with pytest.raises(TypeError):
        kfac.kfac_preference_loss(kfac.PreferenceLoss(z, t, torch.zeros(3), o[:1]))
    with pytest.raises(ValueError):
        kfac.ClipList([kfac.ClipTensor(z, torch.zeros(6, 4))])
    with pytest.raises(ValueError):
        kfac.ClipList([kfac.ClipTensor(torch.zeros(6, 4).t())])
    with pytest.raises(TypeError):
        kfac.ClipList([kfac.ClipTensor(z.half(), y=z)])
    with pytest.raises(TypeError):
        kfac.ClipList([kfac.ClipTensor(z, w=z.half())])
