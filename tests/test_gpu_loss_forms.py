"""Forms of the losses that are called apart from the usual ones: without a
gradient, with 32-bit targets, on other streams.  Bounds as in loss_ref.py."""
import numpy as np
import pytest
import torch

from second_order_optimisation_gb300 import kfac
from tests import loss_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF = float("inf")
# small kernels, rows by warps, a CTA to a row, clusters of several sizes, more rows than CTAs
SHAPES = [(5, 1), (9, 31), (300, 65), (20, 1000), (200, 3001), (1300, 9001), (9, 4097), (7, 33000), (40, 50001), (7, 262145)]


def _draw(rows, vocab, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(rows, vocab, generator=g) * 2).to(TYPES[dtype])
    t = torch.randint(0, vocab, (rows,), generator=g)
    if rows >= 7 and vocab > 2:
        z[1] = -INF                     # nothing to choose
        z[2, torch.arange(vocab) != t[2]] = -INF
        z[3] = float("nan")             # ignored
        t[3] = -1
    return z, z.double().numpy(), t


def vec(a, dtype=torch.float32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device=DEV)


def nums(t):
    return t.detach().double().cpu().numpy()


def word(ws):
    torch.cuda.synchronize()
    return int(ws[:4].view(torch.int32).item())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("index,gradient", [(torch.int32, True), (torch.int32, False), (torch.int64, False)])
@pytest.mark.parametrize("ent", [0.0, 0.02])
def test_policy(dtype, rows, vocab, index, gradient, ent):
    z, zn, t = _draw(rows, vocab, dtype, rows + vocab)
    tn, tau = t.numpy(), 0.9
    live = tn >= 0
    rng = np.random.default_rng(vocab)
    lp = ref.rows_of(zn, tn, tau, live)["logp"]
    lp = np.where(np.isfinite(lp), lp, 0.0)
    old = (lp - np.log(np.array([0.5, 0.9, 1.1, 1.6])[rng.integers(0, 4, rows)])).astype(np.float32)
    rf = (lp + rng.normal(size=rows) * 0.4).astype(np.float32)
    adv = rng.normal(size=rows).astype(np.float32)
    w = live / max(1, live.sum())
    zd = z.to(DEV)
    stats, logp, kl = (torch.full((n,), 7.0, device=DEV) for n in (5, rows, rows))
    d = torch.full_like(zd, 7.0) if gradient else None
    ws = kfac.kfac_policy_loss(kfac.PolicyLoss(
        zd, t.to(DEV, index), vec(adv), vec(old), stats, logp, d, vec(rf), kl=kl, kl_coef=0.3, entropy_coef=ent, temperature=tau))
    want = ref.policy(zn, tn, live, adv.astype(float), old.astype(float), rf.astype(float), w, 0.2, 0.2, 0.3, ent, 1.0, tau)
    r = want["r"]
    if not ent:
        want["stats"][3] = 0
    ref.close(nums(stats), want["stats"], want["stol"], "stats")
    ref.close(nums(logp), r["logp"], r["tol"], "logp")
    diff = np.where(live & ~r["none"], rf - np.where(np.isfinite(r["logp"]), r["logp"], 0), 0)
    ref.close(nums(kl), want["kl"], (np.exp(diff) + 1 + np.abs(diff)) * (r["tol"] + 16 * ref.E), "kl")
    if gradient:
        ref.close(nums(d), want["d"], want["tol"] + ref.ROUND[dtype] * np.abs(want["d"]) + ref.TINY[dtype], "dlogits")
    assert word(ws) == (kfac.ERRW_NONFINITE if (live & r["none"]).any() else 0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("index,gradient", [(torch.int32, True), (torch.int32, False), (torch.int64, False)])
def test_preference(dtype, rows, vocab, index, gradient):
    z, zn, t = _draw(rows, vocab, dtype, rows + vocab)
    tn, tau = t.numpy(), 1.1
    off = np.array([0, rows // 3, rows // 2, rows // 2, rows - 1], np.int32)  # one sequence empty, the last row of none
    live = (tn >= 0) & (np.arange(rows) < off[-1])
    r0 = ref.preference(zn, tn, live, off, np.zeros(4), np.ones(2), "sigmoid", 0.3, 0.1, True, 1.0, tau)
    rf = (r0["l"] + np.array([0.4, -0.9, 1.3, -0.2])).astype(np.float32)
    zd = z.to(DEV)
    loss, pl, sl, tl = (torch.full((n,), 7.0, device=DEV) for n in (1, 2, 4, rows))
    d = torch.full_like(zd, 7.0) if gradient else None
    ws = kfac.kfac_preference_loss(kfac.PreferenceLoss(
        zd, t.to(DEV, index), vec(off, torch.int32), loss, sl, d, vec(rf), None, pl, tl, "sigmoid", 0.3, 0.1, True, tau))
    want = ref.preference(zn, tn, live, off, rf.astype(float), np.full(2, 0.5), "sigmoid", 0.3, 0.1, True, 1.0, tau)
    ref.close(nums(tl), want["r"]["logp"], want["r"]["tol"], "token_logp")
    ref.close(nums(sl), want["l"], want["ltol"], "seq_logp")
    ref.close(nums(pl), want["f"], want["ftol"], "pair_loss")
    ref.close(nums(loss), [want["loss"]], want["losstol"], "loss")
    if gradient:
        ref.close(nums(d), want["d"], want["tol"] + ref.ROUND[dtype] * np.abs(want["d"]) + ref.TINY[dtype], "dlogits")
    assert word(ws) == (kfac.ERRW_NONFINITE if (live & want["r"]["none"]).any() else 0)


@pytest.mark.parametrize("rows,vocab", [(9, 31), (200, 3001), (7, 33000)])
def test_32_bit_targets_past_the_vocabulary(rows, vocab):
    z = torch.randn(rows, vocab, device=DEV)
    t = torch.zeros(rows, dtype=torch.int32, device=DEV)
    t[3], t[4] = vocab, -(1 << 31)
    old, stats = torch.full((rows,), -3.0, device=DEV), torch.empty(5, device=DEV)
    d = torch.full_like(z, 7.0)
    assert word(kfac.kfac_policy_loss(kfac.PolicyLoss(z, t, old, old, stats, dlogits=d))) == kfac.ERRW_TARGET
    assert bool((d[3:5] == 0).all()) and bool(torch.isfinite(d).all())
    loss, d = torch.empty(1, device=DEV), torch.full_like(z, 7.0)
    off = torch.tensor([0, 5, rows], dtype=torch.int32, device=DEV)
    assert word(kfac.kfac_preference_loss(kfac.PreferenceLoss(z, t, off, loss, dlogits=d))) == kfac.ERRW_TARGET
    assert bool((d[3:5] == 0).all()) and bool(torch.isfinite(d).all())


def test_the_current_stream_is_the_default():
    assert kfac._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert kfac._stream(None) == side.cuda_stream
    assert kfac._stream(side) == kfac._stream(side.cuda_stream) == side.cuda_stream
