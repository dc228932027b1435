"""Losses on logits on the GPU against their definitions in 64 bits
(loss_ref.py, which derives the bounds).  Inputs are rounded to the tensor's
type first, so only the kernels' own arithmetic is compared."""
import math

import numpy as np
import pytest
import torch

from second_order_optimisation_gb300 import kfac
from tests import loss_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LOWEST = {"bf16": float(torch.finfo(torch.bfloat16).min), "f16": -65504.0, "f32": float(torch.finfo(torch.float32).min)}
SENTINEL = 7.0


def word(ws):
    torch.cuda.synchronize()
    return int(ws[:4].view(torch.int32).item())


def matrix(a, dtype, ld=None, shift=0, fill=NAN):
    """`a` (or its shape) on the GPU as a view with row pitch ld, starting
    `shift` elements into its buffer; everything else in the buffer is `fill`."""
    rows, cols = a.shape if isinstance(a, np.ndarray) else a
    ld = ld or cols
    buf = torch.full((rows * ld + shift + 16,), fill, dtype=TYPES[dtype], device=DEV)
    v = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    if isinstance(a, np.ndarray):
        v.copy_(torch.from_numpy(a))
    return buf, v


def untouched(buf, view):
    """Nothing of the buffer outside the view was written."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert bool((buf[mask] == SENTINEL).all())


def draw(rows, vocab, dtype, seed, special=True):
    """Logits (64 bits, exactly representable in dtype) and targets, with the
    rows that can go wrong where there is room for them."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 3
    z[:, vocab // 2] += 6
    t = torch.randint(0, vocab, (rows,), generator=g)
    if special and rows >= 7:
        z[1] = -INF                                    # nothing to choose
        z[2, torch.arange(vocab) != vocab // 3] = -INF  # one choice
        t[2] = vocab // 3
        z[3] = LOWEST[dtype]                           # all at the type's lowest value
        z[4, : vocab // 2] = LOWEST[dtype]
        t[4] = vocab - 1
        z[5] = NAN                                     # ignored: NaN must not get out
        t[5] = -1
        z[6, 0] = INF                                  # ignored too
        t[6] = -100
    z = z.to(TYPES[dtype])
    return z.double().numpy(), t.numpy()


def nums(t):
    return t.detach().double().cpu().numpy()


def vec(a, dtype=torch.float32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device=DEV)


def check_grad(got, want, tol, dtype, what="dlogits"):
    with np.errstate(invalid="ignore"):
        ref.close(nums(got), want, tol + ref.ROUND[dtype] * np.abs(want) + ref.TINY[dtype], what)


SHAPES = [(1, 1), (1, 2), (3, 7), (9, 31), (8, 32), (7, 1000), (33, 18), (300, 65), (9, 4097), (8, 8192), (7, 33000),
          (7, 50001), (2, 131077), (7, 262145)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("tau,pad,shift", [(1.0, 0, 0), (0.7, 3, 1)])
def test_logprob_and_its_gradient(dtype, rows, vocab, tau, pad, shift):
    z, t = draw(rows, vocab, dtype, rows * 7 + vocab)
    live = t >= 0
    _, zd = matrix(z, dtype, vocab + pad, shift)
    td = vec(t, torch.int32 if pad else torch.int64)
    logp, lse, h = (torch.full((rows,), SENTINEL, device=DEV) for _ in range(3))
    saved = torch.full((rows, 2), SENTINEL, device=DEV)
    kfac.kfac_token_logprob(kfac.TokenLogprob(zd, td, logp, lse, h, tau, saved))
    r = ref.rows_of(z, t, tau, live)
    ref.close(nums(logp), r["logp"], r["tol"], "logp")
    zmax = np.where(live, np.abs(np.where(np.isfinite(z), z, 0)).max(1), 0) / tau
    ref.close(nums(lse), r["lse"], np.where(np.isfinite(r["lse"]), ref.E * (8 * np.abs(r["lse"]) + 4 * zmax + 128), 0), "lse")
    ref.close(nums(h), r["h"], r["hol"], "entropy")
    only = torch.empty(rows, device=DEV)
    kfac.kfac_token_logprob(kfac.TokenLogprob(zd, td, only, temperature=tau))
    ref.close(nums(only), r["logp"], r["tol"], "logp alone")

    rng = np.random.default_rng(rows)
    g, gh = rng.normal(size=rows).astype(np.float32), rng.normal(size=rows).astype(np.float32)
    if rows > 7:
        g[7] = gh[7] = 0
    for with_h in (True, False):
        for ld_d, shift_d in ((vocab + pad, shift), (vocab + 5, 0)):
            buf, dd = matrix((rows, vocab), dtype, ld_d, shift_d, SENTINEL)
            kfac.kfac_token_logprob_grad(kfac.TokenLogprobGrad(zd, td, saved, vec(g), dd, h if with_h else None,
                                                              vec(gh) if with_h else None, tau))
            want, tol = ref.dlogits(r, t, live, g.astype(float), gh.astype(float) if with_h else None, 1.0, tau)
            check_grad(dd, want, tol, dtype)
            untouched(buf, dd)


def test_logprob_bad_targets_and_nonfinite_logits():
    z = torch.randn(6, 50, device=DEV)
    t = torch.tensor([3, 50, 1 << 40, 4, 5, 6], device=DEV)
    z[3, 10] = NAN
    z[4, 10] = INF
    z[5, 6] = -INF  # the target itself cannot be chosen
    logp, lse, h = (torch.empty(6, device=DEV) for _ in range(3))
    saved = torch.empty(6, 2, device=DEV)
    kfac.kfac_token_logprob(kfac.TokenLogprob(z, t, logp, lse, h, saved=saved))
    assert torch.isnan(logp).tolist() == [False, True, True, True, True, False]
    assert math.isinf(float(logp[5])) and float(logp[5]) < 0
    assert bool(torch.isfinite(h[5])) and bool(torch.isfinite(lse[5]))
    d = torch.full_like(z, SENTINEL)
    kfac.kfac_token_logprob_grad(kfac.TokenLogprobGrad(z, t, saved, torch.ones(6, device=DEV), d))
    assert bool((d[1:3] == 0).all()) and bool(torch.isnan(d[3:5]).any(1).all()) and bool(torch.isfinite(d[5]).all())
    p = torch.softmax(z[5].double(), 0)
    want = -p
    want[6] += 1
    assert float((d[5].double() - want).abs().max()) < 64 * ref.E


@pytest.mark.parametrize("dtype", list(TYPES))
def test_logprob_of_a_target_at_the_lowest_value(dtype):
    z = torch.randn(3, 3000).to(TYPES[dtype])
    z[:, 7] = LOWEST[dtype]
    t = np.array([7, 7, 8])
    zn = z.double().numpy()
    logp, saved, d = torch.empty(3, device=DEV), torch.empty(3, 2, device=DEV), torch.empty_like(z, device=DEV)
    kfac.kfac_token_logprob(kfac.TokenLogprob(z.to(DEV), vec(t, torch.int64), logp, saved=saved))
    r = ref.rows_of(zn, t, 1.0, np.ones(3, bool))
    ref.close(nums(logp), r["logp"], 4 * ref.E * np.abs(r["logp"]) + r["tol"])
    g = np.ones(3)
    kfac.kfac_token_logprob_grad(kfac.TokenLogprobGrad(z.to(DEV), vec(t, torch.int64), saved, vec(g), d))
    r["ymax"][:] = 20  # of the terms that are not 0
    want, tol = ref.dlogits(r, t, np.ones(3, bool), g, None, 1.0, 1.0)
    check_grad(d, want, tol, dtype)


# ------------------------------------------------------------ policy loss

RATIOS = np.array([0.5, 0.75, 0.9, 0.97, 1.03, 1.1, 1.25, 1.6])  # none within 0.03 of a clipping bound


def _policy(dtype, rows, vocab, tau=1.0, pad=0, shift=0, kl=True, ent=0.02, mode="token", seed=0, same_ld=True, scale=1.0,
            outputs=True, z_t=None):
    z, t = z_t if z_t is not None else draw(rows, vocab, dtype, seed + rows * 5 + vocab)
    rng = np.random.default_rng(seed + vocab)
    base = ref.rows_of(z, t, tau, t >= 0)
    lp = np.where(np.isfinite(base["logp"]), base["logp"], 0.0)
    old = (lp - np.log(RATIOS[rng.integers(0, 8, rows)])).astype(np.float32)
    rf = (lp + rng.normal(size=rows) * 0.4).astype(np.float32)
    kw, live, seqs = {}, t >= 0, 0
    if mode in ("seq_token", "seq_mean"):
        cuts = np.sort(rng.integers(0, rows + 1, 3))
        off = np.concatenate([[min(1, rows)], np.maximum(cuts, min(1, rows)), [max(rows - 1, min(1, rows))]]).astype(np.int32)
        seqs = len(off) - 1
        sadv = rng.normal(size=seqs).astype(np.float32)
        seq = np.searchsorted(off, np.arange(rows), side="right") - 1
        inside = (seq >= 0) & (seq < seqs)
        live = live & inside
        adv = np.where(inside, sadv[np.clip(seq, 0, seqs - 1)], 0.0)
        kw.update(seq_offsets=vec(off, torch.int32), seq_mean=mode == "seq_mean")
        advd = vec(sadv)
        if mode == "seq_mean":
            n = np.array([max(1, (live & (seq == s)).sum()) for s in range(seqs)])
            w = np.where(live, 1.0 / (seqs * n[np.clip(seq, 0, seqs - 1)]), 0.0)
    else:
        adv = rng.normal(size=rows).astype(np.float32)
        advd = vec(adv)
    if mode == "weight":
        w = rng.uniform(0.2, 1, rows).astype(np.float32)
        w[rng.random(rows) < 0.2] = 0
        kw["weight"] = vec(w)
        live = live & (w != 0)
        w = np.where(live, w.astype(float), 0)
    elif mode in ("token", "seq_token"):
        w = live / max(1, live.sum())
    _, zd = matrix(z, dtype, vocab + pad, shift)
    buf, dd = matrix((rows, vocab), dtype, vocab + pad if same_ld else vocab + 5, shift if same_ld else 0, SENTINEL)
    stats = torch.full((5,), SENTINEL, device=DEV)
    logp, klo, h = ((torch.full((rows,), SENTINEL, device=DEV) for _ in range(3)) if outputs else (None, None, None))
    ws = kfac.kfac_policy_loss(kfac.PolicyLoss(
        zd, vec(t, torch.int64), advd, vec(old), stats, logp, dd, vec(rf) if kl else None, kl=klo if kl else None, entropy=h,
        clip_low=0.2, clip_high=0.2, kl_coef=0.3 if kl else 0.0, entropy_coef=ent, temperature=tau, grad_scale=scale, **kw))
    want = ref.policy(z, t, live, adv.astype(float), old.astype(float), rf.astype(float) if kl else None, w, 0.2, 0.2,
                      0.3 if kl else 0.0, ent, scale, tau)
    r = want["r"]
    st = nums(stats)
    if not (outputs or ent):  # no entropy was asked for
        want["stats"][3] = 0
    ref.close(st, want["stats"], want["stol"], "stats")
    if outputs:
        ref.close(nums(logp), r["logp"], r["tol"], "logp")
        ref.close(nums(h), r["h"], r["hol"], "entropy")
        if kl:
            d = np.where(live & ~r["none"], rf - np.where(np.isfinite(r["logp"]), r["logp"], 0), 0)
            ref.close(nums(klo), want["kl"], (np.exp(d) + 1 + np.abs(d)) * (r["tol"] + 16 * ref.E), "kl")
    check_grad(dd, want["d"], want["tol"], dtype)
    untouched(buf, dd)
    expect = kfac.ERRW_NONFINITE if (live & r["none"]).any() else 0
    assert word(ws) == expect


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_policy_shapes(dtype, rows, vocab):
    _policy(dtype, rows, vocab)


@pytest.mark.parametrize("rows,vocab", [(1100, 18), (9, 4097), (7, 33000)])
@pytest.mark.parametrize("mode", ["token", "weight", "seq_token", "seq_mean"])
@pytest.mark.parametrize("kl,ent", [(True, 0.0), (False, 0.05)])
def test_policy_weights_and_terms(rows, vocab, mode, kl, ent):
    _policy("bf16", rows, vocab, kl=kl, ent=ent, mode=mode, outputs=mode != "token", seed=3)


@pytest.mark.parametrize("rows,vocab,dtype", [(20001, 18, "f32"), (4703, 5003, "bf16")])
@pytest.mark.parametrize("mode", ["token", "weight", "seq_token", "seq_mean"])
def test_policy_many_rows(rows, vocab, dtype, mode):
    """More rows than one pass over their table takes, in order (the second) and not."""
    _policy(dtype, rows, vocab, mode=mode, seed=5)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [5, 31, 1000, 33000, 50001])
@pytest.mark.parametrize("pad,shift,same", [(3, 1, True), (0, 0, False), (8, 4, True), (1, 3, False)])
def test_policy_strides(dtype, vocab, pad, shift, same):
    _policy(dtype, 9, vocab, tau=1.3, pad=pad, shift=shift, same_ld=same, scale=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_policy_longest_rows(dtype):
    """Rows past what one cluster keeps on the chip."""
    _policy(dtype, 2, 1_500_003, z_t=draw(2, 1_500_003, dtype, 3, special=False))


def test_policy_without_rows_and_without_counted_rows():
    stats = torch.full((5,), SENTINEL, device=DEV)
    e = torch.empty(0, device=DEV)
    ws = kfac.kfac_policy_loss(kfac.PolicyLoss(torch.empty(0, 10, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), e, e, stats))
    assert word(ws) == 0 and bool((stats == 0).all())
    z = torch.full((5, 40), NAN, device=DEV)
    t = torch.full((5,), -1, device=DEV)
    d = torch.full_like(z, SENTINEL)
    v = torch.full((5,), NAN, device=DEV)
    logp = torch.full((5,), SENTINEL, device=DEV)
    ws = kfac.kfac_policy_loss(kfac.PolicyLoss(z, t, v, v, stats, logp, d, ref_logp=v, kl_coef=0.1, entropy_coef=0.1))
    assert word(ws) == 0 and bool((stats == 0).all()) and bool((d == 0).all()) and bool((logp == 0).all())


def test_policy_error_word():
    def call(**kw):
        z = torch.randn(4, 33, device=DEV)
        t = torch.tensor([1, 2, 3, 4], device=DEV)
        if "z" in kw:
            z[1, 5] = kw["z"]
        if "t" in kw:
            t[2] = kw["t"]
        old = torch.full((4,), -3.0, device=DEV)
        if "old" in kw:
            old[0] = kw["old"]
        d, stats = torch.full_like(z, SENTINEL), torch.empty(5, device=DEV)
        ws = kfac.kfac_policy_loss(kfac.PolicyLoss(z, t, torch.ones(4, device=DEV), old, stats, dlogits=d))
        return word(ws), d, stats

    assert call()[0] == 0
    for bad in (NAN, INF):
        w, d, stats = call(z=bad)
        assert w == kfac.ERRW_NONFINITE and bool(torch.isnan(stats[0]))
        assert bool(torch.isnan(d[1]).any()) and bool(torch.isfinite(d[[0, 2, 3]]).all())
    w, d, stats = call(t=33)
    assert w == kfac.ERRW_TARGET and bool((d[2] == 0).all()) and bool(torch.isfinite(stats).all())
    w, d, stats = call(t=1 << 33, z=NAN)
    assert w == kfac.ERRW_TARGET | kfac.ERRW_NONFINITE
    assert call(z=-INF)[0] == 0
    assert call(old=NAN)[0] == kfac.ERRW_NONFINITE


# ------------------------------------------------------------ preference loss

def _preference(dtype, rows, vocab, off, kind="sigmoid", smooth=0.0, average=False, tau=1.0, pad=0, shift=0, same_ld=True,
                weights=False, reference=True, seed=1, special=True, scale=1.0):
    z, t = draw(rows, vocab, dtype, seed + vocab, special)
    off = np.asarray(off, np.int32)
    pairs = (len(off) - 1) // 2
    rng = np.random.default_rng(seed)
    at = np.arange(rows)
    live = (t >= 0) & (at >= off[0]) & (at < off[-1])
    beta = 0.3
    r0 = ref.preference(z, t, live, off, np.zeros(2 * pairs), np.ones(pairs), kind, beta, smooth, average, 1.0, tau)
    # the margin h is of order 1, and beta h not near the hinge
    rf = np.zeros(2 * pairs, np.float32)
    if reference:
        rf = (r0["l"] + rng.uniform(0.3, 2.0, 2 * pairs) * np.tile([1, -1], pairs)).astype(np.float32)
    pw = rng.uniform(0.3, 1, pairs).astype(np.float32) if weights else np.full(pairs, 1 / pairs)
    _, zd = matrix(z, dtype, vocab + pad, shift)
    buf, dd = matrix((rows, vocab), dtype, vocab + pad if same_ld else vocab + 5, shift if same_ld else 0, SENTINEL)
    loss = torch.full((1,), SENTINEL, device=DEV)
    pl, sl, tl = (torch.full((n,), SENTINEL, device=DEV) for n in (pairs, 2 * pairs, rows))
    ws = kfac.kfac_preference_loss(kfac.PreferenceLoss(
        zd, vec(t, torch.int64), vec(off, torch.int32), loss, sl, dd, vec(rf) if reference else None,
        vec(pw) if weights else None, pl, tl, kind, beta, smooth, average, tau, scale))
    want = ref.preference(z, t, live, off, rf.astype(float), pw.astype(float), kind, beta, smooth, average, scale, tau)
    ref.close(nums(tl), want["r"]["logp"], want["r"]["tol"], "token_logp")
    ref.close(nums(sl), want["l"], want["ltol"], "seq_logp")
    ref.close(nums(pl), want["f"], want["ftol"], "pair_loss")
    ref.close(nums(loss), [want["loss"]], want["losstol"], "loss")
    check_grad(dd, want["d"], want["tol"], dtype)
    untouched(buf, dd)
    assert word(ws) == (kfac.ERRW_NONFINITE if (live & want["r"]["none"]).any() else 0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab,off", [
    (2, 1, [0, 1, 2]), (1, 5, [0, 1, 1]), (3, 7, [0, 0, 3]), (9, 31, [0, 4, 4, 6, 9]), (20, 1000, [1, 8, 13, 13, 18]),
    (40, 4097, [0, 10, 25, 30, 40]), (8, 50001, [0, 3, 8]), (7, 131077, [0, 2, 7]), (300, 65, list(range(0, 301, 25))),
    (12, 64, [0, 0, 0, 6, 6])])
def test_preference_shapes(dtype, rows, vocab, off):
    _preference(dtype, rows, vocab, off)


@pytest.mark.parametrize("kind,smooth", [("sigmoid", 0.0), ("sigmoid", 0.15), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_preference_kinds(kind, smooth, average, weights):
    _preference("bf16", 30, 517, [0, 9, 17, 20, 29], kind, smooth, average, tau=0.8, weights=weights, scale=3.0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,shift,same", [(3, 1, True), (0, 0, False), (8, 4, True)])
def test_preference_strides(dtype, pad, shift, same):
    _preference(dtype, 20, 1001, [0, 6, 20], pad=pad, shift=shift, same_ld=same)


def test_preference_without_reference_and_longest_rows():
    _preference("bf16", 6, 40, [0, 3, 6], reference=False, special=False)
    _preference("bf16", 2, 1_500_003, [0, 1, 2], special=False)


def test_preference_many_pairs_over_many_rows():
    """More rows than one pass over the SMs takes, sequences of very different lengths."""
    rng = np.random.default_rng(2)
    off = np.concatenate([[0], np.sort(rng.integers(0, 2001, 31)), [2001]])
    _preference("bf16", 2001, 259, off, "ipo", average=True)


def test_preference_offsets_out_of_range_stay_in_bounds():
    """Offsets past the rows, or negative, are read as the nearest valid row."""
    z, t = torch.randn(6, 20, device=DEV), torch.randint(0, 20, (6,), device=DEV)
    res = []
    for off in ([0, 2, 6], [-5, 2, 1 << 30]):
        loss, d = torch.empty(1, device=DEV), torch.empty_like(z)
        kfac.kfac_preference_loss(kfac.PreferenceLoss(z, t, torch.tensor(off, dtype=torch.int32, device=DEV), loss, dlogits=d))
        res.append((loss, d))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_preference_error_word():
    def call(bad=None, target=None, inside=True):
        z, t = torch.randn(8, 33, device=DEV), torch.arange(8, device=DEV)
        row = 1 if inside else 7
        if bad is not None:
            z[row, 5] = bad
        if target is not None:
            t[row] = target
        loss, d = torch.empty(1, device=DEV), torch.full_like(z, SENTINEL)
        ws = kfac.kfac_preference_loss(kfac.PreferenceLoss(
            z, t, torch.tensor([0, 2, 4, 5, 7], dtype=torch.int32, device=DEV), loss, dlogits=d))
        return word(ws), loss, d

    assert call()[0] == 0
    w, loss, d = call(NAN)
    assert w == kfac.ERRW_NONFINITE and bool(torch.isnan(loss).all()) and bool(torch.isfinite(d[4:]).all())
    w, loss, d = call(target=33)
    assert w == kfac.ERRW_TARGET and bool(torch.isfinite(loss).all()) and bool((d[1] == 0).all())
    w, loss, d = call(NAN, inside=False)  # a row of no sequence is not read
    assert w == 0 and bool((d[7] == 0).all()) and bool(torch.isfinite(loss).all())


# ------------------------------------------------------------ how they are called

def _both_losses(z, t, off, ws=(None, None), stream=None):
    n = z.shape[0]
    o = [torch.empty(5, device=DEV), torch.empty(n, device=DEV), torch.empty_like(z), torch.empty(1, device=DEV),
         torch.empty_like(z)]
    old = torch.full((n,), -5.0, device=DEV)
    a = kfac.PolicyLoss(z, t, torch.ones(n, device=DEV), old, o[0], o[1], o[2], entropy_coef=0.01)
    b = kfac.PreferenceLoss(z, t, off, o[3], dlogits=o[4])

    def run():
        kfac.kfac_policy_loss(a, ws[0], stream)
        kfac.kfac_preference_loss(b, ws[1], stream)
    return run, o, a, b


@pytest.mark.parametrize("rows,vocab", [(64, 18), (70, 5003), (33, 70001)])
def test_repeatable_on_dirty_workspaces_streams_and_graphs(rows, vocab):
    g = torch.Generator(device=DEV).manual_seed(rows)
    z = torch.randn(rows, vocab, device=DEV, generator=g).bfloat16()
    t = torch.randint(-1, vocab, (rows,), device=DEV, generator=g)
    off = torch.tensor([0, rows // 3, rows // 2, rows // 2, rows], dtype=torch.int32, device=DEV)
    run, want, a, b = _both_losses(z, t, off)
    run()
    torch.cuda.synchronize()
    ws = [torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV) for n in
          (kfac.kfac_policy_loss_workspace_size(a), kfac.kfac_preference_loss_workspace_size(b))]
    run2, o, *_ = _both_losses(z, t, off, ws)
    for _ in range(3):
        run2()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(o, want))
    assert all(bool((w[-256:] == 0xA5).all()) for w in ws)       # nothing past the workspace
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run3, o, *_ = _both_losses(z, t, off, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    run3()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(o, want))
    run4, o, *_ = _both_losses(z, t, off, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run4()
    for _ in range(2):
        for x in o:
            x.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(o, want))


def test_offsets_past_two_to_the_31():
    """Rows whose first element lies past 2^31 elements."""
    rows, vocab = 16500, 131072
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device=DEV)
    t = torch.full((rows,), -1, device=DEV)
    pick = [0, 1, 16383, 16384, 16385, rows - 1]
    g = torch.Generator(device=DEV).manual_seed(1)
    for i in pick:
        z[i] = torch.randn(vocab, device=DEV, generator=g).bfloat16()
        t[i] = (i * 37) % vocab
    d = torch.full_like(z, SENTINEL)
    stats, logp = torch.empty(5, device=DEV), torch.empty(rows, device=DEV)
    old = torch.full((rows,), -12.0, device=DEV)
    kfac.kfac_policy_loss(kfac.PolicyLoss(z, t, torch.ones(rows, device=DEV), old, stats, logp, d))
    small, ds, lps = z[pick].contiguous(), torch.empty(6, vocab, dtype=z.dtype, device=DEV), torch.empty(6, device=DEV)
    kfac.kfac_policy_loss(kfac.PolicyLoss(small, t[pick].contiguous(), torch.ones(6, device=DEV), old[:6].contiguous(), stats, lps, ds))
    assert torch.equal(logp[pick], lps) and torch.equal(d[pick], ds)
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[pick] = False
    assert int((d.view(torch.int16).ne(0).any(1) & rest).sum()) == 0


@pytest.mark.parametrize("vocab", [10, 70001])
def test_preference_without_rows(vocab):
    loss, pl = torch.full((1,), SENTINEL, device=DEV), torch.full((2,), SENTINEL, device=DEV)
    ws = kfac.kfac_preference_loss(kfac.PreferenceLoss(
        torch.empty(0, vocab, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV),
        torch.zeros(5, dtype=torch.int32, device=DEV), loss, pair_loss=pl))
    assert word(ws) == 0
    assert abs(float(loss) - math.log(2)) < 4 * ref.E and torch.allclose(pl, loss.expand(2), atol=4 * ref.E, rtol=0)
