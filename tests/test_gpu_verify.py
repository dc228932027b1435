"""The verification of drafted tokens on the GPU against its rules in 64 bits.

The accepted and new tokens have to be equal: the inputs are drawn from fixed seeds, and
next to no two quotients or sides of a comparison are as near as fp32's error (1e-6)."""
import numpy as np
import pytest
import torch

from tests import verify_ref as ref
from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


def _inputs(off, vocab, dtype, seed=0, near=0.7):
    rng = np.random.default_rng(seed)
    rows = off[-1]
    z = torch.from_numpy(rng.normal(size=(rows, vocab)) * 2).to(DT[dtype])
    zd = (z.double() + near * torch.from_numpy(rng.normal(size=(rows, vocab)))).to(DT[dtype])
    e = rng.exponential(size=(rows, vocab))
    tokens = (zd.double().numpy() - np.log(e)).argmax(1)
    u = torch.from_numpy(rng.random(rows)).float()
    noise = torch.from_numpy(rng.exponential(size=(len(off) - 1, vocab))).float()
    return z, zd, torch.from_numpy(tokens), u, noise


def _run(z, tokens, off, u=None, noise=None, zd=None, saved=None, inplace=False, ws=None, stream=None, **kw):
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    z, tokens, u, noise, zd, saved = map(cuda, (z, tokens, u, noise, zd, saved))
    seqs = len(off) - 1
    accepted = torch.full((seqs,), -5, dtype=torch.int32, device="cuda")
    out = tokens if inplace else torch.full_like(tokens, -7)
    logp = torch.full((len(tokens),), 5.0, device="cuda")
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = kfac.kfac_verify_draft(kfac.VerifyDraft(z, tokens, offsets, accepted, out, logp, zd, saved, u, noise, **kw), ws, stream)
    torch.cuda.synchronize()
    return accepted.cpu(), out.cpu(), logp.cpu(), int(ws.view(torch.int32)[0])


def _check(got, want, before=None):
    accepted, out, logp, bits = got
    wa, wo, wl, tol, wbits = want
    assert accepted.tolist() == wa and bits == wbits
    for i, (t, lp) in enumerate(zip(wo, wl)):
        if t is None:  # of no sequence
            assert int(out[i]) == (-7 if before is None else int(before[i])) and float(logp[i]) == 5.0
            continue
        assert int(out[i]) == t
        if lp is not None and np.isnan(lp):
            assert np.isnan(float(logp[i]))
        else:
            assert abs(float(logp[i]) - lp) <= tol[i]


OFFS = [[0, 1], [0, 5], [0, 1, 3, 6, 6, 14, 15], [0, 40, 41]]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 5, 17, 129, 1000, 5003])
@pytest.mark.parametrize("off", OFFS)
def test_drafts_with_their_distribution(dtype, vocab, off):
    z, zd, t, u, e = _inputs(off, vocab, dtype, vocab + len(off))
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy(), tau=0.8, tau_d=1.25)
    _check(_run(z, t, off, u, e, zd, temperature=0.8, draft_temperature=1.25), want)


@pytest.mark.parametrize("vocab", [3, 500, 9001])
@pytest.mark.parametrize("off", OFFS)
def test_drafts_looked_up(vocab, off):
    z, _, t, u, e = _inputs(off, vocab, "bf16", vocab)
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy())
    _check(_run(z, t, off, u, e), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab", [1, 9, 700, 20011])
@pytest.mark.parametrize("off", OFFS)
def test_greedy(dtype, vocab, off):
    z, _, t, _, _ = _inputs(off, vocab, dtype, vocab)
    best = torch.from_numpy(np.argmax(z.double().numpy(), 1))
    t = torch.where(torch.arange(len(t)) % 4 != 3, best, t)
    want = ref.verify(z.double().numpy(), t.numpy(), off, greedy=True, tau=0.5)
    _check(_run(z, t.int(), off, greedy=True, temperature=0.5), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_greedy_takes_the_lowest_of_equal_scores(dtype):
    off, vocab = [0, 3, 6, 8], 4099
    z = torch.randn(8, vocab, generator=torch.Generator().manual_seed(2)).clamp(max=2.0).to(DT[dtype])
    low = torch.finfo(DT[dtype]).min
    z[0, [17, 900, 4098]] = 3.0
    z[1, [4097, 4098]] = 3.0
    z[2, [0, 1]] = 3.0
    z[3] = low
    z[4] = low
    z[4, :700] = -INF
    z[5] = -INF
    z[5, 4000:] = low
    t = torch.tensor([17, 4097, 0, 0, 700, 0, 5, 0])
    want = ref.verify(z.double().numpy(), t.numpy(), off, greedy=True)
    got = _run(z, t, off, greedy=True)
    assert got[0].tolist() == want[0] == [2, 2, 0] and got[1].tolist() == want[1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,offset", [(1003, 0), (1008, 0), (1005, 3), (1024, 8)])
def test_rows_at_any_pitch(dtype, pitch, offset):
    off, vocab = [0, 4, 9], 1003
    z, zd, t, u, e = _inputs(off, vocab, dtype, 11)

    def put(x, pad, first):
        buf = torch.full((len(x) * (vocab + pad) + first,), NAN, dtype=x.dtype, device="cuda")
        v = buf[first:].view(len(x), vocab + pad)[:, :vocab]
        v.copy_(x)
        return v

    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    _check(_run(put(z, pitch - vocab, offset), t, off, u, put(e, 2, 1), put(zd, 1, 5)), want)


def test_saved_sums_of_the_draft():
    """With the draft's maxima and sums its rows are read only where a token is replaced; and they are
    what kfac_token_logprob saves."""
    off, vocab = [0, 6, 7, 12], 3001
    z, zd, t, u, e = _inputs(off, vocab, "bf16", 21)
    saved = torch.empty(len(t), 2, device="cuda")
    kfac.kfac_token_logprob(kfac.TokenLogprob(zd.cuda(), t.cuda(), torch.empty(len(t), device="cuda"), temperature=0.9, saved=saved))
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy(), tau_d=0.9)
    _check(_run(z, t, off, u, e, zd, saved, draft_temperature=0.9), want)


def test_last_rows_of_the_draft_are_not_read():
    off, vocab = [0, 4, 5, 9], 300
    z, zd, t, u, e = _inputs(off, vocab, "f32", 22)
    for r in (3, 4, 8):
        zd[r] = NAN
        t[r] = 1 << 40
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    got = _run(z, t, off, u, e, zd)
    _check(got, want)
    assert got[3] == 0


@pytest.mark.parametrize("int32", [False, True])
def test_tokens_in_place_and_rows_of_no_sequence(int32):
    off, vocab = [3, 7, 7, 12], 600
    z, zd, t, u, e = _inputs([0, 5, 10, 15], vocab, "f16", 23)
    t = t.int() if int32 else t
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    _check(_run(z, t.clone(), off, u, e, zd, inplace=True), want, before=t)


def test_offsets_outside_the_rows():
    off, vocab = [-4, 3, 8, 99], 50
    z, zd, t, u, e = _inputs([0, 4, 8, 12], vocab, "f32", 24)
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    _check(_run(z, t, off, u, e, zd), want)


def test_masked_scores():
    """-inf in either row: a token the policy forbids, one the draft could not have drawn, all but one masked,
    and rows of the type's lowest value."""
    off, vocab = [0, 2, 4, 6, 8, 10, 12], 70
    z, zd, t, u, e = _inputs(off, vocab, "bf16", 25)
    low = torch.finfo(torch.bfloat16).min
    z[0, t[0]] = -INF                       # forbidden: not accepted, and not drawn
    zd[2, t[2]] = -INF                      # q = 0: accepted
    z[4] = -INF
    z[4, 9] = 1.0                           # one token is left
    z[6] = low
    zd[6] = low                             # p = q: accepted
    z[8] = low
    z[8, 40:] = -INF
    zd[8] = -INF
    zd[8, :40] = 0.0
    t[8] = 7
    zd[10] = z[10]                          # p = q, u next to 1: accepted all the same
    u[10] = 1 - 2.0 ** -24
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    got = _run(z, t, off, u, e, zd)
    assert got[0].tolist()[0] == 0 and got[0].tolist()[1] == 1 and got[0].tolist()[3] == 1
    assert int(got[1][0]) != int(t[0])
    want[0][5], got[0][5] = 0, 0            # (p = q to the last bit lies on the border)
    for k in (10, 11):
        want[1][k] = got[1][k] = 0
        want[2][k] = got[2][k] = 0.0
    _check(got, want)


def test_nothing_left_to_draw_from():
    """p = q and u past 1: r is nothing, and the draw is from p."""
    off, vocab = [0, 2], 64
    z, _, t, u, e = _inputs(off, vocab, "f32", 26)
    u[0] = 2.0
    want = int(np.argmax(np.exp(ref.log_softmax(z[0].double().numpy(), 1.0)) / e[0].double().numpy()))
    got = _run(z, t, off, u, e, z)
    assert got[0].tolist() == [0] and got[1].tolist() == [want, -1]


def test_rows_without_a_distribution():
    off, vocab = [0, 3, 6, 9, 12, 15, 18], 40
    z, zd, t, u, e = _inputs(off, vocab, "f32", 27, near=0.0)
    u[:] = 0.0                              # accepted unless something is wrong
    z[1] = -INF
    z[3, 5] = NAN
    z[8, 7] = INF
    zd[9] = -INF
    zd[13, 2] = NAN
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    got = _run(z, t, off, u, e, zd)
    assert want[4] == kfac.ERRW_NONFINITE and want[0] == [1, 0, 2, 0, 1, 2]
    _check(got, want)
    z[1] = -INF
    _check(_run(z, t, off, greedy=True), ref.verify(z.double().numpy(), t.numpy(), off, greedy=True))


def test_tokens_outside_the_vocabulary():
    off, vocab = [0, 3, 6, 9], 40
    z, zd, t, u, e = _inputs(off, vocab, "f32", 28, near=0.0)
    u[:] = 0.0
    t[1], t[3], t[7] = -1, 40, 1 << 40
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    got = _run(z, t, off, u, e, zd)
    assert want[4] == kfac.ERRW_TARGET and want[0] == [1, 0, 1]
    _check(got, want)


def test_noise_that_is_not_positive():
    off, vocab = [0, 1, 2, 3], 50
    z, _, t, u, e = _inputs(off, vocab, "f32", 29)
    e[0, 13], e[1, [5, 30]], e[2, 20] = 0.0, torch.tensor([NAN, -1.0]), INF
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy())
    _check(_run(z, t, off, u, e), want)
    assert want[1][0] == 13


def test_equal_quotients_take_the_lowest():
    off, vocab = [0, 2], 3000
    z = torch.zeros(2, vocab)
    e = torch.ones(1, vocab)
    got = _run(z, torch.tensor([4, 0]), off, torch.tensor([2.0, 0.0]), e)
    assert got[1].tolist() == [0, -1]                            # every token but 4 has the same quotient
    got = _run(z, torch.tensor([0, 0]), off, torch.tensor([2.0, 0.0]), e)
    assert got[1].tolist() == [1, -1]


def test_many_sequences_and_long_ones():
    rng = np.random.default_rng(30)
    n = rng.integers(1, 4, 3000)
    off = [0] + np.cumsum(n).tolist()
    z, zd, t, u, e = _inputs(off, 24, "f32", 31)
    want = ref.verify(z.double().numpy(), t.numpy(), off, u.double().numpy(), e.double().numpy(), zd.double().numpy())
    _check(_run(z, t, off, u, e, zd), want)
    z, zd, t, u, e = _inputs([0, 700], 30, "f32", 32, near=0.0)  # accepted to the end
    u[:] = 0.5
    got = _run(z, t, [0, 700], u, e, z)
    assert got[0].tolist() == [699]
    _check(got, ref.verify(z.double().numpy(), t.numpy(), [0, 700], u.double().numpy(), e.double().numpy(), z.double().numpy()))


def test_repeated_captured_and_on_another_stream():
    off, vocab = [0, 5, 9], 40000
    z, zd, t, u, e = (x.cuda() for x in _inputs(off, vocab, "bf16", 33))
    first = _run(z, t, off, u, e, zd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = _run(z, t, off, u, e, zd, stream=side)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    acc, out, logp = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty_like(t), torch.empty(9, device="cuda")
    item = kfac.VerifyDraft(z, t, offsets, acc, out, logp, zd, uniform=u, noise=e)
    ws = torch.empty(kfac.kfac_verify_draft_workspace_size(item), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kfac.kfac_verify_draft(item, ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for a, b in [(first, second), (first, (acc.cpu(), out.cpu(), logp.cpu(), 0))]:
        assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_offsets_past_32_bits():
    """The last sequence of rows that lie past 2^32 bytes."""
    rows, vocab = 17000, 131072
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    off = [0, rows - 4, rows]
    sub = _inputs([0, 4], vocab, "bf16", 34)
    z[-4:] = sub[0].cuda()
    t = torch.zeros(rows, dtype=torch.int64)
    t[-4:] = sub[2]
    u = torch.ones(rows)
    u[-4:] = sub[3]
    e = torch.cat([torch.ones(1, vocab), sub[4]])
    got = _run(z, t, off, u, e)
    want = ref.verify(sub[0].double().numpy(), sub[2].numpy(), [0, 4], sub[3].double().numpy(), sub[4].double().numpy())
    assert got[0].tolist()[1] == want[0][0] and got[1][-4:].tolist() == want[1]
    assert got[0].tolist()[0] == 0 and int(got[1][0]) == 1


# ------------------------------------------------------------ many sequences: a cluster to a sequence

def _among_many(off, z, zd, t, u, e, seed=90):
    """The sequences with 400 more behind them, of one to three rows each."""
    rng = np.random.default_rng(seed)
    more = np.cumsum(rng.integers(1, 4, 400)).tolist()
    z2, zd2, t2, u2, e2 = _inputs([0] + more, z.shape[1], {v: k for k, v in DT.items()}[z.dtype], seed)
    cat = lambda a, b: None if a is None else torch.cat([a, b.to(a.dtype)])  # noqa: E731
    return off + [off[-1] + m for m in more], cat(z, z2), cat(zd, zd2), cat(t, t2), cat(u, u2), cat(e, e2)


def _np(x):
    return None if x is None else x.double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab", [1, 7, 130, 1003])
@pytest.mark.parametrize("how", ["rows", "saved", "none", "greedy"])
def test_many_sequences(dtype, vocab, how):
    off, z, zd, t, u, e = _among_many([0, 0, 5, 5, 6, 19], *_inputs([0, 4, 8, 12, 16, 19], vocab, dtype, 41))
    kw = dict(temperature=0.9)
    if how == "greedy":
        best = torch.from_numpy(np.argmax(_np(z), 1))
        t = torch.where(torch.arange(len(t)) % 5 != 3, best, t)
        want = ref.verify(_np(z), t.numpy(), off, greedy=True, tau=0.9)
        got = _run(z, t, off, greedy=True, **kw)
    else:
        saved = None
        if how == "saved":
            saved = torch.empty(len(t), 2, device="cuda")
            kfac.kfac_token_logprob(kfac.TokenLogprob(zd.cuda(), t.cuda(), torch.empty(len(t), device="cuda"), temperature=1.2, saved=saved))
        zd = None if how == "none" else zd
        want = ref.verify(_np(z), t.numpy(), off, _np(u), _np(e), _np(zd), tau=0.9, tau_d=1.2)
        got = _run(z, t, off, u, e, zd, saved, draft_temperature=1.2, **kw)
    _check(got, want)


@pytest.mark.parametrize("dtype,vocab,seqs", [("bf16", 17001, 170), ("f16", 40000, 90), ("f32", 33001, 60), ("bf16", 70003, 50)])
@pytest.mark.parametrize("how", ["rows", "none", "greedy"])
def test_many_sequences_over_large_vocabularies(dtype, vocab, seqs, how):
    rng = np.random.default_rng(5)
    off = [0] + np.cumsum(rng.integers(1, 4, seqs)).tolist()
    z, zd, t, u, e = _inputs(off, vocab, dtype, 51)
    if how == "greedy":
        best = torch.from_numpy(np.argmax(_np(z), 1))
        t = torch.where(torch.arange(len(t)) % 5 != 3, best, t)
        return _check(_run(z, t, off, greedy=True), ref.verify(_np(z), t.numpy(), off, greedy=True))
    zd = None if how == "none" else zd
    _check(_run(z, t, off, u, e, zd), ref.verify(_np(z), t.numpy(), off, _np(u), _np(e), _np(zd)))


def test_many_sequences_with_special_rows():
    """Masked, broken and equal rows, tokens outside the vocabulary, in place, rows of no sequence."""
    off = [2, 4, 6, 8, 10, 13, 16, 19, 22]
    z, zd, t, u, e = _inputs([0, 3, 6, 9, 12, 15, 18, 20, 22], 50, "f32", 61, near=0.0)
    u[:] = 0.0
    z[2, t[2]] = -INF                       # forbidden
    z[4] = -INF                             # nothing to draw from
    zd[6] = -INF
    z[8, 3] = NAN
    t[10], t[14] = -1, 50
    z[17] = INF
    e[6, :] = NAN
    u[19] = 2.0                             # p = q, not accepted: r is nothing
    zd[19] = z[19]
    off, z, zd, t, u, e = _among_many(off, z, zd, t, u, e)
    want = ref.verify(_np(z), t.numpy(), off, _np(u), _np(e), _np(zd))
    assert want[4] == kfac.ERRW_NONFINITE | kfac.ERRW_TARGET
    _check(_run(z, t, off, u, e, zd), want)
    _check(_run(z, t.clone(), off, u, e, zd, inplace=True), want, before=t)


def test_many_sequences_repeated_and_captured():
    off = np.arange(0, 1201, 3).tolist()
    z, zd, t, u, e = (x.cuda() for x in _inputs(off, 3000, "bf16", 71))
    first = _run(z, t, off, u, e, zd)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    acc, out, logp = torch.empty(400, dtype=torch.int32, device="cuda"), torch.empty_like(t), torch.empty(1200, device="cuda")
    item = kfac.VerifyDraft(z, t, offsets, acc, out, logp, zd, uniform=u, noise=e)
    ws = torch.empty(kfac.kfac_verify_draft_workspace_size(item), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kfac.kfac_verify_draft(item, ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first[:3], (acc.cpu(), out.cpu(), logp.cpu())))
