"""The verification of drafted tokens without a GPU: that the rules give the policy's
distribution, and what the entry point refuses."""
import ctypes

import numpy as np
import pytest
import torch

from tests import verify_ref as ref
from second_order_optimisation_gb300 import kfac

INVALID, UNSUPPORTED = kfac.KFAC_ERR_INVALID, kfac.KFAC_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kfac.load()


@pytest.mark.parametrize("lookup", [False, True])
def test_first_token_is_distributed_as_the_policy(lookup):
    """Over 20000 drafts the first token's counts are a draw from p: a chi-square with 5
    degrees of freedom is above 30 once in 60000 times (the seed is fixed)."""
    rng = np.random.default_rng(3)
    vocab, n = 6, 20000
    z, zd = rng.normal(size=vocab) * 1.5, rng.normal(size=vocab)
    p = np.exp(ref.log_softmax(z, 1.0))
    q = np.exp(ref.log_softmax(zd, 1.0))
    counts = np.zeros(vocab)
    for _ in range(n):
        x = 2 if lookup else rng.choice(vocab, p=q)
        _, out, _, _, _ = ref.verify(np.stack([z, z]), [x, 0], [0, 2], rng.random(2), rng.exponential(size=(1, vocab)),
                                     None if lookup else np.stack([zd, zd]))
        counts[out[0]] += 1
    assert ((counts - n * p) ** 2 / (n * p)).sum() < 30


def _vd(**kw):
    d = dict(dtype=kfac.KFAC_BF16, logits=0x1000, ld=100, rows=6, vocab=100, tokens=0x2000, token_i32=0, temperature=1.0,
             seq_offsets=0x3000, seqs=2, draft=0x4000, ld_draft=100, draft_saved=None, draft_temperature=1.0, uniform=0x5000,
             noise=0x6000, ld_noise=100, greedy=0, accepted=0x7000, out_tokens=0x8000, logp=None)
    d.update(kw)
    return kfac.VerifyDesc(**d)


BAD = [(dict(logits=None), INVALID), (dict(tokens=None), INVALID), (dict(seq_offsets=None), INVALID), (dict(accepted=None), INVALID),
       (dict(out_tokens=None), INVALID), (dict(uniform=None), INVALID), (dict(noise=None), INVALID), (dict(rows=-1), INVALID),
       (dict(seqs=0), INVALID), (dict(vocab=0), INVALID), (dict(ld=99), INVALID), (dict(ld_draft=99), INVALID), (dict(ld_noise=99), INVALID),
       (dict(draft=None, draft_saved=0x9000), INVALID), (dict(draft_saved=0x9004), INVALID), (dict(dtype=3), INVALID),
       (dict(logits=0x1001), INVALID), (dict(draft=0x4001), INVALID), (dict(temperature=0.0), INVALID), (dict(temperature=NAN), INVALID),
       (dict(draft_temperature=INF), INVALID), (dict(draft_temperature=-1.0), INVALID), (dict(vocab=(1 << 24) + 1, ld=1 << 25, ld_draft=1 << 25, ld_noise=1 << 25), UNSUPPORTED),
       (dict(rows=1 << 31), UNSUPPORTED), (dict(seqs=(1 << 20) + 1), UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", BAD)
def test_verify_refuses(lib, bad, status):
    d = ctypes.byref(_vd(**bad))
    assert lib.kfac_verify_draft_workspace_size(d) == 0
    assert lib.kfac_verify_draft(d, 0x100000, 1 << 40, None) == status


def test_verify_workspace_and_pointers(lib):
    d = ctypes.byref(_vd())
    need = lib.kfac_verify_draft_workspace_size(d)
    assert need > 0
    assert lib.kfac_verify_draft(None, None, 0, None) == INVALID
    for ws, n in [(None, 0), (0x100001, need), (0x100000, need - 1)]:
        assert lib.kfac_verify_draft(d, ws, n, None) == kfac.KFAC_ERR_WORKSPACE
    assert lib.kfac_verify_draft(d, 0x100000, need, None) == INVALID  # not device memory
    # what a greedy call does not read it does not ask for
    g = ctypes.byref(_vd(greedy=1, draft=None, uniform=None, noise=None, draft_temperature=0.0))
    assert lib.kfac_verify_draft_workspace_size(g) > 0


def test_binding_refuses():
    z, t, off = torch.zeros(6, 10), torch.zeros(6, dtype=torch.int64), torch.tensor([0, 3, 6], dtype=torch.int32)
    acc, u, e = torch.zeros(2, dtype=torch.int32), torch.zeros(6), torch.ones(2, 10)
    good = dict(logits=z, tokens=t, seq_offsets=off, accepted=acc, out_tokens=t.clone(), uniform=u, noise=e)
    for bad, err in [(dict(out_tokens=t.int()), TypeError), (dict(accepted=t[:2]), TypeError), (dict(noise=e[:1]), ValueError),
                     (dict(noise=e.double()), TypeError), (dict(uniform=u[:5]), ValueError), (dict(draft=z.half()), TypeError),
                     (dict(draft=z[:5]), TypeError), (dict(seq_offsets=off.long()), TypeError), (dict(tokens=t[:5]), ValueError),
                     (dict(logits=z.double()), TypeError), (dict(draft=z, draft_saved=torch.zeros(6)), ValueError)]:
        with pytest.raises(err):
            kfac.kfac_verify_draft(kfac.VerifyDraft(**{**good, **bad}))
