"""Drafts from the policy itself: p = q to the last bit, and every token is accepted with u next to 1."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab,seqs", [(70, 6), (1003, 40), (50001, 3), (131072, 1)])
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_equal_rows_are_accepted(dtype, vocab, seqs, tau):
    k = 5
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    z = (3 * torch.randn(seqs * k, vocab, device="cuda", generator=gen)).to(DT[dtype])
    tokens = torch.randint(vocab, (seqs * k,), device="cuda", generator=gen)
    off = torch.arange(0, seqs * k + 1, k, dtype=torch.int32, device="cuda")
    u = torch.full((seqs * k,), 1 - 2.0 ** -24, device="cuda")
    noise = torch.ones(seqs, vocab, device="cuda")
    accepted, out = torch.empty(seqs, dtype=torch.int32, device="cuda"), torch.empty_like(tokens)
    kfac.kfac_verify_draft(kfac.VerifyDraft(z, tokens, off, accepted, out, draft=z.clone(), uniform=u, noise=noise,
                                            temperature=tau, draft_temperature=tau))
    assert accepted.tolist() == [k - 1] * seqs
    drafted = torch.arange(seqs * k, device="cuda") % k < k - 1
    assert torch.equal(out[drafted], tokens[drafted])
    # the last token is drawn from p: with equal noise its most likely one, the lowest of equals
    p = z.double()[~drafted]
    best = torch.where(p == p.amax(1, keepdim=True), torch.arange(vocab, device="cuda"), vocab).amin(1)
    assert torch.equal(out[~drafted], best)
