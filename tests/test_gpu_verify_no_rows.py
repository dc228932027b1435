"""Verification of sequences that are all empty: nothing is there to be read."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [1, 1000, 131072])
@pytest.mark.parametrize("seqs", [1, 700])
@pytest.mark.parametrize("how", ["none", "noise", "draft", "saved", "greedy"])
def test_no_rows(vocab, seqs, how):
    z = torch.empty(0, vocab, dtype=torch.bfloat16, device="cuda")
    tokens = torch.empty(0, dtype=torch.int64, device="cuda")
    off = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    accepted = torch.full((seqs,), -5, dtype=torch.int32, device="cuda")
    logp = torch.empty(0, device="cuda")
    kw = {}
    if how in ("noise", "draft", "saved"):
        kw = dict(uniform=torch.empty(0, device="cuda"), noise=torch.ones(seqs, vocab, device="cuda"))
    if how in ("draft", "saved"):
        kw["draft"] = z.clone()
    if how == "saved":
        kw["draft_saved"] = torch.empty(0, 2, device="cuda")
    item = kfac.VerifyDraft(z, tokens, off, accepted, tokens.clone(), logp, greedy=how == "greedy", **kw)
    ws = torch.full((kfac.kfac_verify_draft_workspace_size(item),), 255, dtype=torch.uint8, device="cuda")
    kfac.kfac_verify_draft(item, ws)
    torch.cuda.synchronize()
    assert accepted.tolist() == [0] * seqs and int(ws.view(torch.int32)[0]) == 0


def test_offsets_past_no_rows():
    """Offsets are read as the nearest that there is: 0."""
    z = torch.empty(0, 50, dtype=torch.float32, device="cuda")
    tokens = torch.empty(0, dtype=torch.int32, device="cuda")
    off = torch.tensor([-3, 4, 9, 2], dtype=torch.int32, device="cuda")
    accepted = torch.full((3,), -5, dtype=torch.int32, device="cuda")
    kfac.kfac_verify_draft(kfac.VerifyDraft(z, tokens, off, accepted, tokens.clone()))
    assert accepted.tolist() == [0, 0, 0]
