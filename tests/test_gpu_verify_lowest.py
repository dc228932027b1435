"""Greedy verification of rows whose largest score is the type's lowest finite value, behind masked scores
that fill whole batches of a thread's loads."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF = float("inf")
BATCH = {"bf16": 4096, "f16": 4096, "f32": 2048}  # elements that a CTA's threads load at a time


def _greedy(z, tokens, off):
    accepted = torch.full((len(off) - 1,), -5, dtype=torch.int32, device="cuda")
    out, logp = torch.full_like(tokens, -7), torch.empty(len(tokens), device="cuda")
    ws = kfac.kfac_verify_draft(kfac.VerifyDraft(z, tokens, torch.tensor(off, dtype=torch.int32, device="cuda"), accepted, out, logp,
                                                 greedy=True))
    torch.cuda.synchronize()
    return accepted.tolist(), out.tolist(), logp.cpu(), int(ws.view(torch.int32)[0])


@pytest.mark.parametrize("dtype", list(DT))
def test_lowest_scores_up_to_the_edge(dtype):
    """The row's last elements are no whole group of 16 bytes: the lowest index is not theirs."""
    n, low = BATCH[dtype], torch.finfo(DT[dtype]).min
    vocab = 2 * n - 16 // DT[dtype].itemsize * 11 + 1
    z = torch.full((4, (vocab + 7) // 8 * 8), -INF, dtype=DT[dtype], device="cuda")[:, :vocab]
    first = [n, n + 5, vocab - 1, n + 77]
    for r, i in enumerate(first):
        z[r, i:] = low
    accepted, out, logp, bits = _greedy(z, torch.tensor([n, 0, vocab - 1, 0], device="cuda"), [0, 2, 4])
    assert accepted == [1, 1] and out == first and bits == 0
    want = -torch.tensor([vocab - i for i in first], dtype=torch.float64).log()
    assert ((logp - want).abs() <= 2.0 ** -24 * (8 * want.abs() + 128)).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab,offset", [(7, 0), (1, 1), (1, 0), (0, 1), (0, 0)])
def test_lowest_scores_behind_masked_batches(dtype, vocab, offset):
    """Nothing is left of a row but lowest scores: at its end, one of them, between masked ones, from a batch's
    first or last element on, in rows that begin and end anywhere."""
    n, low = BATCH[dtype], torch.finfo(DT[dtype]).min
    vocab += 3 * n
    first = [0, 1, n - 1, n, n + 1, 2 * n - 1, 2 * n, 2 * n + 9, vocab - 1, 3 * n - 1, n + 300, 17]
    rows = len(first)
    z = torch.full((rows * vocab + 8,), -INF, dtype=DT[dtype], device="cuda")[offset:offset + rows * vocab].view(rows, vocab)
    for r, i in enumerate(first):
        z[r, i:] = low
        if r % 3 == 1:
            z[r, i + 1:] = -INF                 # one token is left
        if r % 3 == 2:
            z[r, i + 2:vocab - 1] = -INF
    tokens = torch.tensor([i if r % 4 != 3 else 3 for r, i in enumerate(first)], device="cuda")
    accepted, out, logp, bits = _greedy(z, tokens, [0, 4, 8, 12])
    assert accepted == [3, 3, 3] and out == first and bits == 0
    want = -torch.isfinite(z).sum(1).double().log().cpu()
    assert ((logp - want).abs() <= 2.0 ** -24 * (8 * want.abs() + 128)).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_lowest_scores_of_many_long_rows(dtype):
    """As many rows as leave each to one CTA, 131072 scores in many batches."""
    rows, vocab, low = 1300, 131072, torch.finfo(DT[dtype]).min
    z = torch.full((rows, vocab), -INF, dtype=DT[dtype], device="cuda")
    z[:, vocab // 2:] = low
    z[3, vocab // 2:] = -INF
    z[3, -1] = low
    z[7, 5000] = low
    z[11] = -INF                                # nothing left: no distribution
    best = torch.full((rows,), vocab // 2, device="cuda")
    best[3], best[7] = vocab - 1, 5000
    accepted, out, logp, bits = _greedy(z, best.clone(), list(range(0, rows + 1, 2)))
    want = best.clone()
    want[11] = -1
    n = [1] * (rows // 2)
    assert accepted == n and out == want.tolist() and bits == kfac.ERRW_NONFINITE
    assert torch.isnan(logp[11]) and float(logp[3]) == 0.0
