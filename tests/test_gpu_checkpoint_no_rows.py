"""Weight gradients of layers that saw no row: nothing is loaded, and beta out is what remains."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dA,dG", [(1, 1), (65, 32), (300, 257), (2500, 2000)])
@pytest.mark.parametrize("beta", [0.0, 0.5])
@pytest.mark.parametrize("count", [1, 3, 50])
def test_no_rows(dA, dG, beta, count):
    a, g = kfac.Checkpoint.empty(0, dA), kfac.Checkpoint.empty(0, dG)
    old = torch.randn(dG, dA, device="cuda", generator=torch.Generator(device="cuda").manual_seed(dA))
    items = [kfac.WeightGrad(a, g, old.to(t, copy=True), 3.0, beta) for t in [torch.float32, torch.bfloat16, torch.float16] * (count // 3 + 1)][:count]
    want = [beta * it.out.double() for it in items]
    if beta == 0:
        items[0].out.fill_(float("nan"))  # it is not read
        want[0].zero_()
    ws = torch.full((kfac.kfac_weight_grad_workspace_size(items),), 255, dtype=torch.uint8, device="cuda")
    kfac.kfac_weight_grad(items, ws)
    torch.cuda.synchronize()
    assert int(ws.view(torch.int32)[0]) == 0
    for it, w in zip(items, want):  # (half of a value is exact, but for the least ones of 16 bits)
        assert bool(((it.out.double() - w).abs() <= 2.0 ** -25).all())


def test_store_and_load_of_no_rows_beside_others():
    x, e = torch.ones(3, 40, device="cuda"), torch.empty(0, 7, device="cuda", dtype=torch.float16)
    c, n = kfac.Checkpoint.empty(3, 40), kfac.Checkpoint.empty(0, 7)
    items = [kfac.CheckpointItem(e, n), kfac.CheckpointItem(x, c), kfac.CheckpointItem(e, n)]
    kfac.kfac_checkpoint_store(items)
    x.zero_()
    kfac.kfac_checkpoint_load(items)
    assert bool((x == 1).all())
