"""Tiles of a product that come in several pieces, from pairs of CTAs that do not wait for one another."""
import pytest
import torch

from tests import checkpoint_ref as ref
from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _kept(rows, cols, gen):
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    c = kfac.Checkpoint.empty(rows, cols)
    item = kfac.CheckpointItem(x, c)
    kfac.kfac_checkpoint_store([item])
    kfac.kfac_checkpoint_load([item])
    return c, x.double()


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("shapes", [[(9000, 200, 130)], [(5200, 1300, 1100)], [(12000, 257, 30), (8000, 300, 520), (70, 90, 1000)],
                                    [(3600, 513, 300)] * 60])
def test_pieces(shapes, out):
    """Both CTAs' and all warps' parts are added up once each, in one order, whatever the workspace held; more
    products than a launch takes have counters of their own."""
    gen = torch.Generator(device="cuda").manual_seed(len(shapes))
    made, items, want = {}, [], []
    for i, (rows, dA, dG) in enumerate(shapes):
        if (rows, dA, dG) not in made:
            made[rows, dA, dG] = (*_kept(rows, dA, gen), *_kept(rows, dG, gen))
        a, av, g, gv = made[rows, dA, dG]
        beta = 0.5 if i % 2 else 0.0
        o = torch.randn(dG, dA, device="cuda", generator=gen).to(DT[out])
        p, size = 0.25 * (gv.t() @ av), 0.25 * (gv.abs().t() @ av.abs())
        w = p + beta * o.double()
        want.append((o, w, ref.SUM * (size + beta * o.double().abs()) + ref.ROUND[out] * w.abs() + 2.0 ** -25))
        items.append((a, g, beta))
    need = kfac.kfac_weight_grad_workspace_size([kfac.WeightGrad(a, g, o, 0.25, b) for (a, g, b), (o, _, _) in zip(items, want)])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    runs = []
    for fill in (0, 255, 1):
        outs = [o.clone() for o, _, _ in want]
        ws.fill_(fill)
        kfac.kfac_weight_grad([kfac.WeightGrad(a, g, o, 0.25, b) for (a, g, b), o in zip(items, outs)], ws)
        assert int(ws.view(torch.int32)[0]) == 0
        runs.append(outs)
    for (_, w, tol), o, o2, o3 in zip(want, *runs):
        assert bool(((o.double() - w).abs() <= tol).all()) and torch.equal(o, o2) and torch.equal(o, o3)


@pytest.mark.parametrize("packed", [False, True])
def test_pieces_of_factors_replayed(packed):
    gen = torch.Generator(device="cuda").manual_seed(9)
    kept = [_kept(rows, d, gen) for rows, d in ((7000, 300), (9000, 700), (500, 40))]
    Fs = [torch.zeros(c.width, c.width, device="cuda") for c, _ in kept]
    Fs = [kfac.pack_upper(F) if packed else F for F in Fs]
    srcs = [kfac.FactorSource(c, F, alpha=0.5, beta=0.0, packed=packed) for (c, _), F in zip(kept, Fs)]
    ws = torch.empty(kfac.kfac_factor_update_workspace_size(srcs), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kfac.kfac_factor_update(srcs, ws)
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert int(ws.view(torch.int32)[0]) == 0
    for (c, v), F in zip(kept, Fs):
        got = (kfac.unpack_upper(F, c.width) if packed else F).double()
        want, size = 0.5 * (v.t() @ v), 0.5 * (v.abs().t() @ v.abs())
        assert bool(((got - want).abs() <= ref.SUM * size + ref.E * want.abs())[torch.ones_like(want, dtype=torch.bool).triu()].all())
