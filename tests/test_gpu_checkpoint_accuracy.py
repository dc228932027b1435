"""Long sums over rows keep their bits: what is added up in one tensor-core accumulator is short.

Where all terms have one sign every rounding goes the same way.  A step of 32 rows adds to an accumulator of
24 bits without rounding up and loses half a unit in its last place on average.  While a sum grows evenly to S
the unit is 0.67 to 0.75 times 2^-24 S on average, so N steps lose about 0.36 N 2^-24 S: 40 steps (1280 rows) 8.5e-7
of the sum, 256 steps 5.4e-6.  The sums of 40 steps are added with rounding to nearest, 16 of them at 20000 rows,
which is off by 16 / 2 * 2^-24 = 4.8e-7 at most.  The spread of a chunk's loss (0.29 units a step) is 1e-7 and is
averaged over the chunks.  2e-6 is above the sum of all (1.5e-6), and below what one long accumulator loses.
(Values of one size would not do: on e4m3's grid their sums fit 24 bits and are exact.)
"""
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
BOUND = 2e-6


def _kept(rows, cols, gen, one=False):
    """A checkpoint of positive values over some binades, and the values that it stands for."""
    x = torch.exp(torch.randn(rows, cols, device="cuda", generator=gen))
    c = kfac.Checkpoint.empty(rows, cols, one)
    item = kfac.CheckpointItem(x, c, one)
    kfac.kfac_checkpoint_store([item])
    kfac.kfac_checkpoint_load([item])
    return c, (torch.cat([x, torch.ones_like(x[:, :1])], 1) if one else x).double()


# (the last ones make as many tiles as run at once: none is split, and a tile's sums go over all rows)
@pytest.mark.parametrize("rows,dA,dG", [(1280, 300, 270), (5003, 300, 270), (20000, 4863, 1024)])
def test_weight_grad_of_one_sign(rows, dA, dG):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    a, av = _kept(rows, dA, gen, True)
    g, gv = _kept(rows, dG, gen)
    out = torch.empty(dG, dA + 1, device="cuda")
    kfac.kfac_weight_grad([kfac.WeightGrad(a, g, out)])
    want = gv.t() @ av
    assert float(((out.double() - want).abs() / want).max()) <= BOUND


@pytest.mark.parametrize("rows,d", [(1280, 300), (5003, 300), (20000, 2815)])
def test_factor_of_one_sign(rows, d):
    gen = torch.Generator(device="cuda").manual_seed(rows + 1)
    a, av = _kept(rows, d, gen, True)
    F = torch.zeros(d + 1, d + 1, device="cuda")
    kfac.kfac_factor_update([kfac.FactorSource(a, F, alpha=1.0, beta=0.0)])
    want = av.t() @ av
    assert float(((F.double() - want).abs() / want).triu().max()) <= BOUND
