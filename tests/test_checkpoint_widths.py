"""A factor that is too small for its checkpoint is refused before anything is enqueued."""
import pytest
import torch

from second_order_optimisation_gb300 import kfac, workloads
from second_order_optimisation_gb300.step import KfacStep


def _ck(rows, cols, one=False):
    return kfac.Checkpoint.empty(rows, cols, one, device="cpu")


@pytest.fixture(scope="module")
def step():
    return KfacStep([workloads.Layer("head", 100, 40, 1, 1, 0, 1, 1)], 8, device="cpu")


def test_step_takes_a_layer_s_widths(step):
    srcs = step.factor_sources([_ck(8, 100)], [_ck(8, 40)])
    assert [s.F.shape[0] for s in srcs] == [100, 40]


@pytest.mark.parametrize("x,g", [((8, 100, True), (8, 40)), ((8, 99), (8, 40)), ((8, 100), (8, 40, True)), ((8, 100), (8, 39)),
                                 ((8, 100), (8, 64))])
def test_step_refuses_other_widths(step, x, g):
    """Also those that the padded pitch of a factor's rows would hold."""
    with pytest.raises(ValueError):
        step.factor_sources([_ck(*x)], [_ck(*g)])
    with pytest.raises(ValueError):
        step.run([_ck(*x)], [_ck(*g)], [torch.zeros(40, 100, dtype=torch.bfloat16)], stream=0)


@pytest.mark.parametrize("F,packed", [(torch.zeros(40, 64)[:, :40], False), (torch.zeros(41, 64)[:, :40], False),
                                      (torch.zeros(40, 41), False), (torch.zeros(40 * 41 // 2), True), (torch.zeros(860), True)])
def test_binding_refuses_a_factor_that_is_too_small(F, packed):
    src = kfac.FactorSource(_ck(8, 40, True), F, packed=packed)
    for call in (kfac.kfac_factor_update_workspace_size, kfac.kfac_factor_update):
        with pytest.raises(kfac.KfacError) as e:
            call([src])
        assert e.value.status == kfac.KFAC_ERR_INVALID


@pytest.mark.parametrize("F,packed", [(torch.zeros(41, 64)[:, :41], False), (torch.zeros(50, 50), False), (torch.zeros(861), True)])
def test_binding_takes_a_factor_that_is_large_enough(F, packed):
    import __graft_entry__
    __graft_entry__.build()
    assert kfac.kfac_factor_update_workspace_size([kfac.FactorSource(_ck(8, 40, True), F, packed=packed)]) > 0
