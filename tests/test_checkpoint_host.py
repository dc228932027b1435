"""Checkpoints and their uses without a GPU: the format, what the entry points refuse, and
the reference's gradient against differences."""
import ctypes

import numpy as np
import pytest
import torch

from tests import checkpoint_ref as ref
from second_order_optimisation_gb300 import kfac

INVALID, UNSUPPORTED, WORKSPACE = kfac.KFAC_ERR_INVALID, kfac.KFAC_ERR_UNSUPPORTED, kfac.KFAC_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return kfac.load()


# ------------------------------------------------------------ the reference

def test_reference_elements_are_e4m3():
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    v = ref.e4m3_values()
    assert np.array_equal(np.isnan(b), np.isnan(v)) and np.array_equal(b[~np.isnan(b)], v[~np.isnan(v)])


def test_reference_rounds_as_e4m3_does():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(size=(64, 5)) * np.exp(rng.normal(size=(64, 5)) * 4), np.full((1, 5), 300.0)])
    x = np.concatenate([x, ref.e4m3_values()[:120].reshape(-1, 5)[:19] + 2.0 ** -10, -np.ones((3, 5)) * 17.0])  # ties too
    q, ex = ref.store(x)
    y = torch.from_numpy(x * np.exp2(-np.repeat(ex, 32, 0)[:len(x)].astype(float))).float().to(torch.float8_e4m3fn)
    assert np.array_equal(y.view(torch.uint8).numpy() & 127, q & 127)
    err = np.abs(ref.values(q, ex) - x)
    assert (err <= np.maximum(2.0 ** -4 * np.abs(x), np.exp2(np.repeat(ex, 32, 0)[:len(x)] - 10.0))).all()


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0 * (1 + 2.0 ** -20), 1), (224.0, -1), (1.0, -8), (0.0, -127),
                                   (2.0 ** -140, -127), (448.0 * 2.0 ** -127, -127), (3.4e38, 120)])
def test_exponent(top, e):
    assert ref.exponent(top) == e


def test_reference_weight_gradient_is_the_difference():
    rng = np.random.default_rng(2)
    a, g, w = rng.normal(size=(7, 4)), rng.normal(size=(7, 3)), rng.normal(size=(3, 4))
    d, _ = ref.weight_grad(g, a, 0.5)
    num = np.zeros_like(w)
    for i in np.ndindex(*w.shape):  # of 0.5 sum g . (a w^T), quadratic terms none
        lo, hi = w.copy(), w.copy()
        lo[i] -= 1e-3
        hi[i] += 1e-3
        num[i] = 0.5 * ((g * (a @ hi.T)).sum() - (g * (a @ lo.T)).sum()) / 2e-3
    assert np.abs(d - num).max() < 1e-9


def test_places_of_the_exponents():
    rows, width = 300, 260
    at = {int(ref.place(rows, t, c)) for t in range(10) for c in range(width)}
    assert len(at) == 10 * width and max(at) < kfac.checkpoint_scale_bytes(rows, width)
    # a column's four blocks lie side by side, tiles of 128 rows after one another
    assert [int(ref.place(rows, t, 0)) for t in range(6)] == [0, 1, 2, 3, 512, 513]
    assert int(ref.place(rows, 0, 128)) == 3 * 512 and int(ref.place(rows, 0, 33)) == 16 + 4


# ------------------------------------------------------------ refusals

def test_scale_bytes(lib):
    for rows, width in [(1, 1), (128, 128), (129, 128), (5000, 2049), (0, 5)]:
        assert lib.kfac_checkpoint_scale_bytes(rows, width) == kfac.checkpoint_scale_bytes(rows, width)
    assert lib.kfac_checkpoint_scale_bytes(-1, 5) == 0 and lib.kfac_checkpoint_scale_bytes(5, 0) == 0


def _ck(**kw):
    d = dict(dtype=kfac.KFAC_BF16, x=0x1000, ld=100, rows=40, cols=100, append_one=0, q=0x2000, ldq=112, scales=0x3000)
    d.update(kw)
    return (kfac.CheckpointDesc * 1)(kfac.CheckpointDesc(**d))


CK_BAD = [(dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scales=None), INVALID), (dict(rows=-1), INVALID),
          (dict(cols=0), INVALID), (dict(ld=99), INVALID), (dict(ldq=96), INVALID), (dict(dtype=3), INVALID),
          (dict(dtype=9), INVALID), (dict(x=0x1001), INVALID), (dict(append_one=1, cols=112, ld=112), INVALID),
          (dict(ldq=104), UNSUPPORTED), (dict(q=0x2008), UNSUPPORTED), (dict(scales=0x3008), UNSUPPORTED),
          (dict(cols=1048577, ld=1048577, ldq=1048592), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
          (dict(), INVALID)]  # (the last: pointers that are not device memory)


@pytest.mark.parametrize("bad,status", CK_BAD)
def test_store_and_load_refuse(lib, bad, status):
    assert lib.kfac_checkpoint_store(_ck(**bad), 1, None) == status
    assert lib.kfac_checkpoint_load(_ck(**bad), 1, None) == status


def test_store_and_load_of_nothing(lib):
    for f in (lib.kfac_checkpoint_store, lib.kfac_checkpoint_load):
        assert f(None, 0, None) == kfac.KFAC_OK
        assert f(None, 1, None) == INVALID and f(None, -1, None) == INVALID
        assert f(_ck(rows=0, x=None, q=None, scales=None), 1, None) == kfac.KFAC_OK


def _wg(**kw):
    d = dict(q_a=0x1000, ldq_a=112, scales_a=0x2000, q_g=0x3000, ldq_g=64, scales_g=0x4000, rows=40, dA=100, dG=50,
             out=0x5000, ld=100, out_dtype=kfac.KFAC_F32, alpha=1.0, beta=0.0)
    d.update(kw)
    return (kfac.WeightGradDesc * 1)(kfac.WeightGradDesc(**d))


WG_BAD = [(dict(q_a=None), INVALID), (dict(scales_a=None), INVALID), (dict(q_g=None), INVALID), (dict(scales_g=None), INVALID),
          (dict(out=None), INVALID), (dict(rows=-1), INVALID), (dict(dA=0), INVALID), (dict(dG=0), INVALID), (dict(ld=99), INVALID),
          (dict(ldq_a=96), INVALID), (dict(ldq_g=48), INVALID), (dict(out_dtype=3), INVALID), (dict(out=0x5002), INVALID),
          (dict(alpha=float("nan")), INVALID), (dict(beta=float("inf")), INVALID), (dict(ldq_a=104), UNSUPPORTED),
          (dict(q_g=0x3008), UNSUPPORTED), (dict(scales_a=0x2004), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", WG_BAD)
def test_weight_grad_refuses(lib, bad, status):
    assert lib.kfac_weight_grad_workspace_size(_wg(**bad), 1) == 0
    assert lib.kfac_weight_grad(_wg(**bad), 1, 0x100000, 1 << 40, None) == status


def test_weight_grad_workspace_and_pointers(lib):
    need = lib.kfac_weight_grad_workspace_size(_wg(), 1)
    assert need >= 4
    assert lib.kfac_weight_grad(_wg(), 1, None, 0, None) == WORKSPACE
    assert lib.kfac_weight_grad(_wg(), 1, 0x100001, need, None) == WORKSPACE
    assert lib.kfac_weight_grad(_wg(), 1, 0x100000, need - 1, None) == WORKSPACE
    assert lib.kfac_weight_grad(_wg(), 1, 0x100000, need, None) == INVALID  # not device memory
    assert lib.kfac_weight_grad(None, 0, None, 0, None) == kfac.KFAC_OK
    assert lib.kfac_weight_grad(None, 1, None, 0, None) == INVALID


def _fd(**kw):
    d = dict(dtype=kfac.KFAC_E4M3, x=0x1000, n=40, h=1, w=1, c=100, kh=1, kw=1, stride_h=1, stride_w=1, pad_h=0, pad_w=0,
             append_one=0, F=0x2000, ldf=100, alpha=1.0, beta=0.0, layout=0, scales=0x3000, ldx=112)
    d.update(kw)
    return (kfac.FactorDesc * 1)(kfac.FactorDesc(**d))


@pytest.mark.parametrize("bad,status", [(dict(scales=None), INVALID), (dict(ldx=96), INVALID), (dict(ldf=99), INVALID),
                                        (dict(ldx=0), INVALID), (dict(ldx=104), UNSUPPORTED), (dict(x=0x1008), UNSUPPORTED),
                                        (dict(scales=0x3004), UNSUPPORTED), (dict(append_one=1, ldf=101), UNSUPPORTED),
                                        (dict(c=65537, ldf=65537, ldx=65552), UNSUPPORTED), (dict(h=2), UNSUPPORTED), (dict(kh=3, pad_h=1), UNSUPPORTED)])
def test_factor_update_refuses_checkpoints(lib, bad, status):
    arr = _fd(**bad)
    assert lib.kfac_factor_update_workspace_size(arr, 1) == 0
    assert lib.kfac_factor_update(arr, 1, 0x100000, 1 << 40, None) == status


def test_binding_refuses():
    c = kfac.Checkpoint.empty(40, 100, device="cpu")
    x = torch.zeros(40, 100)
    bad = [kfac.CheckpointItem(x[:39], c), kfac.CheckpointItem(x, c, append_one=True), kfac.CheckpointItem(x.t(), c),
           kfac.CheckpointItem(x, kfac.Checkpoint(c.q[:, :96], c.scales, 40, 100)),
           kfac.CheckpointItem(x, kfac.Checkpoint(c.q, c.scales[:100], 40, 100))]
    for item in bad:
        with pytest.raises(ValueError):
            kfac.kfac_checkpoint_store([item])
    with pytest.raises(TypeError):
        kfac.kfac_checkpoint_load([kfac.CheckpointItem(x.double(), c)])
    with pytest.raises(TypeError):
        kfac.kfac_checkpoint_load([kfac.CheckpointItem(x, kfac.Checkpoint(c.q.int(), c.scales, 40, 100))])
    g = kfac.Checkpoint.empty(40, 10, device="cpu")
    for item in [kfac.WeightGrad(c, g, torch.zeros(100, 10)), kfac.WeightGrad(c, g, torch.zeros(100, 10).t()),
                 kfac.WeightGrad(c, kfac.Checkpoint.empty(39, 10, device="cpu"), torch.zeros(10, 100))]:
        with pytest.raises(ValueError):
            kfac.kfac_weight_grad([item])
    with pytest.raises(TypeError):
        kfac.kfac_weight_grad([kfac.WeightGrad(c, g, torch.zeros(10, 100, dtype=torch.float64))])
    with pytest.raises(kfac.KfacError):  # host memory
        kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, c)], stream=0)
