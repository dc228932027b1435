"""Checkpoints, their weight gradients and factors on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

from tests import checkpoint_ref as ref
from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


def _x(rows, cols, dtype, seed=0, spread=2.0):
    """Values whose columns and rows differ in size, rounded to dtype, and as fp64."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) * np.exp(spread * rng.normal(size=cols)) * np.exp(rng.normal(size=(rows, 1)))
    t = torch.from_numpy(x).float().to(DT[dtype])
    return t, t.double().numpy()


def _pitched(t, pitch, offset=0, fill=7.0):
    """t on the GPU as a view with a row pitch and a base offset (elements), and what it lies in."""
    rows, cols = t.shape
    buf = torch.full((rows * pitch + offset + 16,), fill, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    v.copy_(t)
    return v, buf


def _kept(x, one=False, device="cuda"):
    """A checkpoint of fp64 values made by the reference, and its values."""
    q, ex = ref.store(x, one)
    c = kfac.Checkpoint.empty(len(x), x.shape[1], one, device)
    c.q.fill_(255)  # (past the width nothing may be read)
    c.q[:, :q.shape[1]] = torch.from_numpy(q).to(device)
    c.scales.copy_(torch.from_numpy(ref.scale_bytes(ex, len(x))))
    return c, ref.values(q, ex)


def _err(ws):
    return int(ws.view(torch.int32)[0])


# ------------------------------------------------------------ store and load

SHAPES = [(1, 1), (1, 300), (31, 7), (32, 16), (33, 17), (127, 129), (128, 128), (129, 64), (260, 257), (500, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("one", [False, True])
def test_store_and_load(dtype, rows, cols, one):
    t, x = _x(rows, cols, dtype, rows + cols)
    q, ex = ref.store(x, one)
    c = kfac.Checkpoint.empty(rows, cols, one)
    c.q.fill_(0xA5)
    c.scales.fill_(0xA5)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(t.cuda(), c, one)])
    got = c.q.cpu().numpy()
    assert np.array_equal(got[:, :cols + one], q) and (got[:, cols + one:] == 0xA5).all()
    assert np.array_equal(c.scales.cpu().numpy(), ref.scale_bytes(ex, rows))
    out = torch.full((rows, cols), 9.0, dtype=DT[dtype], device="cuda")
    kfac.kfac_checkpoint_load([kfac.CheckpointItem(out, c, one)])
    want = torch.from_numpy(ref.values(q, ex)[:, :cols]).to(DT[dtype])
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,offset", [(75, 0), (80, 0), (80, 1), (77, 3), (96, 8)])
def test_store_and_load_at_any_pitch(dtype, pitch, offset):
    t, x = _x(70, 73, dtype, 5)
    v, buf = _pitched(t, pitch, offset)
    c = kfac.Checkpoint.empty(70, 73)
    c.q = torch.full((71, 96), 0x33, dtype=torch.uint8, device="cuda")  # a wider pitch, a row more
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(v, c)])
    q, ex = ref.store(x)
    assert np.array_equal(c.q.cpu().numpy()[:70, :73], q)
    assert (c.q[70] == 0x33).all() and (c.q[:, 73:] == 0x33).all()
    w, wide = _pitched(torch.zeros(70, 73, dtype=DT[dtype]), pitch, offset)
    kfac.kfac_checkpoint_load([kfac.CheckpointItem(w, c)])
    assert torch.equal(w.cpu(), torch.from_numpy(ref.values(q, ex)).to(DT[dtype]))
    w.fill_(7.0)
    assert (wide == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 5, 130])
def test_every_width_at_every_alignment(dtype, rows):
    """Rows that begin and end anywhere: what is beside them stays as it was."""
    step = 8 if dtype == "bf16" else 4
    for cols in [*range(1, 2 * step + 3), *range(126, 128 + step + 2), 250, 257]:
        x, v = _x(rows, cols, dtype, cols)
        q, ex = ref.store(v, True)
        want = torch.from_numpy(ref.values(q, ex)[:, :cols]).float().to(DT[dtype]).cuda()
        for offset in range(step):
            xd, buf = _pitched(x, cols + offset % 3, offset)
            c = kfac.Checkpoint.empty(rows, cols, True)
            c.q.fill_(7)
            kfac.kfac_checkpoint_store([kfac.CheckpointItem(xd, c, True)])
            assert np.array_equal(c.q[:, :cols + 1].cpu().numpy(), q) and bool((c.q[:, cols + 1:] == 7).all()), (cols, offset)
            assert np.array_equal(c.scales.cpu().numpy(), ref.scale_bytes(ex, rows))
            c.q[:, cols + 1:] = 255
            buf.fill_(3.0)
            kfac.kfac_checkpoint_load([kfac.CheckpointItem(xd, c, True)])
            assert torch.equal(xd, want), (cols, offset)
            assert int((buf == 3.0).sum()) == buf.numel() - rows * cols + int((want == 3.0).sum()), (cols, offset)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_store_of_special_values(dtype):
    big = torch.finfo(DT[dtype]).max
    tiny = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}[dtype]
    t = torch.randn(96, 24, generator=torch.Generator().manual_seed(4)).to(DT[dtype])
    t[5, 0], t[6, 1], t[7, 2] = INF, -INF, NAN
    t[:32, 3] = INF
    t[:32, 4] = NAN
    t[:, 5] = 0.0
    t[3, 6], t[40, 6] = big, -big
    t[:, 7] = tiny * torch.arange(96)
    t[:, 8] = 448.0
    t[9, 9], t[10, 9] = big, INF
    t[0, 10] = -0.0
    x = t.double().numpy()
    q, ex = ref.store(x)
    c = kfac.Checkpoint.empty(96, 24)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(t.cuda(), c)])
    got = c.q.cpu().numpy()[:, :24]
    bad = ~np.isfinite(x)
    assert np.array_equal(got[~bad], q[~bad]) and ((got[bad] & 127) == 127).all()
    assert np.array_equal(c.scales.cpu().numpy(), ref.scale_bytes(ex, 96))
    out = torch.empty(96, 24, dtype=DT[dtype], device="cuda")
    kfac.kfac_checkpoint_load([kfac.CheckpointItem(out, c)])
    want = torch.from_numpy(ref.values(q, ex)).to(DT[dtype])
    assert torch.equal(out.cpu().isnan(), torch.from_numpy(bad)) and torch.equal(out.cpu()[~torch.from_numpy(bad)], want[~torch.from_numpy(bad)])


def test_load_rounds_to_its_type():
    t, x = _x(64, 20, "f32", 6, spread=8.0)  # past fp16's range on both sides
    q, ex = ref.store(x)
    c = kfac.Checkpoint.empty(64, 20)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(t.cuda(), c)])
    for dt in DT.values():
        out = torch.empty(64, 20, dtype=dt, device="cuda")
        kfac.kfac_checkpoint_load([kfac.CheckpointItem(out, c)])
        assert torch.equal(out.cpu(), torch.from_numpy(ref.values(q, ex)).float().to(dt))


def test_many_matrices_in_one_call():
    items, want = [], []
    for i in range(70):  # more than one launch takes, types mixed, one without rows
        dtype = ["bf16", "f16", "f32"][i % 3]
        t, x = _x(0 if i == 33 else 1 + 7 * i, 1 + (i * 37) % 150, dtype, i)
        one = i % 2 == 1
        items.append(kfac.CheckpointItem(t.cuda(), kfac.Checkpoint.empty(*t.shape, one), one))
        want.append(ref.store(x, one) if len(x) else None)
    before = kfac.launch_count()
    kfac.kfac_checkpoint_store(items)
    assert kfac.launch_count() == before + 2
    for it, w in zip(items, want):
        if w is not None:
            assert np.array_equal(it.checkpoint.q.cpu().numpy()[:, :it.checkpoint.width], w[0])
            assert np.array_equal(it.checkpoint.scales.cpu().numpy(), ref.scale_bytes(w[1], len(w[0])))
    kfac.kfac_checkpoint_store([])
    kfac.kfac_checkpoint_load([])


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 bytes in 16 bits: its last rows."""
    rows, cols = 66000, 32800
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    t, v = _x(80, cols, "bf16", 8)
    x[-80:] = t.cuda()
    c = kfac.Checkpoint.empty(rows, cols)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, c)])
    first = (rows - 80) % 32  # rows of the tail's first block before the tail
    q, _ = ref.store(np.concatenate([np.zeros((first, 400)), v[:, -400:]]))
    assert np.array_equal(c.q[-80:, -400:].cpu().numpy() if c.q.shape[1] == cols else c.q[-80:, cols - 400:cols].cpu().numpy(), q[first:])
    x.fill_(1.0)
    kfac.kfac_checkpoint_load([kfac.CheckpointItem(x, c)])
    assert int(torch.count_nonzero(x[:-80])) == 0
    assert (x[-80:].float().cpu().numpy() - v).__abs__().max() <= 2.0 ** -4 * np.abs(v).max()


# ------------------------------------------------------------ weight gradient

WG = [(1, 1, 1), (5, 3, 2), (32, 65, 32), (33, 16, 130), (128, 128, 128), (129, 257, 127), (1000, 300, 260), (2500, 129, 250),
      (4100, 70, 33)]


@pytest.mark.parametrize("rows,dA,dG", WG)
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_weight_grad(rows, dA, dG, out):
    a, av = _kept(_x(rows, dA, "f32", 1, 1.0)[1])
    g, gv = _kept(_x(rows, dG, "f32", 2, 1.0)[1])
    alpha = 1.0 / rows
    o = torch.full((dG, dA + 5), 3.0, dtype=DT[out], device="cuda")
    ws = kfac.kfac_weight_grad([kfac.WeightGrad(a, g, o[:, :dA], alpha)])
    want, tol = ref.weight_grad(gv, av, np.float32(alpha).astype(float))
    got = o.double().cpu().numpy()
    assert (np.abs(got[:, :dA] - want) <= tol + ref.ROUND[out] * np.abs(want) + 2.0 ** -25).all()
    assert (got[:, dA:] == 3.0).all() and _err(ws) == 0


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_weight_grad_accumulates(out):
    rows = 300
    a, av = _kept(_x(rows, 140, "f32", 1, 1.0)[1])
    g, gv = _kept(_x(rows, 131, "f32", 2, 1.0)[1])
    old = torch.randn(131, 140).to(DT[out])
    o = old.cuda()
    kfac.kfac_weight_grad([kfac.WeightGrad(a, g, o, 0.25, 0.5)])
    want, tol = ref.weight_grad(gv, av, 0.25, 0.5, old.double().numpy())
    assert (np.abs(o.double().cpu().numpy() - want) <= tol + ref.ROUND[out] * np.abs(want)).all()


def test_weight_grad_of_long_sums_of_one_sign():
    """Where every term is positive a sum that loses a bit at each step would show."""
    rows = 20000
    a, av = _kept(np.abs(_x(rows, 140, "f32", 1, 0.5)[1]))
    g, gv = _kept(np.abs(_x(rows, 20, "f32", 2, 0.5)[1]))
    o = torch.empty(20, 140, device="cuda")
    kfac.kfac_weight_grad([kfac.WeightGrad(a, g, o)])
    want, tol = ref.weight_grad(gv, av, 1.0)
    assert (np.abs(o.double().cpu().numpy() - want) <= tol + ref.E * np.abs(want)).all()


def test_weight_grad_batch_and_rows_of_zero():
    """More problems than one launch takes; without rows beta out remains."""
    items, want = [], []
    for i in range(60):
        rows, dA, dG = (0 if i == 7 else 1 + 31 * i), 1 + (i * 53) % 200, 1 + (i * 29) % 140
        if rows:
            a, av = _kept(_x(rows, dA, "f32", i, 1.0)[1])
            g, gv = _kept(_x(rows, dG, "f32", i + 100, 1.0)[1])
        else:
            a, g = kfac.Checkpoint.empty(0, dA), kfac.Checkpoint.empty(0, dG)
            av, gv = np.zeros((0, dA)), np.zeros((0, dG))
        beta = 0.5 if i % 3 == 1 else 0.0
        old = torch.randn(dG, dA)
        items.append(kfac.WeightGrad(a, g, old.cuda(), 0.125, beta))
        want.append(ref.weight_grad(gv, av, 0.125, beta, old.double().numpy()))
    ws = kfac.kfac_weight_grad(items)
    for it, (w, tol) in zip(items, want):
        assert (np.abs(it.out.double().cpu().numpy() - w) <= tol + ref.E * np.abs(w)).all()
    assert _err(ws) == 0


def test_weight_grad_is_repeatable_and_captured():
    a, _ = _kept(_x(1500, 200, "f32", 1, 1.0)[1])
    g, _ = _kept(_x(1500, 150, "f32", 2, 1.0)[1])
    outs = [torch.empty(150, 200, device="cuda") for _ in range(3)]
    kfac.kfac_weight_grad([kfac.WeightGrad(a, g, outs[0])])
    kfac.kfac_weight_grad([kfac.WeightGrad(a, g, outs[1])])
    item = kfac.WeightGrad(a, g, outs[2])
    ws = torch.empty(kfac.kfac_weight_grad_workspace_size([item]), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kfac.kfac_weight_grad([item], ws)
    for _ in range(3):
        outs[2].zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("what", ["nan", "overflow"])
def test_weight_grad_reports_values_that_are_not_finite(what):
    x = _x(64, 40, "f32", 1, 1.0)[1]
    if what == "nan":
        x[3, 5] = NAN
    else:
        x[:, 5] = 1e30
    a, _ = _kept(x)
    gx = np.ones((64, 9))
    if what == "overflow":
        gx[:, 4] = 1e20
    g, _ = _kept(gx)
    o = torch.empty(9, 40, device="cuda")
    ws = kfac.kfac_weight_grad([kfac.WeightGrad(a, g, o)])
    bad = ~torch.isfinite(o.cpu())
    assert _err(ws) == kfac.ERRW_NONFINITE
    want = torch.zeros(9, 40, dtype=torch.bool)
    want[(slice(None) if what == "nan" else 4), 5] = True
    assert torch.equal(bad, want)


# ------------------------------------------------------------ factors

@pytest.mark.parametrize("rows,cols,one", [(1, 1, False), (32, 64, True), (100, 128, True), (260, 129, False), (3000, 300, True)])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("beta", [0.0, 0.95])
def test_factor_update_from_a_checkpoint(rows, cols, one, packed, beta):
    c, v = _kept(_x(rows, cols, "f32", 3, 1.0)[1], one)
    d = cols + one
    old = torch.randn(d, d)
    F = old.cuda()
    src = kfac.pack_upper(F) if packed else torch.cat([F, torch.full((d, 3), 5.0, device="cuda")], 1)
    alpha = (1 - beta) / rows
    ws = kfac.kfac_factor_update([kfac.FactorSource(c, src if packed else src[:, :d], alpha=alpha, beta=beta, packed=packed)])
    got = (kfac.unpack_upper(src, d) if packed else src[:, :d]).double().cpu().numpy()
    al, be = float(np.float32(alpha)), float(np.float32(beta))
    want, tol = ref.weight_grad(v, v, al, be, old.double().numpy())
    up = np.triu(np.ones((d, d), bool))
    assert (np.abs(got - want) <= tol + ref.E * np.abs(want))[up].all()
    if not packed:
        assert np.array_equal(got[~up], old.double().numpy()[~up]) and (src[:, d:] == 5.0).all()
    assert _err(ws) == 0


def test_factor_update_of_checkpoints_beside_other_sources():
    """One call with every kind of source gives each its own result, bit by bit."""
    t, x = _x(200, 96, "bf16", 9)
    c, _ = _kept(x)
    srcs = [t.cuda(), c, t.float().cuda(), t.half().cuda(), c]
    F = [torch.eye(96, device="cuda") for _ in srcs]
    alone = [torch.eye(96, device="cuda") for _ in srcs]
    kfac.kfac_factor_update([kfac.FactorSource(s, f, alpha=0.01, beta=0.9) for s, f in zip(srcs, F)])
    for s, f in zip(srcs, alone):
        kfac.kfac_factor_update([kfac.FactorSource(s, f, alpha=0.01, beta=0.9)])
    for a, b in zip(F, alone):
        assert torch.equal(a, b)
    assert torch.equal(F[1], F[4])


def test_host_memory_is_refused():
    x = torch.zeros(40, 100, device="cuda")
    c = kfac.Checkpoint.empty(40, 100)
    host = kfac.Checkpoint.empty(40, 100, device="cpu")
    for it in [kfac.CheckpointItem(x.cpu(), c), kfac.CheckpointItem(x, host), kfac.CheckpointItem(x, kfac.Checkpoint(c.q, host.scales, 40, 100))]:
        with pytest.raises(kfac.KfacError):
            kfac.kfac_checkpoint_store([it])
    with pytest.raises(kfac.KfacError):
        kfac.kfac_weight_grad([kfac.WeightGrad(c, host, torch.zeros(100, 100, device="cuda"))])
    with pytest.raises(kfac.KfacError):
        kfac.kfac_factor_update([kfac.FactorSource(kfac.Checkpoint(c.q, host.scales, 40, 100), torch.eye(100, device="cuda"))],
                                workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("rows,dA,dG", [(3100, 900, 1500), (7000, 300, 200), (6200, 2500, 2300)])
def test_weight_grad_of_tiles_in_pieces(rows, dA, dG):
    """Few tiles of many stages, and a last round that would leave most pairs idle: tiles in several pieces."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, dA, device="cuda", generator=g)
    y = torch.randn(rows, dG, device="cuda", generator=g)
    a, b = kfac.Checkpoint.empty(rows, dA), kfac.Checkpoint.empty(rows, dG)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, a), kfac.CheckpointItem(y, b)])
    kfac.kfac_checkpoint_load([kfac.CheckpointItem(x, a), kfac.CheckpointItem(y, b)])
    old = torch.randn(dG, dA, device="cuda", generator=g)
    outs = [old.clone() for _ in range(2)]
    for o in outs:
        ws = kfac.kfac_weight_grad([kfac.WeightGrad(a, b, o, 0.5, 0.25)])
    want = 0.25 * old.double() + 0.5 * (y.double().t() @ x.double())
    size = 0.25 * old.double().abs() + 0.5 * (y.double().abs().t() @ x.double().abs())
    assert bool(((outs[0].double() - want).abs() <= ref.SUM * size + ref.E * want.abs()).all())
    assert torch.equal(outs[0], outs[1]) and _err(ws) == 0


# ------------------------------------------------------------ more tiles than run at once

def _pair(rows, dA, dG, seed, pitch=0):
    """Checkpoints of random values and these values, on the GPU; nothing behind a row may be read."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for d in (dA, dG):
        x = torch.randn(rows, d, device="cuda", generator=g) * torch.exp(torch.randn(d, device="cuda", generator=g))
        c = kfac.Checkpoint.empty(rows, d)
        if pitch:
            c.q = torch.empty(rows, c.q.shape[1] + pitch, dtype=torch.uint8, device="cuda")
        c.q.fill_(127)  # NaN
        kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, c)])
        kfac.kfac_checkpoint_load([kfac.CheckpointItem(x, c)])
        out += [c, x.double()]
    return out


@pytest.mark.parametrize("rows", [1, 300, 1500])
@pytest.mark.parametrize("dA,dG,out", [(257, 19400, "f32"), (259, 19300, "bf16"), (260, 19201, "f16")])
def test_weight_grad_of_a_few_columns_more_than_tiles(rows, dA, dG, out):
    """76 tiles of 256 x 256, and narrow ones for a few columns more."""
    a, av, g, gv = _pair(rows, dA, dG, rows, pitch=16 * (rows % 2))
    old = torch.randn(dG, dA + 3, device="cuda").to(DT[out])
    outs = [old.clone() for _ in range(3)]
    for o, beta in zip(outs, (0.0, 0.5, 0.5)):
        ws = kfac.kfac_weight_grad([kfac.WeightGrad(a, g, o[:, :dA], 0.25, beta)])
        assert _err(ws) == 0
    p, size = 0.25 * (gv.t() @ av), 0.25 * (gv.abs().t() @ av.abs())
    for o, beta in zip(outs, (0.0, 0.5)):
        want, most = p + beta * old[:, :dA].double(), size + beta * old[:, :dA].double().abs()
        assert bool(((o[:, :dA].double() - want).abs() <= ref.SUM * most + ref.ROUND[out] * want.abs() + 2.0 ** -25).all())
        assert torch.equal(o[:, dA:], old[:, dA:])
    assert torch.equal(outs[1], outs[2])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("rows,cols", [(70, 2816), (2100, 2819)])
def test_factor_of_a_few_columns_more_than_tiles(rows, cols, packed):
    """66 tiles on and above the diagonal, and 78 with the columns that are more."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    d = cols + 1
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    c = kfac.Checkpoint.empty(rows, cols, True)
    kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, c, True)])
    kfac.kfac_checkpoint_load([kfac.CheckpointItem(x, c, True)])
    v = torch.cat([x, torch.ones(rows, 1, device="cuda")], 1).double()
    old = torch.randn(d, d, device="cuda", generator=gen)
    F = [kfac.pack_upper(old) if packed else old.clone() for _ in range(2)]
    for f in F:
        ws = kfac.kfac_factor_update([kfac.FactorSource(c, f, alpha=0.25, beta=0.5, packed=packed)])
        assert _err(ws) == 0
    assert torch.equal(F[0], F[1])
    got = (kfac.unpack_upper(F[0], d) if packed else F[0]).double()
    want = 0.25 * (v.t() @ v) + 0.5 * old.double()
    size = 0.25 * (v.abs().t() @ v.abs()) + 0.5 * old.double().abs()
    up = torch.triu(torch.ones(d, d, dtype=torch.bool, device="cuda"))
    assert bool(((got - want).abs() <= ref.SUM * size + ref.E * want.abs())[up].all())
    if not packed:
        assert torch.equal(F[0][~up], old[~up])


def test_weight_grad_of_more_problems_and_tiles_than_a_launch_takes():
    a, av, g, gv = _pair(200, 514, 500, 3)
    outs = [torch.empty(500, 514, device="cuda") for _ in range(51)]
    ws = kfac.kfac_weight_grad([kfac.WeightGrad(a, g, o, 0.5) for o in outs])
    want, size = 0.5 * (gv.t() @ av), 0.5 * (gv.abs().t() @ av.abs())
    for o in outs:
        assert bool(((o.double() - want).abs() <= ref.SUM * size + ref.E * want.abs()).all())
    assert _err(ws) == 0


@pytest.mark.parametrize("a,g", [(1e-36, 1e36), (1e30, 1e-30), (1e-20, 1e-18), (1e30, 1e30)])
def test_weight_grad_of_extreme_exponents(a, g):
    """Exponents whose product leaves fp32 on the way, or in the end."""
    ca, av, cg, gv = _pair(160, 257, 300, 5)
    for c, v, s in ((ca, av, a), (cg, gv, g)):
        x = v.float() * s
        kfac.kfac_checkpoint_store([kfac.CheckpointItem(x, c)])
        kfac.kfac_checkpoint_load([kfac.CheckpointItem(x, c)])
        v.copy_(x.double())
    o = torch.empty(300, 257, device="cuda")
    ws = kfac.kfac_weight_grad([kfac.WeightGrad(ca, cg, o)])
    if a * g > 1e40:
        assert not bool(torch.isfinite(o).any()) and _err(ws) == kfac.ERRW_NONFINITE
        return
    want, size = gv.t() @ av, gv.abs().t() @ av.abs()
    # (products of subnormal sums lose what is below 2^-149, one a block of exponents)
    assert bool(((o.double() - want).abs() <= ref.SUM * size + ref.E * want.abs() + 160 / 32 * 2.0 ** -149).all())
    assert _err(ws) == 0


def test_an_output_layer_of_a_wide_vocabulary():
    """More columns than a factor may have: kept, restored, and multiplied."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows, vocab, dA = 70, 131075, 65
    y = torch.randn(rows, vocab, device="cuda", generator=gen)
    x = torch.randn(rows, dA, device="cuda", generator=gen)
    a, g = kfac.Checkpoint.empty(rows, dA), kfac.Checkpoint.empty(rows, vocab)
    items = [kfac.CheckpointItem(x, a), kfac.CheckpointItem(y, g)]
    before = y.clone()
    kfac.kfac_checkpoint_store(items)
    kfac.kfac_checkpoint_load(items)
    assert bool(((y - before).abs() <= 2.0 ** -4 * before.abs() + 2.0 ** -10 * before.abs().max() / 224).all())
    out = torch.empty(vocab, dA, device="cuda")
    ws = kfac.kfac_weight_grad([kfac.WeightGrad(a, g, out)])
    want, size = y.double().t() @ x.double(), y.double().abs().t() @ x.double().abs()
    assert bool(((out.double() - want).abs() <= ref.SUM * size + ref.E * want.abs()).all()) and _err(ws) == 0
    with pytest.raises(kfac.KfacError):
        kfac.kfac_factor_update([kfac.FactorSource(g, torch.empty(16, device="cuda"), alpha=1.0, beta=0.0, packed=True)])
