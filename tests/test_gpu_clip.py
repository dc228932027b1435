"""kfac_clip_norm on the GPU against its definition in 64 bits.

Bounds (e = 2^-24): a thread adds at most 64 products one after the other in
fp32, everything else is added in fp64, so the sum of products is off by at most
64 e sum |x y|, the norm by half of that over the norm, plus its own rounding;
a scaled value by the scale's error, its product and its rounding."""
import math

import numpy as np
import pytest
import torch

from second_order_optimisation_gb300 import kfac

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")
E = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: E}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-37}


def word(ws):
    torch.cuda.synchronize()
    return int(ws[:4].view(torch.int32).item())


def nums(t):
    return t.detach().double().cpu().numpy()


def strided(shape, dtype, ld=None, shift=0, gen=None, scale=1.0, fill=NAN):
    """A random matrix (or vector) inside a buffer of `fill`."""
    n = math.prod(shape)
    if len(shape) == 2 and ld:
        buf = torch.full((shape[0] * ld + shift + 8,), fill, dtype=dtype, device=DEV)
        v = buf[shift:shift + shape[0] * ld].view(shape[0], ld)[:, :shape[1]]
    else:
        buf = torch.full((n + shift + 8,), fill, dtype=dtype, device=DEV)
        v = buf[shift:shift + n].view(shape)
    v.copy_(torch.randn(shape, generator=gen) * scale)
    return v


def check(tensors, max_norm, eta=0.0, use_list=False, err=0):
    """Runs the call and compares norm, scale, out and w with the definition."""
    before = [(nums(t.x), nums(t.y) if t.y is not None else None, nums(t.w) if t.w is not None else None) for t in tensors]
    norm, scale = torch.full((1,), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)
    ws = kfac.kfac_clip_norm(kfac.ClipList(tensors) if use_list else tensors, max_norm, norm, scale, eta)
    assert word(ws) == err
    total = sum((x * (y if y is not None else x)).sum() for x, y, _ in before)
    mass = sum(np.abs(x * (y if y is not None else x)).sum() for x, y, _ in before)
    want = math.sqrt(max(0.0, total))
    tol = (64 * E * mass / (2 * want) if want else math.sqrt(64 * E * mass)) + E * want + 1e-45
    assert abs(float(norm) - want) <= tol, (float(norm), want, tol)
    sc = min(1.0, max_norm / want) if want else 1.0
    rel = tol / want if want else 0.0
    assert abs(float(scale) - sc) <= (rel + 2 * E) * sc
    for t, (x, _, w) in zip(tensors, before):
        if t.out is not None:
            got = nums(t.out)
            v = sc * x
            assert (np.abs(got - v) <= (rel + 4 * E + ROUND[t.out.dtype]) * np.abs(v) + TINY[t.out.dtype]).all()
        if w is not None:
            v = w - eta * sc * x
            assert (np.abs(nums(t.w) - v) <= (rel + 8 * E) * np.abs(eta * sc * x) + E * np.abs(v) + 1e-37).all()
    return norm, scale


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("metric", [False, True])
def test_types_and_shapes(dtype, out, metric):
    g = torch.Generator().manual_seed(4)
    ts = []
    for shape, ld, shift in [((1,), None, 0), ((7,), None, 3), ((3, 5), None, 1), ((33, 65), 72, 0), ((33, 65), 67, 1),
                             ((200, 130), None, 0), ((1, 9000), None, 5), ((9000, 1), 3, 0), ((40, 1024), 1032, 4),
                             ((30000,), None, 0), ((5, 4, 3), None, 0), ((), None, 0), ((0,), None, 0), ((0, 4), None, 0)]:
        x = strided(shape, TYPES[dtype], ld, shift, g)
        y = None
        if metric:
            y = strided(shape, TYPES[dtype], None if shift else ld, 0, g, 0.1)
            y.add_(x)
        o = strided(shape, TYPES[out], ld and ld + 8, shift and 2, g)
        ts.append(kfac.ClipTensor(x, o, y))
    check(ts, 3.0)
    check(ts, 1e9)
    check(ts, INF, use_list=True)


@pytest.mark.parametrize("ydt", ["bf16", "f16"])
def test_metric_of_fp32_steps_and_16_bit_gradients(ydt):
    """The natural gradient step (fp32) and the gradient that it comes from."""
    g = torch.Generator().manual_seed(11)
    ts = []
    for shape, ldx, ldy in [((64, 147), 192, None), ((64, 147), None, None), ((256, 576), None, None), ((1000, 2049), 2112, 2112),
                            ((5,), None, None), ((400, 1000), None, 1003)]:
        x = strided(shape, torch.float32, ldx, 0, g)
        y = strided(shape, TYPES[ydt], ldy, 1 if len(shape) == 1 else 0, g, 0.1)
        y.add_(x.to(y.dtype))
        ts.append(kfac.ClipTensor(x, None, y, strided(shape, torch.float32, ldx and ldx + 1, 0, g)))
    check(ts, 0.5, eta=0.25)
    check(ts[:2] + ts[4:5], 0.5, eta=0.25)


def test_norm_alone_and_no_tensors():
    g = torch.Generator().manual_seed(5)
    check([kfac.ClipTensor(strided((50, 60), torch.float32, gen=g))], 2.0)
    norm, scale = check([], 2.0)
    assert float(norm) == 0.0 and float(scale) == 1.0
    norm, scale = check([kfac.ClipTensor(torch.zeros(100000, device=DEV), torch.empty(100000, device=DEV))], 2.0)
    assert float(norm) == 0.0 and float(scale) == 1.0


@pytest.mark.parametrize("dtype", list(TYPES))
def test_weight_step(dtype):
    g = torch.Generator().manual_seed(6)
    ts = []
    for shape, ld in [((64, 130), 192), ((64, 130), None), ((130,), None), ((1000, 513), None), ((3, 20000), 20011)]:
        x = strided(shape, TYPES[dtype], ld, 0, g)
        y = strided(shape, TYPES[dtype], ld, 0, g, 0.1)
        y.add_(x)
        ts.append(kfac.ClipTensor(x, None, y, strided(shape, torch.float32, ld and ld + 3, 1, g)))
    check(ts, 0.5, eta=0.25)
    check(ts, INF, eta=0.25)
    check([kfac.ClipTensor(t.x, torch.empty_like(t.x), None, t.w) for t in ts], 1.0, eta=-2.0)


def test_in_place():
    g = torch.Generator().manual_seed(7)
    xs = [strided(s, torch.bfloat16, ld, 0, g) for s, ld in (((300, 77), 80), ((5000,), None), ((64, 64), None))]
    ts = [kfac.ClipTensor(x, x) for x in xs]
    same = [x.clone() for x in xs]
    check(ts, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(xs, same))       # nothing to clip: not rewritten
    check(ts, 4.0)
    total = math.sqrt(sum(float((x.double() ** 2).sum()) for x in xs))
    assert abs(total - 4.0) < 4.0 * 2.0 ** -9


def test_more_tensors_than_one_launch_takes():
    g = torch.Generator().manual_seed(8)
    ts = [kfac.ClipTensor(strided((1 + k % 37, 1 + k % 11), torch.float32, gen=g), torch.empty(1 + k % 37, 1 + k % 11, device=DEV))
          for k in range(1100)]
    check(ts, 1.5)


def test_many_allocations_and_memory_elsewhere():
    """Tensors in more allocations than a call remembers, in no order; host memory among them is refused."""
    g = torch.Generator().manual_seed(12)
    room = [torch.empty(2_700_000, device=DEV) for _ in range(290)]
    ts = []
    for k in torch.randperm(290, generator=g).tolist():
        x = room[k][k % 5:k % 5 + 90 + k]
        x.copy_(torch.randn(90 + k, generator=g))
        ts.append(kfac.ClipTensor(x, room[(k * 7) % 290][5000:5090 + k]))
    check(ts, 2.0)
    for at in (0, 150, 289):
        bad = list(ts)
        bad[at] = kfac.ClipTensor(torch.zeros(50), torch.zeros(50))
        norm = torch.full((1,), 7.0, device=DEV)
        with pytest.raises(kfac.KfacError):
            kfac.kfac_clip_norm(bad, 2.0, norm)
        assert float(norm) == 7.0


@pytest.mark.parametrize("scale", [1e-30, 1e-24, 1e-10, 1e10, 1e25, 1e36])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("metric", [False, True])
def test_squares_outside_fp32(scale, dtype, metric):
    """Values whose squares overflow or vanish in fp32."""
    g = torch.Generator().manual_seed(9)
    ts = []
    for n in (1000, 20000):
        x = strided((n,), TYPES[dtype], gen=g, scale=scale)
        y = (x.float() * 0.5).to(TYPES[dtype]) if metric else None
        ts.append(kfac.ClipTensor(x, torch.empty_like(x), y))
    check(ts, float(np.float32(scale * 20)))
    ts.append(kfac.ClipTensor(strided((3000,), TYPES[dtype], gen=g), torch.empty(3000, dtype=TYPES[dtype], device=DEV)))
    if not metric:
        check(ts, float(np.float32(max(scale, 1.0) * 20)))


def test_metric_that_is_not_positive():
    x = torch.ones(500, device=DEV)
    out, norm, scale = torch.empty_like(x), torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    ws = kfac.kfac_clip_norm([kfac.ClipTensor(x, out, -x)], 1.0, norm, scale)
    assert word(ws) == 0 and float(norm) == 0.0 and float(scale) == 1.0 and torch.equal(out, x)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_nonfinite_values_propagate_and_are_reported(bad):
    x, z = torch.randn(20000, device=DEV), torch.randn(300, device=DEV)
    x[12345] = bad
    ox, oz, norm, scale = torch.empty_like(x), torch.empty_like(z), torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    ws = kfac.kfac_clip_norm([kfac.ClipTensor(z, oz), kfac.ClipTensor(x, ox)], 1.0, norm, scale)
    assert word(ws) == kfac.ERRW_NONFINITE
    if math.isnan(bad):
        assert math.isnan(float(norm)) and math.isnan(float(scale)) and bool(torch.isnan(oz).all())
    else:
        assert math.isinf(float(norm)) and float(scale) == 0.0
        assert bool((oz == 0).all()) and math.isnan(float(ox[12345]))
    x[12345] = 0
    assert word(kfac.kfac_clip_norm([kfac.ClipTensor(z, oz), kfac.ClipTensor(x, ox)], 1.0)) == 0


def test_repeatable_on_dirty_workspaces_streams_and_graphs():
    g = torch.Generator().manual_seed(10)
    for sizes in ((100, 3000), (70000, 123456, 9), (3_000_001, 20_000_000)):
        xs = [strided((n,), torch.bfloat16, gen=g) for n in sizes]
        first = None
        ts = [kfac.ClipTensor(x, torch.empty_like(x)) for x in xs]
        c = kfac.ClipList(ts)
        ws = torch.full((kfac.kfac_clip_norm_workspace_size(c) + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        norm = torch.empty(1, device=DEV)
        side = torch.cuda.Stream()
        for k in range(4):
            side.wait_stream(torch.cuda.current_stream())
            kfac.kfac_clip_norm(c, 3.0, norm, workspace=None if k == 1 else ws, stream=side if k == 2 else None)
            torch.cuda.synchronize()
            got = [norm.clone()] + [t.out.clone() for t in ts]
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(got, first))
            [t.out.fill_(5) for t in ts]
            torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kfac.kfac_clip_norm(c, 3.0, norm, workspace=ws)
        for _ in range(2):
            [t.out.fill_(5) for t in ts]
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip([norm] + [t.out for t in ts], first))
        assert bool((ws[-256:] == 0xA5).all())
