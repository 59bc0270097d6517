"""GPU checks of the orthogonalized updates against 64-bit references: within
1.5 times the error that the kernels' roundings make on the CPU."""
import numpy as np
import pytest

from tests import sublayer_reference as ref
from tests.test_gpu_checkpoint import device, dtype_of
from tests.test_gpu_layer_norm import held, nan
from tests.test_gpu_training_alignment import Inside
from tests.test_orthogonalize_host import ABC, matrix

pytestmark = pytest.mark.gpu

EPS = 1e-7


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def check(out, x, steps=5, abc=ABC, eps=EPS, dtype="f32"):
    value, tolerance = ref.orthogonalize(x, steps, *abc, eps, f32=dtype == "f32")
    got = out.double().cpu().numpy()
    assert got.shape == value.shape
    assert np.linalg.norm(got - value) <= tolerance, (np.linalg.norm(got - value), tolerance, np.linalg.norm(value))


def run(tide, xs, dtype, **kw):
    outs = [nan(x.shape, "bf16") for x in xs]
    tide.orthogonalize([device(x, dtype) for x in xs], outs, **kw)
    return outs


# one tile, short pieces of k, tiles on and below the diagonal, both orientations; G split along k
SIZES = [(1, 1), (1, 7), (7, 1), (5, 9), (9, 5), (16, 16), (33, 70), (70, 33), (128, 128), (129, 257), (257, 129), (300, 300),
         (520, 1000), (1000, 520), (130, 5000), (5000, 130), (640, 2300)]


@pytest.mark.parametrize("kind", ["noise", "strong"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(tide, rows, cols, kind):
    dtype = "f32" if (rows + cols) % 2 else "bf16"
    x = held(matrix(np.random.default_rng(rows + cols), rows, cols, kind), dtype)
    check(run(tide, [x], dtype)[0], x, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("count,rows,cols", [(2, 9, 20), (40, 300, 200), (64, 300, 410), (150, 20, 30), (131, 33, 17),
                                             (12, 520, 700), (3, 1100, 1300), (3, 1300, 1100)])
def test_many(tide, count, rows, cols, dtype):
    """Pieces of the list, and more tiles than workgroups."""
    rng = np.random.default_rng(count)
    xs = [held(matrix(rng, rows, cols, "strong" if i % 3 == 0 else "noise"), dtype) for i in range(count)]
    outs = run(tide, xs, dtype)
    for i in {0, 1, count // 2, count - 2, count - 1}:
        check(outs[i], xs[i], dtype=dtype)
    # a matrix's result does not depend on its place; of the sums' order, which the count may change, only roundings do
    again = run(tide, xs[::-1], dtype)[::-1]
    for a, b in zip(outs, again):
        assert bool((a == b).all())


@pytest.mark.parametrize("rows,cols", [(4096, 8200), (8200, 4096)])
def test_large(tide, rows, cols):
    """Large tiles, split products, and two pieces of about 1 GiB; the reference in
    64 bits on the GPU."""
    import torch

    gen = torch.Generator("cuda").manual_seed(rows)
    xs = [torch.randn(rows, cols, generator=gen, device="cuda") for _ in range(4)]
    outs = [nan((rows, cols), "bf16") for _ in xs]
    tide.orthogonalize(xs, outs)
    for x, out in ((xs[0], outs[0]), (xs[3], outs[3])):
        y = x.double() if rows <= cols else x.double().t().contiguous()
        y /= y.norm() + EPS
        for _ in range(5):
            g = y @ y.t().contiguous()
            y = ABC[0] * y + (ABC[1] * g + ABC[2] * (g @ g)) @ y
        y = y if rows <= cols else y.t()
        # the same kind of matrix at 300 x 300 costs less than 0.2% on the CPU, the rounding to bf16 2^-8 / sqrt(3)
        assert float((out.double() - y).norm() / y.norm()) < 0.002 + 2.0**-8 / 3**0.5
        for part in ((slice(-3, None), slice(None)), (slice(None), slice(-3, None))):
            assert float((out.double() - y)[part].norm() / y[part].norm()) < 0.004 + 2.0**-8 / 3**0.5


@pytest.mark.parametrize("abc,steps", [(ABC, 1), (ABC, 2), (ABC, 3), (ABC, 4), (ABC, 8), ((1.5, -0.5, 0.0), 12),
                                       ((1.875, -1.25, 0.375), 6), ((1.0, 0.0, 0.0), 3), ((0.0, 1.0, 0.0), 1)])
def test_steps_and_coefficients(tide, abc, steps):
    for rows, cols in ((60, 140), (140, 60)):
        x = held(matrix(np.random.default_rng(steps), rows, cols, "noise"), "bf16")
        check(run(tide, [x], "bf16", steps=steps, coefficients=abc)[0], x, steps, abc, dtype="bf16")


@pytest.mark.parametrize("unit", [2.0**-100, 2.0**-130, 2.0**70, 2.0**110])
def test_any_magnitude(tide, unit):
    """Squares far outside fp32's range; below eps, eps decides."""
    x = held(np.random.default_rng(2).standard_normal((50, 90)) * unit, "f32")
    check(run(tide, [x], "f32", eps=0.0)[0], x, eps=0.0)
    if unit < 1:
        tiny = unit * 8
        check(run(tide, [x], "f32", eps=tiny)[0], x, eps=float(np.float32(tiny)))


@pytest.mark.parametrize("offset", [1, 3, 6])
@pytest.mark.parametrize("rows,cols", [(5, 9), (33, 70), (70, 33), (200, 301)])
def test_any_alignment_and_stride(tide, rows, cols, offset):
    import torch

    rng = np.random.default_rng(cols)
    for dtype in ("bf16", "f32"):
        xs = [held(matrix(rng, rows, cols, "noise"), dtype) for _ in range(2)]
        same = run(tide, xs, dtype)
        x = [Inside(rows, cols + 3, dtype, offset) for _ in xs]
        out = [Inside(rows, cols + 1, "bf16", offset) for _ in xs]
        for a, t in zip(xs, x):
            t.t[:, :cols].copy_(device(a, dtype))
        tide.orthogonalize([t.t[:, :cols] for t in x], [t.t[:, :cols] for t in out])
        for t, s in zip(out, same):
            assert torch.equal(t.t[:, :cols], s) and t.untouched() and bool((t.t[:, cols:] == 3.0).all())


def test_in_place_and_matrices_that_are_not_finite(tide):
    import torch

    rng = np.random.default_rng(4)
    xs = [held(matrix(rng, 100, 150, "noise"), "bf16") for _ in range(5)]
    want = run(tide, xs, "bf16")
    t = [device(x, "bf16") for x in xs]
    t[1].zero_()
    t[2][7, 9] = float("nan")
    t[4][99, 149] = -float("inf")
    tide.orthogonalize(t, t)
    assert torch.equal(t[0], want[0]) and torch.equal(t[3], want[3])
    assert not t[1].any()
    assert bool(t[2].isnan().all()) and bool(t[4].isnan().all())


def test_nothing_to_do(tide):
    import torch

    for shape in ((0, 5), (5, 0)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        tide.orthogonalize([x], [x])


def test_streams_and_graphs(tide):
    """On two streams at once, and captured: replays with new inputs equal the
    eager results."""
    import torch

    rng = np.random.default_rng(8)
    xs = [held(matrix(rng, 300, 450, "noise"), "f32") for _ in range(3)]
    x, outs = [device(a, "f32") for a in xs], [nan((300, 450), "bf16") for _ in xs]
    call = tide.orthogonalize_call(x, outs)
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for _ in range(3):
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        xs = [held(matrix(rng, 300, 450, "noise"), "f32") for _ in range(3)]
        for t, a in zip(x, xs):
            t.copy_(device(a, "f32"))
        graph.replay()
        torch.cuda.synchronize()
        for o, a in zip(outs, xs):
            check(o, a)
        same = run(tide, xs, "f32")
        assert all(torch.equal(a, b) for a, b in zip(outs, same))


def test_refusals_of_the_binding(tide):
    import torch

    x, o = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    p = torch.empty_like(o)
    for bad, error in (((x, [o]), TypeError), (([], []), TypeError), (([x], [o, p]), ValueError), (([x, x[:3]], [o, p]), ValueError),
                       (([x, o], [p, o]), ValueError), (([x.half()], [o]), TypeError), (([x], [x]), TypeError),
                       (([x], [o[:, :7]]), ValueError), (([x.cpu()], [o]), ValueError), (([x[0]], [o]), ValueError)):
        with pytest.raises(error):
            tide.orthogonalize(*bad)
    for kw in (dict(steps=0), dict(coefficients=(9.0, 0.0, 0.0)), dict(eps=-1.0)):
        with pytest.raises(tide.TideError):
            tide.orthogonalize([x], [o], **kw)
    with pytest.raises(tide.TideError):
        tide.orthogonalize([x, x], [o, o])
    with pytest.raises(tide.TideError):
        tide.orthogonalize([x], [o], workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
