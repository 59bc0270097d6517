"""GPU checks of layer norm and its gradients against 64-bit references, within
bounds of fp32 arithmetic and one rounding to each result's type."""
import itertools

import numpy as np
import pytest

from tests import sublayer_reference as ref
from tests.test_gpu_checkpoint import device, dtype_of
from tests.test_gpu_training_alignment import Inside

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def held(a, dtype):
    """The float64 values that a's rounding to `dtype` holds."""
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype_of(dtype)).double().numpy()


def close(got, want, dtype, what):
    value, err = want
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - value) <= ref.rounded(value, err, dtype))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0], got[bad][0], np.broadcast_to(value, got.shape)[bad][0])


def inputs(rng, rows, cols, xt, yt, at, shift=0.0):
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-3, 4, (rows, 1)) + shift
    w, b = 1 + 0.3 * rng.standard_normal(cols), rng.standard_normal(cols)
    dy = rng.standard_normal((rows, cols)) * 1e-2
    return held(x, xt), held(w, at), held(b, at), held(dy, yt)


def nan(shape, dtype):
    import torch

    return torch.full(shape, float("nan"), dtype=dtype_of(dtype), device="cuda")


class Norm:
    """Both passes on device copies of float64 arrays."""

    def __init__(self, tide, x, w, b, dy, xt, yt, at, accumulate=False):
        rows, cols = x.shape
        self.types = xt, yt, at
        self.x, self.dy = device(x, xt), device(dy, yt)
        self.w, self.b = (None if v is None else device(v, at) for v in (w, b))
        self.out, self.mean, self.rstd = nan((rows, cols), yt), nan((rows,), "f32"), nan((rows,), "f32")
        tide.layer_norm(self.x, self.w, self.b, self.out, self.mean, self.rstd, eps=EPS)
        self.dx = nan((rows, cols), xt)
        self.dw, self.db = nan((cols,), at), nan((cols,), at)
        if accumulate:
            self.dw.copy_(self.w)
            self.db.copy_(self.b)
        tide.layer_norm_grad(self.dy, self.x, self.w, self.mean, self.rstd, self.dx, self.dw, self.db, accumulate=accumulate)

    def check(self, x, w, b, dy, accumulate=False):
        xt, yt, at = self.types
        one, zero = np.ones(x.shape[1]), np.zeros(x.shape[1])
        want = ref.layer_norm(x, one if w is None else w, zero if b is None else b, EPS)
        close(self.out, want["out"], yt, "out")
        close(self.mean, want["mean"], "f32", "mean")
        close(self.rstd, want["rstd"], "f32", "rstd")
        mean, rstd = self.mean.double().cpu().numpy(), self.rstd.double().cpu().numpy()
        want = ref.layer_norm_grad(dy, x, one if w is None else w, mean, rstd, *((w, b) if accumulate else ()))
        close(self.dx, want["dx"], xt, "dx")
        close(self.dw, want["dweight"], at, "dweight")
        close(self.db, want["dbias"], at, "dbias")


# rows, columns: a wave, a workgroup of each size a row; rows read by loops; each with whole and short pieces; more rows
# than workgroups
SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (4, 512), (5, 513), (6, 1000), (7, 1024), (3, 1025), (9, 2048), (3, 4095),
         (2, 4096), (2, 4097), (2, 8192), (3, 8200), (2, 16384), (2, 16385), (3, 20011), (300, 96), (5000, 40), (2500, 1030),
         (1100, 4100), (1, 16), (1000, 128), (777, 121), (333, 256), (4097, 200), (20000, 17), (70, 790), (40, 6200), (530, 12300), (20, 14000)]
TYPES = list(itertools.product(["bf16", "f32"], repeat=2))


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(tide, rows, cols, xt, yt):
    at = "f32" if (rows + cols) % 2 else "bf16"
    data = inputs(np.random.default_rng(rows + cols), rows, cols, xt, yt, at)
    Norm(tide, *data, xt, yt, at).check(*data)


@pytest.mark.parametrize("xt,yt", TYPES)
def test_a_mean_far_above_the_deviations(tide, xt, yt):
    for cols in (200, 3001, 20000):
        data = inputs(np.random.default_rng(cols), 5, cols, xt, yt, "f32", shift=1000.0)
        Norm(tide, *data, xt, yt, "f32").check(*data)


@pytest.mark.parametrize("at", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(33, 130), (600, 2500), (9, 16400)])
def test_accumulate(tide, rows, cols, at):
    data = inputs(np.random.default_rng(rows), rows, cols, "bf16", "f32", at)
    Norm(tide, *data, "bf16", "f32", at, accumulate=True).check(*data, accumulate=True)


@pytest.mark.parametrize("rows,cols", [(33, 130), (7, 16400)])
def test_without_weight_and_bias(tide, rows, cols):
    import torch

    x, w, b, dy = inputs(np.random.default_rng(1), rows, cols, "f32", "bf16", "f32")
    Norm(tide, x, None, None, dy, "f32", "bf16", "f32").check(x, None, None, dy)
    n = Norm(tide, x, w, None, dy, "f32", "bf16", "f32")
    n.check(x, w, None, dy)
    # neither of the sums, or one of them, is wanted; nor the statistics
    dx, db = torch.empty_like(n.dx), torch.empty_like(n.db)
    tide.layer_norm_grad(n.dy, n.x, n.w, n.mean, n.rstd, dx)
    assert torch.equal(dx, n.dx)
    tide.layer_norm_grad(n.dy, n.x, n.w, n.mean, n.rstd, dx, None, db)
    assert torch.equal(db, n.db)
    out = torch.empty_like(n.out)
    tide.layer_norm(n.x, n.w, None, out, eps=EPS)
    assert torch.equal(out, n.out)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("offset", [1, 3, 6])
@pytest.mark.parametrize("rows,cols", [(5, 7), (6, 1001), (4, 2048), (3, 16389)])
def test_any_alignment_and_stride(tide, rows, cols, offset, xt, yt):
    """Rows with gaps, on any element: the same results, and nothing written
    outside the rows."""
    import torch

    data = inputs(np.random.default_rng(cols), rows, cols, xt, yt, "bf16")
    n = Norm(tide, *data, xt, yt, "bf16")
    x, dy, out, dx = (Inside(rows, cols + g, t, offset) for t, g in ((xt, 3), (yt, 5), (yt, 1), (xt, 2)))
    x.t[:, :cols].copy_(n.x)
    dy.t[:, :cols].copy_(n.dy)
    w, b, dw, db = (Inside(1, cols, "bf16", offset) for _ in range(4))
    w.t[0].copy_(n.w)
    b.t[0].copy_(n.b)
    mean, rstd = Inside(1, rows, "f32", offset), Inside(1, rows, "f32", offset)
    tide.layer_norm(x.t[:, :cols], w.t[0], b.t[0], out.t[:, :cols], mean.t[0], rstd.t[0], eps=EPS)
    tide.layer_norm_grad(dy.t[:, :cols], x.t[:, :cols], w.t[0], mean.t[0], rstd.t[0], dx.t[:, :cols], dw.t[0], db.t[0])
    for got, same in ((out.t[:, :cols], n.out), (dx.t[:, :cols], n.dx), (dw.t[0], n.dw), (db.t[0], n.db),
                      (mean.t[0], n.mean), (rstd.t[0], n.rstd)):
        assert torch.equal(got, same)
    assert all(t.untouched() for t in (out, dx, dw, db, mean, rstd))
    for t in (out, dx):
        assert bool((t.t[:, cols:] == 3.0).all())


@pytest.mark.parametrize("cols", [40, 700, 3000, 9000, 17000])
def test_rows_that_are_not_finite(tide, cols):
    """They come out as NaN, and the others as without them."""
    import torch

    rows = 9
    data = inputs(np.random.default_rng(cols), rows, cols, "bf16", "bf16", "f32")
    n = Norm(tide, *data, "bf16", "bf16", "f32")
    x = n.x.clone()
    x[2, cols // 2] = float("nan")
    x[5, 0] = float("inf")
    x[7, cols - 1] = -float("inf")
    out, mean, rstd, dx = (torch.empty_like(t) for t in (n.out, n.mean, n.rstd, n.dx))
    tide.layer_norm(x, n.w, n.b, out, mean, rstd, eps=EPS)
    tide.layer_norm_grad(n.dy, x, n.w, mean, rstd, dx)
    keep = torch.tensor([r not in (2, 5, 7) for r in range(rows)], device="cuda")
    for got, same in ((out, n.out), (dx, n.dx)):
        assert torch.equal(got[keep], same[keep])
        assert bool(got[~keep].isnan().all())
    assert bool(rstd[~keep].isnan().all())


def test_constant_rows(tide):
    """No deviation: out is the bias, whatever the constant."""
    import torch

    for cols in (1, 300, 5000, 17000):
        x = torch.tensor([0.0, 1.0, -3.5, 2.0**100], device="cuda")[:, None].repeat(1, cols)
        b = torch.randn(cols, device="cuda")
        out, mean, rstd = torch.empty_like(x), *(torch.empty(4, device="cuda") for _ in range(2))
        tide.layer_norm(x, None, b, out, mean, rstd, eps=EPS)
        # 2^100's mean may be off by its sum's and division's roundings, which are taken back
        assert torch.equal(out[:3], b.expand(3, cols)) and torch.equal(mean, x[:, 0])
        assert bool(((rstd[:3].double() - EPS**-0.5).abs() < 8 * 2.0**-24 * EPS**-0.5).all())


def test_no_rows(tide):
    import torch

    none = torch.empty(0, 50, dtype=torch.bfloat16, device="cuda")
    stat = torch.empty(0, device="cuda")
    tide.layer_norm(none, None, None, none, stat, stat)
    dw, db = torch.ones(50, device="cuda"), torch.ones(50, device="cuda")
    tide.layer_norm_grad(none, none, None, stat, stat, none, dw, db, accumulate=True)
    assert bool((dw == 1).all()) and bool((db == 1).all())
    tide.layer_norm_grad(none, none, None, stat, stat, none, dw, db)
    assert not dw.any() and not db.any()


def test_more_than_2_31_values(tide):
    import torch

    rows, cols = 300_000, 7300
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    data = inputs(np.random.default_rng(3), 4, cols, "bf16", "bf16", "f32")
    x[-4:].copy_(device(data[0], "bf16"))
    w, b = device(data[1], "f32"), device(data[2], "f32")
    dy = torch.zeros_like(x)
    dy[-4:].copy_(device(data[3], "bf16"))
    out, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    tide.layer_norm(x, w, b, out, mean, rstd, eps=EPS)
    tide.layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db)
    want = ref.layer_norm(*data[:3], EPS)
    close(out[-4:], want["out"], "bf16", "out")
    assert torch.equal(out[:-4:1000], b.bfloat16().expand_as(out[:-4:1000])) and not dx[:-4].any()
    grads = ref.layer_norm_grad(data[3], data[0], data[1], mean[-4:].double().cpu().numpy(),
                                rstd[-4:].double().cpu().numpy())
    close(dx[-4:], grads["dx"], "bf16", "dx")
    # the other rows add zeros
    close(dw, grads["dweight"], "f32", "dweight")
    close(db, grads["dbias"], "f32", "dbias")


def test_streams_and_graphs(tide):
    """On two streams at once, and captured: replays with new inputs equal the
    eager results."""
    import torch

    data = inputs(np.random.default_rng(8), 900, 1500, "bf16", "bf16", "f32")
    n = Norm(tide, *data, "bf16", "bf16", "f32")
    torch.cuda.synchronize()
    call = tide.layer_norm_grad_call(n.dy, n.x, n.w, n.mean, n.rstd, n.dx, n.dw, n.db)
    fwd = tide.layer_norm_call(n.x, n.w, n.b, n.out, n.mean, n.rstd, EPS)
    want = [t.clone() for t in (n.out, n.dx, n.dw, n.db)]
    for _ in range(3):
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            s.wait_stream(torch.cuda.current_stream())
            call(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((n.out, n.dx, n.dw, n.db), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd()
        call()
    for seed in range(3):
        data = inputs(np.random.default_rng(seed), 900, 1500, "bf16", "bf16", "f32")
        n.x.copy_(device(data[0], "bf16"))
        n.dy.copy_(device(data[3], "bf16"))
        n.w.copy_(device(data[1], "f32"))
        n.b.copy_(device(data[2], "f32"))
        graph.replay()
        torch.cuda.synchronize()
        n.check(*data)


def test_refusals_of_the_binding(tide):
    import torch

    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w, stat = torch.ones(16, device="cuda"), torch.ones(4, device="cuda")
    out = torch.empty_like(x)
    for bad, error in (((x.half(), w, w, out), TypeError), ((x, w.half(), w, out), TypeError),
                       ((x, w, w.bfloat16(), out), TypeError), ((x, w[:15], w, out), ValueError),
                       ((x, w, w, out[:3]), ValueError), ((x, w, w, out.t()), ValueError),
                       ((x, w, w, out, stat[:3]), ValueError), ((x.cpu(), w, w, out), ValueError),
                       ((x[0], w, w, out), ValueError), ((x, w.cpu(), w, out), ValueError)):
        with pytest.raises(error):
            tide.layer_norm(*bad)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for bad, error in (((x, x, w, stat, stat, dx.float(), dw, dw), TypeError),
                       ((x, x, w, stat, stat, dx, dw.bfloat16(), dw), TypeError),
                       ((x[:, :8], x, w, stat, stat, dx, dw, dw), ValueError),
                       ((x, x, w, stat[1:], stat, dx, dw, dw), ValueError)):
        with pytest.raises(error):
            tide.layer_norm_grad(*bad)
    with pytest.raises(TypeError):
        tide.layer_norm_grad(x, x, w, stat, stat, dx, dw, dw, workspace=torch.empty(1 << 16, device="cuda"))
    with pytest.raises(tide.TideError):
        tide.layer_norm_grad(x, x, w, stat, stat, dx, dw, dw, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
