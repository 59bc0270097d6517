"""GPU checks of the 8-bit activation checkpoints and of the weight gradient
that reads them, against 64-bit references."""
import numpy as np
import pytest

from tests import training_reference as ref

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "int8"]
DTYPES = ["bf16", "f32"]


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def dtype_of(name):
    import torch

    return {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[name]


def empty_packed(tide, rows, cols, fmt, fill=0x55):
    import torch

    c, s = tide.checkpoint_layout(cols)
    codes = torch.full((rows, c), fill, dtype=torch.uint8, device="cuda").view(dtype_of(fmt))
    return codes, torch.full((rows, s), fill, dtype=torch.uint8, device="cuda")


def bits(t):
    import torch

    return t.contiguous().view(torch.uint8).cpu().numpy()


def device(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype_of(dtype)).cuda()


def values(rng, rows, cols, dtype):
    """Values over many magnitudes, as float64 that the type holds exactly."""
    import torch

    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-6, 7, (rows, 1))
    return torch.from_numpy(x).to(dtype_of(dtype)).double().numpy()


def check_pack(tide, x, t, fmt):
    """Packs the device matrix t of values x and restores it both ways."""
    import torch

    rows, cols = x.shape
    codes, scales = empty_packed(tide, rows, cols, fmt)
    tide.checkpoint_pack(t, codes, scales)
    want_c, want_s = ref.pack(x, fmt)
    got_c, got_s = bits(codes).reshape(want_c.shape), bits(scales).reshape(want_s.shape)
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)
    want = ref.unpack(want_c, want_s, fmt, cols)
    for dtype in DTYPES:
        out = torch.full((rows, cols), 7.0, dtype=dtype_of(dtype), device="cuda")
        tide.checkpoint_unpack(codes, scales, out)
        assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)
    return codes, scales, want


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 1000), (7, 255), (64, 2048), (1, 8192),
                                       (1025, 8), (300, 100), (0, 5), (5, 0)])
def test_pack_and_unpack(tide, rows, cols, fmt, dtype):
    x = values(np.random.default_rng(rows * 10007 + cols), rows, cols, dtype)
    check_pack(tide, x, device(x, dtype), fmt)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("offset,stride", [(0, 201), (1, 200), (3, 207), (0, 256), (8, 208)])
def test_strided_and_misaligned_rows(tide, offset, stride, fmt, dtype):
    """Rows of any pitch and phase; what lies between the rows of `out` stays."""
    import torch

    rows, cols = 37, 200
    x = values(np.random.default_rng(stride + offset), rows, cols, dtype)
    flat = torch.full((offset + rows * stride,), float("nan"), dtype=dtype_of(dtype), device="cuda")
    t = flat.as_strided((rows, cols), (stride, 1), offset)
    t.copy_(device(x, dtype))
    codes, scales, want = check_pack(tide, x, t, fmt)
    t.fill_(1.0)
    tide.checkpoint_unpack(codes, scales, t)
    assert np.array_equal(t.double().cpu().numpy(), want)
    mask = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    mask.as_strided((rows, cols), (stride, 1), offset).fill_(False)
    assert torch.isnan(flat[mask]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_borders(tide, fmt, dtype):
    """Blocks of zeros, of subnormals and of the largest numbers, maxima on and
    next to the unit's limits, values on and next to the middle between two
    codes, infinities and NaN (which take their block alone)."""
    import torch

    d = dtype_of(dtype)
    big, tiny = torch.finfo(d).max, torch.finfo(d).tiny * 2.0 ** (-7 if dtype == "bf16" else -23)
    blocks = []
    for top in (448.0, 127.5, 127.0, 112.0, 240.0, 2.0**-110, 2.0**-118, 2.0**-126, 2.0**120, 1.75 * 2.0**127):
        for f in (1.0, 1 - 2.0**-8, 1 + 2.0**-7):
            b = np.zeros(32)
            b[0] = min(top * f, big)
            if fmt == "e4m3":
                t = ref.e4m3_values()
                b[1:32] = ((t[1:] + t[:-1]) / 2)[3:127:4][:31] * top / 448.0
            else:
                b[1:32] = (np.arange(31) * 4 + 0.5) * top / 127.0
            blocks.append(b * np.where(np.arange(32) % 3 == 1, -1.0, 1.0))
    blocks += [np.zeros(32), -np.zeros(32), np.full(32, tiny), np.linspace(-1, 1, 32) * tiny * 50, np.full(32, big),
               np.full(32, -big)]
    for special in (np.nan, np.inf, -np.inf):
        for at in (0, 13, 31):
            b = np.linspace(-3, 3, 32)
            b[at] = special
            blocks.append(b)
        blocks.append(np.linspace(-3, 3, 32))  # untouched by its neighbours
    x = torch.from_numpy(np.concatenate(blocks)[None]).to(d)
    x = torch.where(torch.isinf(x) & torch.from_numpy(np.isfinite(np.concatenate(blocks)[None])), big, x)
    check_pack(tide, x.double().numpy(), x.cuda(), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_past_32_bits(tide, fmt):
    """A matrix of more than 2^31 elements: its last rows."""
    import torch

    rows, cols = (1 << 20) + 5, 2080
    t = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x = values(np.random.default_rng(1), 9, cols, "bf16")
    t[-9:] = device(x, "bf16")
    codes, scales = empty_packed(tide, rows, cols, fmt)
    tide.checkpoint_pack(t, codes, scales)
    want_c, want_s = ref.pack(x, fmt)
    assert np.array_equal(bits(codes[-9:].view(torch.uint8)).reshape(9, -1), want_c)
    assert np.array_equal(bits(scales[-9:]).reshape(9, -1), want_s)
    t.fill_(5.0)
    tide.checkpoint_unpack(codes, scales, t)
    assert np.array_equal(t[-9:].double().cpu().numpy(), ref.unpack(want_c, want_s, fmt, cols))
    assert not t[:-9].any()


def test_unpack_of_every_code_and_scale(tide):
    import torch

    for fmt in FORMATS:
        scales = torch.tensor([10, 11, 100, 127, 200, 246, 255], dtype=torch.uint8).repeat_interleave(8).repeat(7, 1)
        codes = torch.arange(256, dtype=torch.int64).repeat(7, 7).to(torch.uint8)
        want = ref.unpack(codes.numpy(), scales.numpy(), fmt, 7 * 256)
        out = torch.empty(7, 7 * 256, device="cuda")
        tide.checkpoint_unpack(codes.cuda().view(dtype_of(fmt)), scales.cuda(), out)
        assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)


# ------------------------------------------------------------ weight gradient


def grad_inputs(tide, rng, tokens, outs, ins, fmt):
    import torch

    x = rng.standard_normal((tokens, ins)) * 2.0 ** rng.integers(-3, 4, (1, ins))
    c, s = ref.pack(x, fmt)
    codes, scales = torch.from_numpy(c).cuda().view(dtype_of(fmt)), torch.from_numpy(s).cuda()
    dy = torch.from_numpy(rng.standard_normal((tokens, outs)) * 1e-2).to(torch.bfloat16)
    return dy.cuda(), codes, scales, dy.double().numpy(), ref.unpack(c, s, fmt, ins)


def close(got, want, err, dtype):
    """got (device) within err of want, plus half a step of its type."""
    half = 2.0**-8 if dtype == "bf16" else 2.0**-24
    g = got.double().cpu().numpy()
    bound = err * (1 + half) + half * np.abs(want) + 2.0**-140
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (int(bad.sum()), float((np.abs(g - want) / bound).max()))


SHAPES = [(1, 1, 1), (7, 5, 33), (63, 96, 100), (64, 128, 128), (65, 130, 257), (200, 64, 31), (512, 257, 96),
          (1000, 300, 500), (509, 768, 2048), (4096, 72, 40)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,outs,ins", SHAPES)
def test_weight_grad(tide, tokens, outs, ins, dtype, fmt):
    import torch

    dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(tokens + outs), tokens, outs, ins, fmt)
    dw = torch.full((outs, ins), float("nan"), dtype=dtype_of(dtype), device="cuda")
    tide.checkpoint_weight_grad(dy, codes, scales, dw)
    close(dw, *ref.weight_grad(y, x), dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [64, 130, 320])
def test_weight_grad_of_a_large_layer(tide, tokens, fmt):
    """Enough tiles for the large ones, ragged on both sides."""
    import torch

    outs, ins = 256 * 12 + 8, 256 * 16 - 5
    dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(tokens), tokens, outs, ins, fmt)
    for dtype in DTYPES:
        guard = torch.full((outs * ins + 64,), 3.0, dtype=dtype_of(dtype), device="cuda")
        dw = guard[32:-32].view(outs, ins)
        tide.checkpoint_weight_grad(dy, codes, scales, dw)
        close(dw, *ref.weight_grad(y, x), dtype)
        assert (guard[:32] == 3.0).all() and (guard[-32:] == 3.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("alpha,accumulate", [(1.0, True), (0.125, False), (-1.7, True), (0.0, True)])
@pytest.mark.parametrize("tokens,outs,ins", [(65, 130, 257), (2048, 64, 64)])
def test_weight_grad_alpha_and_accumulate(tide, tokens, outs, ins, alpha, accumulate, dtype):
    dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(3), tokens, outs, ins, "int8")
    old = values(np.random.default_rng(4), outs, ins, dtype)
    dw = device(old, dtype)
    tide.checkpoint_weight_grad(dy, codes, scales, dw, alpha=alpha, accumulate=accumulate)
    close(dw, *ref.weight_grad(y, x, float(np.float32(alpha)), old if accumulate else None), dtype)


def test_weight_grad_without_tokens(tide):
    import torch

    for accumulate in (False, True):
        dw = torch.full((40, 50), 2.0, device="cuda")
        c, s = tide.checkpoint_layout(50)
        tide.checkpoint_weight_grad(torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"),
                                    torch.empty(0, c, dtype=torch.int8, device="cuda"),
                                    torch.empty(0, s, dtype=torch.uint8, device="cuda"), dw, accumulate=accumulate)
        assert (dw == (2.0 if accumulate else 0.0)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("offset,stride", [(0, 130), (1, 136), (8, 136), (0, 131), (0, 200)])
def test_weight_grad_of_strided_dy(tide, offset, stride, fmt):
    import torch

    tokens, outs, ins = 150, 130, 70
    dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(stride), tokens, outs, ins, fmt)
    flat = torch.full((offset + tokens * stride + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = flat.as_strided((tokens, outs), (stride, 1), offset)
    t.copy_(dy)
    dw = torch.empty(outs, ins, device="cuda")
    tide.checkpoint_weight_grad(t, codes, scales, dw)
    close(dw, *ref.weight_grad(y, x), "f32")


def test_weight_grad_keeps_nan_blocks_to_their_columns(tide):
    import torch

    dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(9), 100, 40, 100, "int8")
    scales[17, 1] = 255
    dw = torch.empty(40, 100, device="cuda")
    tide.checkpoint_weight_grad(dy, codes, scales, dw)
    assert torch.isnan(dw[:, 32:64]).all()
    want, err = ref.weight_grad(y, x)
    keep = np.r_[0:32, 64:100]
    close(dw[:, torch.from_numpy(keep).cuda()], want[:, keep], err[:, keep], "f32")


def test_weight_grad_against_differences(tide):
    """The gradient of f(W) = sum(y * r), y = X W^T, is the weight gradient
    from dy = r: f is linear in W, so a difference of f is exact in 64 bits."""
    import torch

    rng = np.random.default_rng(11)
    dy, codes, scales, y, x = grad_inputs(tide, rng, 90, 20, 70, "e4m3")
    dw = torch.empty(20, 70, device="cuda")
    tide.checkpoint_weight_grad(dy, codes, scales, dw)
    w = rng.standard_normal((20, 70))
    _, err = ref.weight_grad(y, x)
    for o, i in ((0, 0), (19, 69), (7, 33)):
        step = np.zeros_like(w)
        step[o, i] = 1.0
        diff = (((x @ (w + step).T) * y).sum() - ((x @ (w - step).T) * y).sum()) / 2
        assert abs(float(dw[o, i]) - diff) <= err[o, i] + 1e-9


# ------------------------------------------------------------ streams, graphs, workspaces


def test_a_layer_between_its_passes(tide):
    """Pack, restore and weight gradient as a step uses them, on a stream of
    its own, eagerly and as a captured graph with new inputs per replay; the
    gradient goes on to the reduce-scatter."""
    import torch

    rng = np.random.default_rng(21)
    tokens, outs, ins, W = 700, 96, 160, 2
    x = torch.empty(tokens, ins, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty(tokens, outs, dtype=torch.bfloat16, device="cuda")
    codes, scales = empty_packed(tide, tokens, ins, "int8")
    back = torch.empty(tokens, ins, dtype=torch.bfloat16, device="cuda")
    grads = [[torch.zeros(outs, ins, dtype=torch.bfloat16, device="cuda")] for _ in range(W)]
    plan = tide.Plan(W, [(outs, ins)])
    shards = [torch.zeros(plan.shard_elems, device="cuda") for _ in range(W)]
    calls = [tide.checkpoint_pack_call(x, codes, scales), tide.checkpoint_unpack_call(codes, scales, back),
             tide.checkpoint_weight_grad_call(dy, codes, scales, grads[0][0]),
             tide.reduce_scatter_call(plan, grads, shards)]
    side = torch.cuda.Stream()

    def fill():
        x.copy_(torch.from_numpy(rng.standard_normal((tokens, ins))))
        dy.copy_(torch.from_numpy(rng.standard_normal((tokens, outs))))
        torch.cuda.synchronize()

    def check():
        torch.cuda.synchronize()
        c, s = ref.pack(x.double().cpu().numpy(), "int8")
        assert np.array_equal(bits(codes).reshape(tokens, -1), c)
        want = ref.unpack(c, s, "int8", ins)
        assert np.array_equal(back.double().cpu().numpy(), want)
        close(grads[0][0], *ref.weight_grad(dy.double().cpu().numpy(), want), "bf16")
        got = torch.cat([t.view(-1, ins) for t in shards])[:outs]
        assert torch.equal(got, grads[0][0].float() + grads[1][0].float())

    fill()
    for c in calls:
        c(side)
    check()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        for c in calls:
            c()
    for _ in range(4):
        fill()
        for t in (codes, scales, back, grads[0][0], *shards):
            t.zero_()
        graph.replay()
        check()


def test_two_weight_gradients_at_once(tide):
    """Calls without a workspace on two streams do not share one."""
    import torch

    jobs = []
    for k in range(2):
        dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(30 + k), 3000, 65, 90, FORMATS[k])
        jobs.append((dy, codes, scales, torch.empty(65, 90, device="cuda"), ref.weight_grad(y, x), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for dy, codes, scales, dw, _, stream in jobs:
            tide.checkpoint_weight_grad(dy, codes, scales, dw, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, dw, (want, err), _ in jobs:
        close(dw, want, err, "f32")


def test_results_repeat_bit_for_bit(tide):
    import torch

    dy, codes, scales, _, _ = grad_inputs(tide, np.random.default_rng(40), 2000, 200, 300, "e4m3")
    ws = torch.empty(tide.checkpoint_weight_grad_workspace(dy, 300), dtype=torch.uint8, device="cuda")
    runs = []
    for k in range(3):
        ws.fill_(255 * (k & 1))
        dw = torch.empty(200, 300, device="cuda")
        tide.checkpoint_weight_grad(dy, codes, scales, dw, workspace=ws)
        runs.append(dw)
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_binding_refusals(tide):
    import torch

    x = torch.zeros(4, 64, device="cuda")
    codes, scales = empty_packed(tide, 4, 64, "int8")
    cases = [
        lambda: tide.checkpoint_pack(x.half(), codes, scales),
        lambda: tide.checkpoint_pack(x[0], codes, scales),
        lambda: tide.checkpoint_pack(x.t(), codes, scales),
        lambda: tide.checkpoint_pack(x[:, :60].t().contiguous().t(), codes, scales),
        lambda: tide.checkpoint_pack(x[:, :30], codes, scales),
        lambda: tide.checkpoint_pack(x[:1].expand(4, 64), codes, scales),
        lambda: tide.checkpoint_pack(x, codes.view(torch.uint8), scales),
        lambda: tide.checkpoint_pack(x, codes, scales.view(torch.int8)),
        lambda: tide.checkpoint_pack(x, codes[:3], scales),
        lambda: tide.checkpoint_unpack(codes, scales[:, :1], x),
        lambda: tide.checkpoint_weight_grad(x, codes, scales, torch.zeros(64, 64, device="cuda")),
        lambda: tide.checkpoint_weight_grad(x.bfloat16(), codes, scales, torch.zeros(63, 64, device="cuda")),
        lambda: tide.checkpoint_weight_grad(x.bfloat16(), codes, scales, torch.zeros(64, 96, device="cuda")),
        lambda: tide.checkpoint_weight_grad(x.bfloat16(), codes, scales, torch.zeros(64, 80, device="cuda")[:, :64]),
        lambda: tide.checkpoint_weight_grad(x.bfloat16(), codes, scales, torch.zeros(64, 64, device="cuda"),
                                            workspace=torch.zeros(64, device="cuda")),
    ]
    for case in cases:
        with pytest.raises((TypeError, ValueError)):
            case()
    dy = torch.zeros(4, 63, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tide.TideError):
        tide.checkpoint_weight_grad(dy, codes, scales, torch.zeros(63, 64, device="cuda"),
                                    workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
