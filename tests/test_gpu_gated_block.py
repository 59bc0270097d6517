"""GPU checks of the gated block and its gradients against 64-bit references,
within bounds of fp32 sums, bf16 operands and one rounding to each result's
type."""
import numpy as np
import pytest

from tests import sublayer_reference as ref
from tests.test_gpu_checkpoint import device, dtype_of
from tests.test_gpu_layer_norm import close, held, nan
from tests.test_gpu_training_alignment import Inside

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def inputs(rng, tokens, hidden, ffn):
    """x, the weights and dout as float64 that bf16 holds; gates from small to
    far out on both sides."""
    x = rng.standard_normal((tokens, hidden)) * 2.0 ** rng.integers(-3, 4, (tokens, 1))
    wg, wu = (rng.standard_normal((ffn, hidden)) * hidden**-0.5 for _ in range(2))
    return [held(a, "bf16") for a in (x, wg, wu, rng.standard_normal((tokens, ffn)) * 1e-2)]


def check_grads(got, want, dtype):
    for (name, (value, bound, rms)), t in zip(want.items(), got):
        own = "bf16" if name == "dx" else dtype
        close(t, (value, bound), own, name)
        assert np.sqrt(((t.double().cpu().numpy() - value) ** 2).sum()) <= rms, name


class Block:
    """All the passes on device copies of float64 arrays."""

    def __init__(self, tide, x, wg, wu, dout, act, dtype="bf16", old=None):
        tokens, hidden = x.shape
        ffn = wg.shape[0]
        self.act, self.dtype = act, dtype
        self.x, self.wg, self.wu, self.dout = (device(a, "bf16") for a in (x, wg, wu, dout))
        self.out, self.plain = nan((tokens, ffn), "bf16"), nan((tokens, ffn), "bf16")
        self.gates = nan((tokens, 2 * ffn), "bf16")
        tide.gated_block(self.x, self.wg, self.wu, self.out, self.gates, activation=act)
        tide.gated_block(self.x, self.wg, self.wu, self.plain, activation=act)
        self.grads = []
        for gates in (None, self.gates):
            dx, dg, du = nan((tokens, hidden), "bf16"), nan((ffn, hidden), dtype), nan((ffn, hidden), dtype)
            if old is not None:
                dg.copy_(device(old[0], dtype))
                du.copy_(device(old[1], dtype))
            tide.gated_block_grad(self.dout, self.x, self.wg, self.wu, dx, dg, du, gates=gates, activation=act,
                                  accumulate=old is not None)
            self.grads.append((dx, dg, du))

    def check(self, x, wg, wu, dout, old=None):
        import torch

        want = ref.gated_block(x, wg, wu, self.act)
        close(self.out, want["out"], "bf16", "out")
        assert torch.equal(self.out, self.plain)
        close(self.gates, want["gates"], "bf16", "gates")
        for got, gates in zip(self.grads, (None, self.gates.double().cpu().numpy())):
            check_grads(got, ref.gated_block_grad(dout, x, wg, wu, self.act, gates, old), self.dtype)


# tokens, hidden, ffn: up to 16 tokens in few and in many workgroups; one small tile; rows that need a copy; split tiles;
# more tiles than workgroups, of each product; large tiles
SIZES = [(1, 8, 1), (1, 64, 32), (3, 40, 33), (16, 100, 70), (16, 2048, 768), (5, 33, 17), (7, 64, 8200), (2, 1000, 8193),
         (17, 64, 64), (64, 72, 130), (130, 257, 131), (200, 520, 1000), (33, 2048, 200), (600, 1000, 700), (2100, 40, 4100),
         (2100, 2200, 96), (520, 8200, 40), (40, 8200, 300), (20, 72, 9001), (130, 264, 4100)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,hidden,ffn", SIZES)
def test_sizes(tide, tokens, hidden, ffn, act):
    data = inputs(np.random.default_rng(tokens + ffn), tokens, hidden, ffn)
    Block(tide, *data, act, "f32" if (tokens + ffn) % 2 else "bf16").check(*data)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,hidden,ffn", [(9, 64, 96), (300, 130, 70), (900, 520, 300)])
def test_accumulate(tide, tokens, hidden, ffn, dtype):
    rng = np.random.default_rng(tokens)
    data = inputs(rng, tokens, hidden, ffn)
    old = [held(rng.standard_normal((ffn, hidden)) * 0.1, dtype) for _ in range(2)]
    Block(tide, *data, "silu", dtype, old).check(*data, old)


@pytest.mark.parametrize("offset", [1, 3, 6])
@pytest.mark.parametrize("tokens,hidden,ffn", [(5, 40, 24), (16, 2001, 100), (70, 133, 57), (300, 256, 96)])
def test_any_alignment_and_stride(tide, tokens, hidden, ffn, offset):
    """Rows with gaps, on any element, and nothing written outside the rows."""
    data = inputs(np.random.default_rng(ffn), tokens, hidden, ffn)
    sizes = dict(x=(tokens, hidden, 3), wg=(ffn, hidden, 1), wu=(ffn, hidden, 2), dout=(tokens, ffn, 5), out=(tokens, ffn, 1),
                 gates=(tokens, 2 * ffn, 3), dx=(tokens, hidden, 2))
    t = {k: Inside(r, c + gap, "bf16", offset) for k, (r, c, gap) in sizes.items()}
    v = {k: t[k].t[:, :c] for k, (_, c, _) in sizes.items()}
    for k, a in zip(("x", "wg", "wu", "dout"), data):
        v[k].copy_(device(a, "bf16"))
    dg, du = Inside(ffn, hidden, "f32", offset), Inside(ffn, hidden, "f32", offset)
    tide.gated_block(v["x"], v["wg"], v["wu"], v["out"], v["gates"], activation="gelu")
    want = ref.gated_block(*data[:3], "gelu")
    close(v["out"], want["out"], "bf16", "out")
    close(v["gates"], want["gates"], "bf16", "gates")
    for gates in (None, v["gates"]):
        tide.gated_block_grad(v["dout"], v["x"], v["wg"], v["wu"], v["dx"], dg.t, du.t, gates=gates, activation="gelu")
        kept = None if gates is None else gates.double().cpu().numpy()
        check_grads((v["dx"], dg.t, du.t), ref.gated_block_grad(data[3], *data[:3], "gelu", kept), "f32")
    assert all(x.untouched() for x in (*t.values(), dg, du))
    for k, (_, c, _) in sizes.items():
        assert bool((t[k].t[:, c:] == 3.0).all())


@pytest.mark.parametrize("tokens", [9, 200])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_gates(tide, tokens, act):
    """Gates at the ends of their range: out and the gradients stay finite, and
    where the activation has reached its limit they are exactly u's."""
    import torch

    hidden, ffn = 32, 40
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([2.0**60, -(2.0**60), 1e4, -1e4, 200.0, -200.0, 0.0, 1.0, -1.0], device="cuda").repeat(23)[:tokens]
    x[:, 1] = 1.0
    wg, wu = (torch.zeros(ffn, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wg[:, 0] = 1.0
    wu[:, 1] = 3.0
    out, gates = nan((tokens, ffn), "bf16"), nan((tokens, 2 * ffn), "bf16")
    tide.gated_block(x, wg, wu, out, gates, activation=act)
    for r in range(9):
        z = float(x[r, 0])
        a, d, _ = ref.act(np.array([z if abs(z) < 1e6 else np.sign(z) * 1e6]), act)
        a = float(a[0]) * (z / 1e6 if z > 1e6 else 1.0)
        assert float(out[r, 0]) == pytest.approx(3 * a, rel=2.0**-8 + 2.0**-18, abs=1e-30)
    dy = torch.ones_like(out)
    for kept in (None, gates):
        dx, dg, du = nan((tokens, hidden), "bf16"), nan((ffn, hidden), "f32"), nan((ffn, hidden), "f32")
        tide.gated_block_grad(dy, x, wg, wu, dx, dg, du, gates=kept, activation=act)
        for t in (dx, dg, du):
            assert bool(t.isfinite().all())
        for r in range(9):
            z = float(np.clip(float(x[r, 0]), -1e6, 1e6))
            d = float(ref.act(np.array([z]), act)[1][0])
            # 40 columns of 3 * slope, each rounded to bf16, and the sum once more
            assert float(dx[r, 0]) == pytest.approx(120 * d, rel=2.0**-7 + 2.0**-15, abs=1e-30)


@pytest.mark.parametrize("tokens", [5, 16, 17, 300])
def test_values_that_are_not_finite_stay_in_their_rows(tide, tokens):
    import torch

    data = inputs(np.random.default_rng(tokens), tokens, 72, 50)
    b = Block(tide, *data, "silu")
    x, dout, wg = b.x.clone(), b.dout.clone(), b.wg.clone()
    x[tokens - 1, 5] = float("nan")
    wg[49, 70] = float("nan")
    out, gates = torch.empty_like(b.out), torch.empty_like(b.gates)
    tide.gated_block(x, wg, b.wu, out, gates)
    assert torch.equal(out[:-1, :-1], b.out[:-1, :-1]) and bool(out[-1].isnan().all()) and bool(out[:, -1].isnan().all())
    assert torch.equal(gates[:-1, 50:], b.gates[:-1, 50:])
    dout[tokens - 2, 3] = float("nan")
    for kept, same in ((None, b.grads[0]), (b.gates, b.grads[1])):
        dx, dg, du = (torch.empty_like(t) for t in same)
        tide.gated_block_grad(dout, b.x, b.wg, b.wu, dx, dg, du, gates=kept)
        keep = torch.arange(tokens, device="cuda") != tokens - 2
        assert torch.equal(dx[keep], same[0][keep]) and bool(dx[tokens - 2].isnan().all())
        cols = torch.arange(50, device="cuda") != 3
        assert torch.equal(dg[cols], same[1][cols]) and torch.equal(du[cols], same[2][cols])
        assert bool(dg[3].isnan().all()) and bool(du[3].isnan().all())


def test_no_tokens(tide):
    import torch

    x, w = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda"), torch.ones(24, 40, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    tide.gated_block(x, w, w, out)
    for dtype in ("bf16", "f32"):
        dg, du = (torch.ones(24, 40, dtype=dtype_of(dtype), device="cuda") for _ in range(2))
        tide.gated_block_grad(out, x, w, w, x, dg, du, accumulate=True)
        assert bool((dg == 1).all()) and bool((du == 1).all())
        tide.gated_block_grad(out, x, w, w, x, dg, du)
        assert not dg.any() and not du.any()


def test_more_than_2_31_gates(tide):
    import torch

    tokens, hidden, ffn, last = 70_000, 64, 16384, 6
    data = inputs(np.random.default_rng(3), last, hidden, ffn)
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[-last:].copy_(device(data[0], "bf16"))
    wg, wu = device(data[1], "bf16"), device(data[2], "bf16")
    dout = torch.zeros(tokens, ffn, dtype=torch.bfloat16, device="cuda")
    dout[-last:].copy_(device(data[3], "bf16"))
    out, gates = torch.empty_like(dout), torch.empty(tokens, 2 * ffn, dtype=torch.bfloat16, device="cuda")
    tide.gated_block(x, wg, wu, out, gates)
    want = ref.gated_block(*data[:3], "silu")
    close(out[-last:], want["out"], "bf16", "out")
    close(gates[-last:], want["gates"], "bf16", "gates")
    assert not out[:-last].any() and not gates[:-last:997].any()
    dx, dg, du = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    for kept in (None, gates):
        tide.gated_block_grad(dout, x, wg, wu, dx, dg, du, gates=kept)
        k = None if kept is None else kept[-last:].double().cpu().numpy()
        # the other tokens add zeros
        check_grads((dx[-last:], dg, du), ref.gated_block_grad(data[3], *data[:3], "silu", k), "bf16")
        assert not dx[:-last].any()


def test_streams_and_graphs(tide):
    """On two streams at once, and captured: replays with new inputs equal the
    eager results."""
    import torch

    data = inputs(np.random.default_rng(8), 700, 200, 300)
    b = Block(tide, *data, "silu")
    torch.cuda.synchronize()
    dx, dg, du = b.grads[0]
    fwd = tide.gated_block_call(b.x, b.wg, b.wu, b.out, b.gates)
    call = tide.gated_block_grad_call(b.dout, b.x, b.wg, b.wu, dx, dg, du)
    kept = tide.gated_block_grad_call(b.dout, b.x, b.wg, b.wu, *b.grads[1], gates=b.gates)
    want = [t.clone() for t in (b.out, b.gates, *b.grads[0], *b.grads[1])]
    for _ in range(3):
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            for c in (fwd, call, kept):
                c(s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((b.out, b.gates, *b.grads[0], *b.grads[1]), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd()
        call()
        kept()
    for seed in range(3):
        data = inputs(np.random.default_rng(seed), 700, 200, 300)
        for t, a in zip((b.x, b.wg, b.wu, b.dout), data):
            t.copy_(device(a, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        b.plain.copy_(b.out)
        b.check(*data)


def test_refusals_of_the_binding(tide):
    import torch

    def m(*shape, dtype=torch.bfloat16, device="cuda"):
        return torch.zeros(*shape, dtype=dtype, device=device)

    x, w, out, gates = m(4, 16), m(8, 16), m(4, 8), m(4, 16)
    for bad, error in (((x.float(), w, w, out), TypeError), ((x, w.half(), w, out), TypeError), ((x, w, w[:7], out), ValueError),
                       ((x, w[:, :8], w, out), ValueError), ((x, w, w, out[:3]), ValueError), ((x.cpu(), w, w, out), ValueError),
                       ((x, w, w, out, gates[:, :15]), ValueError), ((x, w, w, out, gates, "relu"), ValueError)):
        with pytest.raises(error):
            tide.gated_block(*bad)
    for bad, error in (((out, x, w, w, x, w, w.float()), TypeError), ((out[:, :7], x, w, w, x, w, w), ValueError),
                       ((out, x, w, w, x[:3], w, w), ValueError), ((out, x, w, w, x, m(8, 32)[:, :16], w), ValueError)):
        with pytest.raises(error):
            tide.gated_block_grad(*bad)
    with pytest.raises(tide.TideError):
        tide.gated_block_grad(out, x, w, w, x, w, w, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
