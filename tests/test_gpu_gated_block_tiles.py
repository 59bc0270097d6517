"""GPU checks of the gated block and its gradients at sizes whose products go to
the largest tiles, over many steps of k, split and whole, and from rows that are
copied first; against 64-bit references on the GPU, every element within its
bound."""
import pytest

pytestmark = pytest.mark.gpu

# tokens, hidden, ffn.  Forward by one round of tiles of 256; by those of copied, filled up rows (hidden is no multiple of
# 32), dx split in seven and dW over many rounds; all three products by tiles of 256, whole ones and split ones, ragged
SIZES = [(2048, 1024, 4096), (500, 4104, 14300), (2048, 2056, 8200)]


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def inputs(seed, tokens, hidden, ffn):
    """x, the weights and dout in bf16; tokens of many magnitudes."""
    import torch

    gen = torch.Generator("cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x = rand(tokens, hidden) * 2.0 ** torch.randint(-3, 4, (tokens, 1), generator=gen, device="cuda")
    return [t.bfloat16() for t in (x, rand(ffn, hidden) * hidden**-0.5, rand(ffn, hidden) * hidden**-0.5, rand(tokens, ffn) * 1e-2)]


def nan(shape, dtype):
    import torch

    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def check(tide, data, act, dtype, accumulate, views=None):
    """Both passes, from kept gates and without; `views`: other places of x, the
    weights and dout, which hold the same values."""
    import torch

    from tests import sublayer_reference_gpu as ref

    x, wg, wu, dout = views or data
    (tokens, hidden), ffn = x.shape, wg.shape[0]
    out, plain, gates = nan((tokens, ffn), x.dtype), nan((tokens, ffn), x.dtype), nan((tokens, 2 * ffn), x.dtype)
    tide.gated_block(x, wg, wu, out, gates, activation=act)
    tide.gated_block(x, wg, wu, plain, activation=act)
    assert torch.equal(out, plain)
    wide = [t.double() for t in data]
    want = ref.gated_block(*wide[:3], act)
    ref.close(out, *want["out"], "bf16", "out")
    ref.close(gates, *want["gates"], "bf16", "gates")
    old = None
    if accumulate:
        gen = torch.Generator("cuda").manual_seed(1)
        old = [torch.randn(ffn, hidden, generator=gen, device="cuda").mul_(0.1).to(dtype) for _ in range(2)]
    for kept in (None, gates):
        dx, *dw = nan((tokens, hidden), x.dtype), nan((ffn, hidden), dtype), nan((ffn, hidden), dtype)
        if old:
            for a, b in zip(dw, old):
                a.copy_(b)
        tide.gated_block_grad(dout, x, wg, wu, dx, *dw, gates=kept, activation=act, accumulate=accumulate)
        want = ref.gated_block_grad(wide[3], *wide[:3], act, None if kept is None else kept.double(),
                                    old and [t.double() for t in old])
        for (name, (value, bound, rms)), got in zip(want.items(), (dx, *dw)):
            own = "bf16" if got.dtype == torch.bfloat16 else "f32"
            ref.close(got, value, bound, own, (name, kept is not None))
            assert float((got.double() - value).norm()) <= rms, (name, kept is not None)
        del want


@pytest.mark.parametrize("act,dtype,accumulate", [("silu", "bfloat16", False), ("gelu", "float32", True)])
@pytest.mark.parametrize("tokens,hidden,ffn", SIZES)
def test_sizes(tide, tokens, hidden, ffn, act, dtype, accumulate):
    import torch

    check(tide, inputs(tokens + hidden, tokens, hidden, ffn), act, getattr(torch, dtype), accumulate)


def test_rows_on_any_element(tide):
    """Large tiles from copies of rows that start anywhere, with gaps."""
    import torch

    data = inputs(7, 2048, 2056, 8200)
    views = []
    for k, t in enumerate(data):
        wide = nan((t.shape[0], t.shape[1] + 3 + k), t.dtype)
        views.append(wide[:, 1 + k:1 + k + t.shape[1]])
        views[-1].copy_(t)
    check(tide, data, "silu", torch.bfloat16, False, views)
