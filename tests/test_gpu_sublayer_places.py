"""GPU checks that outputs may lie beside inputs: columns of one buffer, matrices
one right behind the other, an update in the place of its own matrix or of the
last row's gap."""
import numpy as np
import pytest

from tests.test_gpu_checkpoint import device
from tests.test_gpu_layer_norm import nan
from tests.test_orthogonalize_host import matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def columns(*widths, rows):
    """Neighbouring columns of one bf16 buffer."""
    buffer = nan((rows, sum(widths)), "bf16")
    return list(buffer.split(list(widths), 1))


@pytest.mark.parametrize("rows,cols", [(1, 40), (9, 200), (70, 1025), (5, 17000)])
def test_layer_norm_in_one_buffer(tide, rows, cols):
    import torch

    rng = np.random.default_rng(cols)
    x, out, dout, dx = columns(cols, cols, cols, cols, rows=rows)
    x.copy_(device(rng.standard_normal((rows, cols)), "bf16"))
    dout.copy_(device(rng.standard_normal((rows, cols)), "bf16"))
    # weight, bias, the statistics and the weights' gradients one behind the other
    vectors = nan((4 * cols + 2 * rows,), "f32")
    w, b, mean, rstd, dw, db = vectors.split([cols, cols, rows, rows, cols, cols])
    w.copy_(device(rng.standard_normal(cols), "f32"))
    b.copy_(device(rng.standard_normal(cols), "f32"))
    tide.layer_norm(x, w, b, out, mean, rstd)
    tide.layer_norm_grad(dout, x, w, mean, rstd, dx, dw, db)
    own = [t.clone() for t in (x, w, b, dout)]
    other = [nan((rows, cols), "bf16"), *(nan((rows,), "f32") for _ in range(2)), nan((rows, cols), "bf16"),
             *(nan((cols,), "f32") for _ in range(2))]
    tide.layer_norm(*own[:3], *other[:3])
    tide.layer_norm_grad(own[3], own[0], own[1], *other[1:])
    for got, want in zip((out, mean, rstd, dx, dw, db), other):
        assert torch.equal(got, want) and bool(want.isfinite().all())


@pytest.mark.parametrize("tokens", [3, 90])
def test_gated_block_in_one_buffer(tide, tokens):
    import torch

    hidden, ffn = 72, 100
    rng = np.random.default_rng(tokens)
    x, out, gates, dout, dx = columns(hidden, ffn, 2 * ffn, ffn, hidden, rows=tokens)
    x.copy_(device(rng.standard_normal((tokens, hidden)), "bf16"))
    dout.copy_(device(rng.standard_normal((tokens, ffn)), "bf16"))
    wg, wu, dwg, dwu = nan((4 * ffn, hidden), "bf16").split(ffn)
    for w in (wg, wu):
        w.copy_(device(rng.standard_normal((ffn, hidden)) * 0.1, "bf16"))
    tide.gated_block(x, wg, wu, out, gates)
    tide.gated_block_grad(dout, x, wg, wu, dx, dwg, dwu, gates=gates)
    a, b, c, d = (t.clone() for t in (x, wg, wu, dout))
    want = [nan(t.shape, "bf16") for t in (out, gates, dx, dwg, dwu)]
    tide.gated_block(a, b, c, *want[:2])
    tide.gated_block_grad(d, a, b, c, *want[2:], gates=want[1])
    for got, w in zip((out, gates, dx, dwg, dwu), want):
        assert torch.equal(got, w) and bool(w.isfinite().all())


def test_updates_in_one_buffer(tide):
    import torch

    rng = np.random.default_rng(1)
    xs = [matrix(rng, 40, 50, "noise") for _ in range(3)]
    want = [nan((40, 50), "bf16") for _ in xs]
    tide.orthogonalize([device(x, "bf16") for x in xs], want)
    t = columns(50, 50, 50, 50, 50, 50, rows=40)
    for a, x in zip(t[::2], xs):
        a.copy_(device(x, "bf16"))
    tide.orthogonalize(t[::2], t[1::2])
    assert all(torch.equal(a, b) for a, b in zip(t[1::2], want))
    tide.orthogonalize(t[::2], t[::2])
    assert all(torch.equal(a, b) for a, b in zip(t[::2], want))


def test_overlaps_are_refused(tide):
    """By the binding's calls too, before anything is launched."""
    import torch

    x = torch.ones(8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, 64, dtype=torch.bfloat16, device="cuda")
    v, stat = torch.ones(64, device="cuda"), torch.ones(8, device="cuda")
    wide = torch.ones(9, 64, dtype=torch.bfloat16, device="cuda")
    for refused in (lambda: tide.layer_norm(x, None, None, x), lambda: tide.layer_norm(wide[:8], None, None, wide[1:]),
                    lambda: tide.layer_norm_grad(x, x, None, stat, stat, x), lambda: tide.layer_norm_grad(x, x, v, stat, stat, wide[:8], v),
                    lambda: tide.gated_block(x, w, w, x), lambda: tide.gated_block_grad(x, wide[:8], w, w, x, w, w.clone()),
                    lambda: tide.orthogonalize([wide[:8], x], [x.clone(), wide[1:]])):
        with pytest.raises(tide.TideError, match="overlaps"):
            refused()
    torch.cuda.synchronize()
    assert all(bool((t == 1).all()) for t in (x, w, v, wide))
