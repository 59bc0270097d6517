"""GPU checks of outputs of the training-step operators that start on any
element of a larger allocation, with rows of any length: values within bounds
of 64-bit references and nothing written outside."""
import numpy as np
import pytest

from tests import training_reference as ref
from tests.test_gpu_checkpoint import DTYPES, close, device, dtype_of, grad_inputs, values
from tests.test_gpu_vocab_loss import Run, make

pytestmark = pytest.mark.gpu

CANARY, MARGIN = 3.0, 48


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


class Inside:
    """A rows x cols tensor `offset` elements past a 16-byte boundary, between canaries."""

    def __init__(self, rows, cols, dtype, offset):
        import torch

        self.all = torch.full((rows * cols + 2 * MARGIN,), CANARY, dtype=dtype_of(dtype), device="cuda")
        self.first, self.last = MARGIN + offset, MARGIN + offset + rows * cols
        self.t = self.all[self.first:self.last].view(rows, cols)
        assert self.t.data_ptr() % 16 == offset * self.all.element_size() % 16

    def untouched(self):
        return bool((self.all[:self.first] == CANARY).all() and (self.all[self.last:] == CANARY).all())


# tokens, outs, ins: short rows; rows past a tile; split along the tokens; large tiles
WEIGHT_GRADS = [(33, 9, 7), (70, 130, 261), (2100, 65, 131), (600, 4111, 4099)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 3, 6])
@pytest.mark.parametrize("tokens,outs,ins", WEIGHT_GRADS)
def test_weight_grad(tide, tokens, outs, ins, offset, dtype, accumulate):
    fmt = "e4m3" if offset == 3 else "int8"
    dy, codes, scales, y, x = grad_inputs(tide, np.random.default_rng(tokens), tokens, outs, ins, fmt)
    dw = Inside(outs, ins, dtype, offset)
    old = values(np.random.default_rng(5), outs, ins, dtype) if accumulate else None
    if accumulate:
        dw.t.copy_(device(old, dtype))
    tide.checkpoint_weight_grad(dy, codes, scales, dw.t, alpha=0.5, accumulate=accumulate)
    close(dw.t, *ref.weight_grad(y, x, 0.5, old), dtype)
    assert dw.untouched()


# tokens, hidden, vocabulary: a tile; dH split along the vocabulary; odd everything
LOSSES = [(40, 21, 55), (70, 133, 6001), (261, 259, 1031)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [1, 2, 5])
@pytest.mark.parametrize("tokens,size,vocab", LOSSES)
def test_vocab_loss_gradients(tide, tokens, size, vocab, offset, dtype):
    import torch

    h, w, t, g = make(np.random.default_rng(size), tokens, size, vocab, 0.2)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    r = Run(tide, h, w, t, g, dtype)
    r.check(want)
    dh, dw = Inside(tokens, size, "bf16", offset), Inside(vocab, size, dtype, offset)
    loss, lse = Inside(1, tokens, "f32", offset), Inside(1, tokens, "f32", offset)
    tide.vocab_loss_grad(h.cuda(), w.cuda(), torch.from_numpy(t).cuda(), torch.from_numpy(g).cuda(), loss.t[0], lse.t[0],
                         dh.t, dw.t)
    for got, same in ((loss.t[0], r.loss), (lse.t[0], r.lse), (dh.t, r.dh), (dw.t, r.dw)):
        assert torch.equal(got, same)
    assert all(x.untouched() for x in (dh, dw, loss, lse))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,offset", [(5, 1, 1), (9, 31, 3), (64, 327, 1), (33, 1001, 2), (7, 4098, 5)])
def test_restore(tide, rows, cols, offset, dtype, fmt):
    x = values(np.random.default_rng(cols), rows, cols, dtype)
    c, s = ref.pack(x, fmt)
    import torch

    out = Inside(rows, cols, dtype, offset)
    tide.checkpoint_unpack(torch.from_numpy(c).cuda().view(dtype_of(fmt)), torch.from_numpy(s).cuda(), out.t)
    assert np.array_equal(out.t.double().cpu().numpy(), ref.unpack(c, s, fmt, cols))
    assert out.untouched()
