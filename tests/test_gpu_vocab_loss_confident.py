"""GPU checks of the vocabulary loss of likely targets among large logits: the
loss is far smaller than the logits whose difference it is."""
import numpy as np
import pytest

from tests.test_gpu_vocab_loss import Run, bf16, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


# few tokens; small tiles without and with a list; large tiles
@pytest.mark.parametrize("tokens,vocab", [(10, 601), (100, 1200), (300, 1200), (2900, 4500)])
@pytest.mark.parametrize("scale", [0.25, 16.0, 64.0, 1024.0])
def test_large_logits(tide, tokens, vocab, scale):
    """Each token looks at one column of the weights, so that its logits are
    exact; the target is the largest for two tokens of three, and logits are 8
    to 32 thousand."""
    rng = np.random.default_rng(tokens)
    size = 24
    # steps of 1/8 are those of bf16 at 31: gaps of 1/8 to 1.5, times scale
    w = 31.0 - rng.integers(3, 13, (vocab, size)) / 8.0
    top = rng.integers(0, vocab, size)
    w[top, np.arange(size)] = 31.0
    at = np.arange(tokens) % size
    h = np.zeros((tokens, size))
    h[np.arange(tokens), at] = scale
    t = np.where(np.arange(tokens) % 3 < 2, top[at], rng.integers(0, vocab, tokens))
    g = rng.uniform(0.5, 1.0, tokens).astype(np.float32)
    z = scale * w.T[at]
    gap = z.max(-1, keepdims=True) - z
    s = np.exp(-gap).sum(-1)
    loss = gap[np.arange(tokens), t] + np.log(s)
    # Of the sum: at most 128 additions in a tile and 12 after it of 2^-24 each; an
    # exponential's argument is off by 4 roundings of 2^-24 of the gap,
    # itself by 2^-23.  Then the logarithm (2^-23), the gap and the sum of both.
    p = np.exp(-gap) / s[:, None]
    err = 2.0**-24 * (140 + (p * (4 * gap + 4)).sum(-1) + 2 * gap[np.arange(tokens), t] + 2 * np.abs(loss))
    for r in (Run(tide, bf16(h), bf16(w), t, None), Run(tide, bf16(h), bf16(w), t, g, "f32")):
        got = r.loss.double().cpu().numpy()
        assert (np.abs(got - loss) <= err).all(), float((np.abs(got - loss) / err).max())
        assert (got >= 0.0).all()
        lse = z.max(-1) + np.log(s)
        assert (np.abs(r.lse.double().cpu().numpy() - lse) <= err + 2.0**-24 * lse).all()
    # every row of dweight: g times the gradients' sum over the tokens of a column,
    # each rounded to bf16 (2^-8) from its exponentials' 11 bits (2^-11)
    dz = p.copy()
    dz[np.arange(tokens), t] = np.expm1(-loss)
    e = np.abs(dz) * (2.0**-8 + 2.0**-10) + err[:, None] * p
    e[np.arange(tokens), t] += err
    dw, bound = np.zeros((size, vocab)), np.zeros((size, vocab))
    np.add.at(dw, at, dz * (g * scale)[:, None])
    np.add.at(bound, at, e * (g * scale)[:, None])
    diff = np.abs(r.dw.double().cpu().numpy().T - dw)
    bound += 2.0**-20 * bound + 2.0**-23 * np.abs(dw) + scale * 2.0**-38
    assert (diff <= bound).all(), float((diff / bound).max())


def test_losses_are_not_negative(tide):
    """States along their targets' weights: losses from 0 up, never below."""
    rng = np.random.default_rng(3)
    h, w, t, _ = make(rng, 3000, 64, 5000)
    h = bf16(h.double().numpy() * rng.uniform(1, 20, (3000, 1)))
    r = Run(tide, h, w, t, None)
    assert bool((r.loss >= 0).all())
    z = h.double().numpy() @ w.double().numpy().T
    m = z.max(-1)
    loss = m + np.log(np.exp(z - m[:, None]).sum(-1)) - z[np.arange(3000), t]
    assert (loss < 1e-6).sum() > 100
