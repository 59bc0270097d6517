"""GPU checks of the gradients of words that are unlikely for every token."""
import numpy as np
import pytest

from tests.test_gpu_vocab_loss import Run, bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


# few tokens; small tiles; with more tokens than one of them; large tiles
@pytest.mark.parametrize("tokens,vocab", [(10, 601), (100, 1200), (300, 1200), (2900, 4500)])
@pytest.mark.parametrize("ranges", [1.0, 1e-6])
def test_unlikely_words(tide, tokens, vocab, ranges):
    """Logits that are the same for all tokens, between words of logit 0 (some in
    every tile) words 1 to 42 below: their rows of dweight are as exact as the
    others'.  dz's exponentials are rounded by 2^-11 and dz by 2^-8; the terms of
    a row have one sign, so its sum is off by no more than that and what the
    sums and exponents in fp32 add (2^-23 for each of the tokens, and 4 roundings
    of 2^-24 of a gap of up to 42)."""
    rng = np.random.default_rng(vocab)
    size = 8
    gap = rng.integers(1, 43, vocab).astype(float)
    gap[::13] = 0.0
    w = np.zeros((vocab, size))
    w[:, 0] = -gap
    h = np.zeros((tokens, size))
    h[:, 0], h[:, 1] = 1.0, 2.0
    t = rng.integers(0, (vocab + 12) // 13, tokens) * 13
    g = (ranges ** rng.random(tokens)).astype(np.float32)
    r = Run(tide, bf16(h), bf16(w), t, g, "f32")
    p = np.exp(-gap) / np.exp(-gap).sum()
    want = g.astype(float).sum() * p
    far = gap > 0
    got = r.dw.double().cpu().numpy()[far]
    bound = 1.01 * (2.0**-8 + 2.0**-11 + (tokens + 64) * 2.0**-23 + 2.0**-15) * want[far]
    for column, factor in ((0, 1.0), (1, 2.0)):
        diff = np.abs(got[:, column] - factor * want[far])
        assert (diff <= factor * bound).all(), float((diff / factor / bound).max())
    assert not got[:, 2:].any()


def test_what_is_below_the_range(tide):
    """Exponentials below 2^-62 are off by 2^-73 at most: gaps of 43 to 90."""
    vocab, size, tokens = 500, 8, 20
    gap = np.where(np.arange(vocab) % 4 == 0, 0.0, 43.0 + np.arange(vocab) % 48)
    w, h = np.zeros((vocab, size)), np.zeros((tokens, size))
    w[:, 0], h[:, 0] = -gap, 1.0
    t, g = np.zeros(tokens, np.int64), np.ones(tokens, np.float32)
    r = Run(tide, bf16(h), bf16(w), t, g, "f32")
    p = np.exp(-gap) / np.exp(-gap).sum()
    diff = np.abs(r.dw[:, 0].double().cpu().numpy() - tokens * p)[gap > 0]
    assert (diff <= tokens * (1.01 * 2.0**-7 * p[gap > 0] + 2.0**-73)).all()
