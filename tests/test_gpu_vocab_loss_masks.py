"""GPU checks of the vocabulary loss where a mask is part of the projection: a
column of weights that a constant of the states adds to every logit, -infinity
or the type's lowest number for the words that are left out, over whole tiles of
the vocabulary, with the other logits far below zero; and rows that such a mask
leaves nothing."""
import numpy as np
import pytest

from tests import training_reference as ref
from tests.test_gpu_vocab_loss import Run, make

pytestmark = pytest.mark.gpu

LOWEST = -(2.0 - 2.0**-7) * 2.0**127  # bf16's


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def masked(rng, tokens, size, vocab, mask, below):
    """States with a last column of 1, weights with a last column of `mask` for
    the words [256, 1024) and the last one and `below` for the others, targets
    among the others."""
    h, w, _, g = make(rng, tokens, size, vocab)
    out = np.zeros(vocab, bool)
    out[256:1024] = out[-1] = True
    h[:, -1] = 1.0
    w[:, -1] = below
    w[np.nonzero(out)[0], -1] = mask
    t = rng.choice(np.nonzero(~out)[0], tokens)
    return h, w, t, g, out


# one tile of few tokens, small tiles with and without a list, large tiles
@pytest.mark.parametrize("tokens", [10, 100, 300, 2900])
@pytest.mark.parametrize("below", [0.0, -200.0, -30000.0])
@pytest.mark.parametrize("mask", [-np.inf, LOWEST])
def test_masked_words(tide, tokens, mask, below):
    """As if the masked words were not there."""
    h, w, t, g, out = masked(np.random.default_rng(tokens), tokens, 72, 4500, mask, below)
    left = np.nonzero(~out)[0]
    small = ref.vocab_loss(h.double().numpy(), w.double().numpy()[left], np.searchsorted(left, t), g.astype(float))
    r = Run(tide, h, w, t, None)
    r.check({k: small[k] for k in ("loss", "lse")})
    r = Run(tide, h, w, t, g, "f32")
    assert not r.dw[out].any()
    r.dw = r.dw[left]
    # 0 times -infinity is NaN, in the formula too
    assert mask == LOWEST or bool(r.dh[:, -1].isnan().all())
    r.check({k: v for k, v in small.items() if k != "dhidden"})
    if mask == LOWEST:
        r.check({"dhidden": small["dhidden"]})


@pytest.mark.parametrize("tokens", [10, 100, 300])
def test_nothing_left_but_the_lowest_number(tide, tokens):
    """Every logit the lowest number: all words are as likely."""
    import torch

    size, vocab = 40, 1500
    h, w, t, g = make(np.random.default_rng(tokens), tokens, size, vocab)
    h[:, :] = 0.0
    h[:, -1] = 1.0
    w[:, -1] = LOWEST
    for r in (Run(tide, h, w, t, None), Run(tide, h, w, t, g, "f32")):
        # sums of 1500 ones, and a logarithm
        assert float((r.loss.double() - np.log(vocab)).abs().max()) < 2.0**-19
        assert bool((r.lse == LOWEST).all())
    want = np.zeros((vocab, size))
    np.add.at(want[:, -1], t, -g.astype(float))
    want[:, -1] += g.astype(float).sum() / vocab
    terms = np.zeros(vocab)
    np.add.at(terms, t, g.astype(float))
    terms += g.astype(float).sum() / vocab
    # dz rounded by 2^-8, its exponentials and sums far less
    assert (np.abs(r.dw.double().cpu().numpy() - want)[:, -1] <= 1.01 * 2.0**-8 * terms).all()
    assert not r.dw[:, :-1].any()


@pytest.mark.parametrize("tokens", [10, 300])
def test_nothing_left_but_minus_infinity(tide, tokens):
    """Every logit of one token -infinity: NaN in its loss, the others' are
    untouched."""
    import torch

    h, w, t, g, out = masked(np.random.default_rng(tokens), tokens, 72, 4500, -np.inf, 0.0)
    h[:, -1] = 0.0
    want = ref.vocab_loss(h.double().numpy(), np.where(np.isinf(w.double().numpy()), 0.0, w.double().numpy()), t)
    w[:, -1] = LOWEST
    h[7] = 0.0
    h[7, -1] = float("inf")
    r = Run(tide, h, w, t, None)
    assert bool(r.loss[7].isnan()) and not bool(torch.isfinite(r.lse[7]))
    keep = torch.from_numpy(np.arange(tokens) != 7).cuda()
    r.loss, r.lse = r.loss[keep], r.lse[keep]
    keep = keep.cpu().numpy()
    r.check({k: (want[k][0][keep], want[k][1][keep]) for k in ("loss", "lse")})
