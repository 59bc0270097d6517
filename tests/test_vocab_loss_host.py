"""Host-side checks of the vocabulary loss (no GPU): every refusal, made
before any device work (the addresses passed here are not device memory), and
the 64-bit reference against differences."""
import ctypes

import numpy as np
import pytest

from tests import training_reference as ref

INVALID, RANGE, ALIGN = -1, -2, -3
P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


CALL = dict(h=P, h_ld=64, w=P, w_ld=64, targets=P, grad=P, tokens=10, size=64, vocab=100, loss=P, lse=P, dh=P, dw=P,
            dtype=0, acc=0, ws=P, ws_bytes=1 << 40)
REFUSED = [
    (dict(h=0), INVALID), (dict(w=0), INVALID), (dict(targets=0), INVALID), (dict(loss=0), INVALID),
    (dict(ws=0), INVALID), (dict(ws_bytes=8), INVALID), (dict(tokens=-1), INVALID), (dict(size=0, h_ld=0, w_ld=0), INVALID),
    (dict(vocab=0), INVALID), (dict(vocab=-3), INVALID), (dict(h_ld=63), INVALID), (dict(w_ld=63), INVALID),
    (dict(tokens=(1 << 24) + 1), RANGE), (dict(vocab=(1 << 22) + 1), RANGE),
    (dict(size=(1 << 22) + 1, h_ld=(1 << 22) + 1, w_ld=(1 << 22) + 1), RANGE),
    (dict(vocab=1 << 22, size=1 << 13, h_ld=1 << 13, w_ld=1 << 13), RANGE), (dict(w_ld=(1 << 22) + 8), RANGE),
    (dict(h=P + 1), ALIGN), (dict(w=P + 1), ALIGN), (dict(targets=P + 4), ALIGN), (dict(loss=P + 2), ALIGN),
    (dict(lse=P + 1), ALIGN), (dict(ws=P + 64), ALIGN),
]
GRAD_REFUSED = REFUSED + [
    (dict(grad=0), INVALID), (dict(dh=0), INVALID), (dict(dw=0), INVALID), (dict(dtype=5), INVALID),
    (dict(acc=2), INVALID), (dict(acc=-1), INVALID), (dict(grad=P + 2), ALIGN), (dict(dh=P + 1), ALIGN),
    (dict(dw=P + 2, dtype=1), ALIGN),
]


@pytest.mark.parametrize("change,status", REFUSED)
def test_loss_refusals(tide, change, status):
    a = {**CALL, **change}
    got = tide.lib.tide_vocab_loss(a["h"] or None, a["h_ld"], a["w"] or None, a["w_ld"], a["targets"] or None,
                                   a["tokens"], a["size"], a["vocab"], a["loss"] or None, a["lse"], a["ws"] or None,
                                   a["ws_bytes"], None)
    assert got == status and tide.lib.tide_last_error()


@pytest.mark.parametrize("change,status", GRAD_REFUSED)
def test_gradient_refusals(tide, change, status):
    a = {**CALL, **change}
    got = tide.lib.tide_vocab_loss_grad(a["h"] or None, a["h_ld"], a["w"] or None, a["w_ld"], a["targets"] or None,
                                        a["grad"] or None, a["tokens"], a["size"], a["vocab"], a["loss"] or None,
                                        a["lse"], a["dh"] or None, a["dw"] or None, a["dtype"], a["acc"],
                                        a["ws"] or None, a["ws_bytes"], None)
    assert got == status and tide.lib.tide_last_error()


def test_no_tokens(tide):
    # nothing to do: no pointers are needed (but dweight's, which stays)
    assert tide.lib.tide_vocab_loss(None, 64, None, 64, None, 0, 64, 100, None, None, None, 0, None) == 0
    assert tide.lib.tide_vocab_loss_grad(None, 64, None, 64, None, None, 0, 64, 100, None, None, None, P, 0, 1, None, 0,
                                         None) == 0


def test_workspace(tide):
    need = ctypes.c_int64(-1)

    def size(h=P, h_ld=4096, w=P, w_ld=4096, tokens=4096, hidden=4096, vocab=128000, grad=1, dtype=0):
        st = tide.lib.tide_vocab_loss_workspace(h, h_ld, w, w_ld, tokens, hidden, vocab, grad, dtype,
                                                ctypes.byref(need))
        return need.value if st == 0 else st

    assert size(grad=2) == INVALID and size(dtype=9) == INVALID and size(h_ld=100) == INVALID
    step = size()
    # the exponentials of 4096 tokens, the tokens' states, and the partial sums of at most three rounds of 256 split
    # tiles (65536 fp32 sums each: 192 MiB), little else (500 pairs of statistics a token: 15.6 MiB)
    assert 4096 * 128000 * 2 < step < 4096 * 128000 * 2 + 4096 * 4096 * 2 + (192 << 20) + (16 << 20)
    # more tokens than 2 GiB of exponentials hold: in pieces, with dweight's sums in fp32 unless dweight holds them
    assert size(tokens=65536, dtype=1) < (2 << 30) + (1 << 30)
    assert size(tokens=65536, dtype=0) - size(tokens=65536, dtype=1) == 128000 * 4096 * 4
    # a weight whose rows are not all on 16 bytes is copied
    assert size(w_ld=4097) - step == 128000 * 4096 * 2
    assert size(w=P + 2) - step == 128000 * 4096 * 2
    # a loss keeps no exponentials; a few tokens neither states
    assert size(grad=0) < 128 << 20
    assert size(grad=0, tokens=17) < 1 << 20
    assert size(tokens=0) == 0


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(5)
    h, w = rng.standard_normal((6, 9)), rng.standard_normal((21, 9))
    t = np.array([0, 20, 7, -100, 21, 7])
    g = rng.standard_normal(6)
    got = ref.vocab_loss(h, w, t, g)

    def f(h, w):
        return (ref.vocab_loss(h, w, t)["loss"][0] * g).sum()

    for name, x, at in (("dhidden", h, lambda d: f(h + d, w) - f(h - d, w)),
                        ("dweight", w, lambda d: f(h, w + d) - f(h, w - d))):
        for i in np.ndindex(x.shape):
            d = np.zeros_like(x)
            d[i] = 1e-5
            assert abs(at(d) / 2e-5 - got[name][0][i]) < 1e-8
