"""Host-side checks of layer norm (no GPU): every refusal, made before any
device work (the addresses passed here are not device memory), and the 64-bit
reference against differences."""
import ctypes

import numpy as np
import pytest

from tests import sublayer_reference as ref

INVALID, RANGE, ALIGN = -1, -2, -3
P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


CALL = dict(x=P, xt=0, x_ld=64, rows=10, cols=64, w=P, b=P, at=1, eps=1e-5, out=P, yt=0, y_ld=64, mean=P, rstd=P)
REFUSED = [
    (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=-1), INVALID), (dict(x_ld=63), INVALID), (dict(y_ld=63), INVALID), (dict(xt=2), INVALID),
    (dict(yt=-1), INVALID), (dict(at=7), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(rows=1 << 31), RANGE), (dict(cols=(1 << 22) + 1, x_ld=(1 << 22) + 1, y_ld=(1 << 22) + 1), RANGE),
    (dict(rows=1 << 29), RANGE), (dict(x_ld=(1 << 22) + 1), RANGE), (dict(x=P + 1), ALIGN), (dict(x=P + 2, xt=1), ALIGN),
    (dict(out=P + 1), ALIGN), (dict(out=P + 2, yt=1), ALIGN), (dict(w=P + 2), ALIGN), (dict(b=P + 2), ALIGN),
    (dict(w=P + 1, at=0), ALIGN), (dict(mean=P + 2), ALIGN), (dict(rstd=P + 1), ALIGN),
]
GRAD = dict(dy=P, yt=0, y_ld=64, x=P, xt=0, x_ld=64, rows=10, cols=64, w=P, at=1, mean=P, rstd=P, dx=P, dx_ld=64, dw=P, db=P,
            acc=0, ws=P, ws_bytes=1 << 30)
GRAD_REFUSED = [(c, s) for c, s in REFUSED if not set(c) & {"out", "b", "eps"}] + [
    (dict(dy=0), INVALID), (dict(mean=0), INVALID), (dict(rstd=0), INVALID), (dict(dx=0), INVALID), (dict(dx_ld=63), INVALID),
    (dict(acc=2), INVALID), (dict(acc=-1), INVALID), (dict(ws=0), INVALID), (dict(ws_bytes=16), INVALID),
    (dict(ws=P + 16), ALIGN), (dict(dw=P + 2), ALIGN), (dict(db=P + 2), ALIGN), (dict(dx=P + 1), ALIGN),
    (dict(dy=P + 1), ALIGN), (dict(dy=P + 2, yt=1), ALIGN),
]


@pytest.mark.parametrize("change,status", REFUSED)
def test_refusals(tide, change, status):
    a = {**CALL, **change}
    got = tide.lib.tide_layer_norm(a["x"] or None, a["xt"], a["x_ld"], a["rows"], a["cols"], a["w"], a["b"], a["at"],
                                   a["eps"], a["out"] or None, a["yt"], a["y_ld"], a["mean"], a["rstd"], None)
    assert got == status and tide.lib.tide_last_error()


@pytest.mark.parametrize("change,status", GRAD_REFUSED)
def test_gradient_refusals(tide, change, status):
    a = {**GRAD, **change}
    got = tide.lib.tide_layer_norm_grad(a["dy"] or None, a["yt"], a["y_ld"], a["x"] or None, a["xt"], a["x_ld"], a["rows"],
                                        a["cols"], a["w"], a["at"], a["mean"] or None, a["rstd"] or None, a["dx"] or None,
                                        a["dx_ld"], a["dw"], a["db"], a["acc"], a["ws"] or None, a["ws_bytes"], None)
    assert got == status and tide.lib.tide_last_error()


def test_no_rows(tide):
    # nothing to do: no pointers are needed
    assert tide.lib.tide_layer_norm(None, 0, 64, 0, 64, None, None, 0, 1e-5, None, 0, 64, None, None, None) == 0
    assert tide.lib.tide_layer_norm_grad(None, 0, 64, None, 0, 64, 0, 64, None, 0, None, None, None, 64, None, None, 0,
                                         None, 0, None) == 0


def test_workspace(tide):
    need = ctypes.c_int64(-1)

    def size(xt=0, yt=0, rows=4096, cols=4096):
        st = tide.lib.tide_layer_norm_grad_workspace(xt, yt, rows, cols, ctypes.byref(need))
        return need.value if st == 0 else st

    assert size(xt=3) == INVALID and size(yt=3) == INVALID and size(cols=0) == INVALID and size(rows=-1) == INVALID
    assert size(rows=1 << 31) == RANGE
    assert size(rows=0) == 0
    # two fp32 sums a column for each workgroup, of which there are at most 2048 and no more than rows
    assert size(rows=1) == 2 * 4 * 4096
    assert 0 < size() <= 2048 * 2 * 4 * 4096
    assert size(rows=1 << 20) <= 2048 * 2 * 4 * 4096
    assert size(cols=1 << 22, rows=64) == 64 * 2 * 4 << 22


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(5)
    rows, n, eps = 3, 7, 1e-3
    x, dy, w, b = rng.standard_normal((rows, n)), rng.standard_normal((rows, n)), rng.standard_normal(n), rng.standard_normal(n)
    fwd = ref.layer_norm(x, w, b, eps)
    got = ref.layer_norm_grad(dy, x, w, fwd["mean"][0], fwd["rstd"][0])

    def f(x, w, b):
        return (ref.layer_norm(x, w, b, eps)["out"][0] * dy).sum()

    for name, t, at in (("dx", x, lambda d: f(x + d, w, b) - f(x - d, w, b)),
                        ("dweight", w, lambda d: f(x, w + d, b) - f(x, w - d, b)),
                        ("dbias", b, lambda d: f(x, w, b + d) - f(x, w, b - d))):
        for i in np.ndindex(t.shape):
            d = np.zeros_like(t)
            d[i] = 1e-5
            assert abs(at(d) / 2e-5 - got[name][0][i]) < 1e-8
