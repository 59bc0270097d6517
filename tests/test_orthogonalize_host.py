"""Host-side checks of the orthogonalized updates (no GPU): every refusal, made
before any device work (the addresses passed here are not device memory), the
workspace, the 64-bit reference against the singular value decomposition, and
what the kernels' roundings cost."""
import ctypes

import numpy as np
import pytest

from tests import sublayer_reference as ref

INVALID, RANGE, ALIGN = -1, -2, -3
P = 0x10000  # an aligned address that nothing reads
ABC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


CALL = dict(x=[P, 2 * P], xt=0, x_ld=64, out=[3 * P, 4 * P], out_ld=64, count=2, rows=40, cols=64, steps=5, abc=ABC, eps=1e-7,
            ws=P, ws_bytes=1 << 40)
WIDE = (1 << 22) + 1
REFUSED = [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=[P, 0]), INVALID), (dict(out=[0, P]), INVALID),
    (dict(count=-1), INVALID), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(x_ld=63), INVALID),
    (dict(out_ld=63), INVALID), (dict(xt=2), INVALID), (dict(steps=0), INVALID), (dict(steps=65), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(ws=0), INVALID), (dict(ws_bytes=1 << 10), INVALID),
    (dict(out=[3 * P, 3 * P]), INVALID), (dict(out=[2 * P, 4 * P]), INVALID), (dict(out=[3 * P, P]), INVALID),
    # operands that leave fp16's range: the polynomial's, the iterate's at once, the iterate's after some steps
    (dict(abc=(20.0, 0.0, 0.0)), INVALID), (dict(abc=(1.0, 20.0, -20.0)), INVALID), (dict(abc=(4.0, 0.0, 0.0)), INVALID),
    (dict(abc=(1.5, 0.0, 0.0), steps=8), INVALID), (dict(abc=(float("nan"), 0.0, 0.0)), INVALID),
    (dict(abc=(1.0, float("inf"), 0.0)), INVALID), (dict(abc=(5.0, -4.775, 2.0315)), INVALID),
    (dict(cols=WIDE, x_ld=WIDE, out_ld=WIDE), RANGE), (dict(rows=WIDE), RANGE), (dict(x_ld=WIDE), RANGE),
    (dict(rows=1 << 18, cols=1 << 18, x_ld=1 << 18, out_ld=1 << 18), RANGE), (dict(ws=P + 64), ALIGN),
    (dict(x=[P, 2 * P + 1]), ALIGN), (dict(xt=1, x=[P + 2, 2 * P]), ALIGN), (dict(out=[3 * P + 1, 4 * P]), ALIGN),
]


def call(tide, a):
    def array(v):
        return None if v is None else (ctypes.c_void_p * 2)(*[p or None for p in v])

    return tide.lib.tide_orthogonalize(array(a["x"]), a["xt"], a["x_ld"], array(a["out"]), a["out_ld"], a["count"], a["rows"],
                                       a["cols"], a["steps"], *a["abc"], a["eps"], a["ws"] or None, a["ws_bytes"], None)


@pytest.mark.parametrize("change,status", REFUSED)
def test_refusals(tide, change, status):
    assert call(tide, {**CALL, **change}) == status and tide.lib.tide_last_error()


def test_nothing_to_do(tide):
    none = dict(x=None, out=None, ws=0)
    for size in (dict(count=0), dict(rows=0), dict(cols=0)):
        assert call(tide, {**CALL, **none, **size}) == 0


# the classical third and fifth order polynomials, and ones that are only just in range
@pytest.mark.parametrize("abc,steps", [((1.5, -0.5, 0.0), 30), ((1.875, -1.25, 0.375), 30), (ABC, 64), ((3.7, 0.0, 0.0), 1),
                                       ((0.0, 0.0, 0.0), 5), ((-1.0, 0.0, 0.0), 9)])
def test_coefficients_that_are_taken(tide, abc, steps):
    # with a workspace that is too small: the next check
    assert call(tide, {**CALL, "abc": abc, "steps": steps, "ws_bytes": 0}) == INVALID
    assert b"workspace" in tide.lib.tide_last_error()


def test_workspace(tide):
    need = ctypes.c_int64(-1)

    def size(count=1, rows=4096, cols=14336, steps=5):
        st = tide.lib.tide_orthogonalize_workspace(count, rows, cols, steps, ctypes.byref(need))
        return need.value if st == 0 else st

    assert size(steps=0) == INVALID and size(rows=-1) == INVALID and size(rows=WIDE) == RANGE
    assert size(count=0) == size(rows=0) == size(cols=0) == 0
    # X twice and the rest of its rounding, G and P, all in 16 bits; partial sums of at most three rounds of 256 tiles
    x = 3 * 4096 * 14336 * 2 + 2 * 4096 * 4096 * 2
    assert x < size() < x + 3 * 256 * 65536 * 4 + (1 << 20)
    assert size() == size(rows=14336, cols=4096)
    # many matrices: about 1 GiB of them at a time
    assert size(count=128, rows=768, cols=2048) < (1 << 30) + 3 * 256 * 65536 * 4 + (1 << 20)
    assert size(count=5000, rows=8, cols=8) < 1 << 24


def matrix(rng, m, n, kind):
    x = rng.standard_normal((m, n))
    if kind == "strong":  # a few directions hold most of it
        r = min(6, m, n)
        x += (rng.standard_normal((m, r)) * np.logspace(2, 0, r)) @ rng.standard_normal((r, n))
    return x * 1e-3


@pytest.mark.parametrize("kind", ["noise", "strong"])
@pytest.mark.parametrize("m,n", [(5, 9), (9, 5), (24, 24), (1, 7)])
def test_reference(m, n, kind):
    """Against the singular value decomposition."""
    x = matrix(np.random.default_rng(m), m, n, kind)
    u, s, v = np.linalg.svd(x, full_matrices=False)
    s = s / (np.sqrt((x**2).sum()) + 1e-7)
    for _ in range(5):
        s = s * (ABC[0] + ABC[1] * s**2 + ABC[2] * s**4)
    assert np.allclose(ref.orthogonalize(x, 5, *ABC, 1e-7)[0], (u * s) @ v, atol=1e-9)


@pytest.mark.parametrize("kind,most", [("noise", 0.002), ("strong", 0.01)])
@pytest.mark.parametrize("m,n", [(40, 40), (60, 200), (200, 60), (300, 300)])
def test_the_roundings(m, n, kind, most):
    """The kernels' roundings, on the CPU, cost 0.2% of the result in the 2-norm at
    most, 1% where a few directions hold almost all of the matrix; without the second
    fp16 of a X they cost more there."""
    x = matrix(np.random.default_rng(m + n), m, n, kind)

    def error(exact):
        value, tolerance = ref.orthogonalize(x, 5, *ABC, 1e-7, exact)
        return (tolerance / 1.5 / np.linalg.norm(value)) - 2.0**-8 / np.sqrt(3)

    assert error(3) < most
    if kind == "strong":
        assert error(0) > 1.5 * error(3)
