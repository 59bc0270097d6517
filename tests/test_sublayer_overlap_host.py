"""Calls of the sublayer's operators with an output that shares memory with an
input or another output are refused before any device work (no GPU: the addresses
passed here are not device memory)."""
import ctypes
import random

import pytest

INVALID = -1
STEP = 1 << 32  # from one argument's address to the next: no two meet


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


def addresses(*names):
    return {n: STEP * (k + 1) for k, n in enumerate(names)}


ROWS, COLS, FFN = 300, 64, 96
NORM = addresses("x", "w", "b", "out", "mean", "rstd")
NORM_GRAD = addresses("dout", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws")
BLOCK = addresses("x", "wg", "wu", "out", "gates", "ws")
BLOCK_GRAD = addresses("dout", "x", "wg", "wu", "gates", "dx", "dwg", "dwu", "ws")
# bytes of each: bf16 matrices, fp32 vectors and weights' gradients
BYTES = {**{n: 2 * ROWS * COLS for n in ("x", "dx")}, **{n: 4 * COLS for n in ("w", "b", "dw", "db")},
         **{n: 4 * ROWS for n in ("mean", "rstd")}}
BLOCK_BYTES = {**{n: 2 * ROWS * FFN for n in ("out", "dout")}, **{n: 2 * COLS * FFN for n in ("wg", "wu")}, "gates": 4 * ROWS * FFN,
               **{n: 2 * ROWS * COLS for n in ("x", "dx")}, **{n: 4 * COLS * FFN for n in ("dwg", "dwu")}}


def norm(tide, a):
    return tide.lib.tide_layer_norm(a["x"], 0, COLS, ROWS, COLS, a["w"], a["b"], 1, 1e-5, a["out"], 0, COLS, a["mean"], a["rstd"],
                                    None)


def norm_grad(tide, a):
    return tide.lib.tide_layer_norm_grad(a["dout"], 0, COLS, a["x"], 0, COLS, ROWS, COLS, a["w"], 1, a["mean"], a["rstd"], a["dx"],
                                         COLS, a["dw"], a["db"], 0, a["ws"], 1 << 30, None)


def block(tide, a):
    return tide.lib.tide_gated_block(a["x"], COLS, a["wg"], COLS, a["wu"], COLS, ROWS, COLS, FFN, 0, a["out"], FFN, a["gates"],
                                     2 * FFN, a["ws"], 1 << 40, None)


def block_grad(tide, a):
    return tide.lib.tide_gated_block_grad(a["dout"], FFN, a["x"], COLS, a["wg"], COLS, a["wu"], COLS, ROWS, COLS, FFN, 0, a["gates"],
                                          2 * FFN, a["dx"], COLS, a["dwg"], a["dwu"], 1, 0, a["ws"], 1 << 40, None)


def pairs(outs, args):
    """Every output with every other argument (but the workspace)."""
    return [(o, n) for o in outs for n in args if n not in (o, "ws")]


CASES = [(norm, NORM, {**BYTES, "out": BYTES["x"]}, o, n) for o, n in pairs(("out", "mean", "rstd"), NORM)]
CASES += [(norm_grad, NORM_GRAD, {**BYTES, "dout": BYTES["x"]}, o, n) for o, n in pairs(("dx", "dw", "db"), NORM_GRAD)]
CASES += [(block, BLOCK, BLOCK_BYTES, o, n) for o, n in pairs(("out", "gates"), BLOCK)]
CASES += [(block_grad, BLOCK_GRAD, BLOCK_BYTES, o, n) for o, n in pairs(("dx", "dwg", "dwu"), BLOCK_GRAD)]


@pytest.mark.parametrize("call,args,nbytes,out,other", CASES, ids=[f"{c[0].__name__}-{c[3]}-{c[4]}" for c in CASES])
def test_an_output_over_another_argument(tide, call, args, nbytes, out, other):
    """At the same address, over the other's end and over its start."""
    for at in (args[other], args[other] + nbytes[other] - 4, args[other] - nbytes[out] + 4):
        assert call(tide, {**args, out: at}) == INVALID, hex(at)
        message = tide.lib.tide_last_error()
        assert b"overlaps" in message or (at == args[other] and b"are the same" in message)


def test_columns_of_one_buffer(tide):
    """Rows of equal pitch: an output's columns that reach into another's."""
    for at in (1, COLS - 1, 200 - 1, 199 + 200):  # into x's row, and from one of its rows into the next
        got = tide.lib.tide_layer_norm(STEP, 0, 200, ROWS, COLS, None, None, 1, 1e-5, STEP + 2 * at, 0, 200, None, None, None)
        assert got == INVALID and b"overlaps" in tide.lib.tide_last_error(), at


def orthogonalize(tide, x, xt, x_ld, out, out_ld, rows, cols):
    two = ctypes.c_void_p * 2
    # with a workspace that is too small: the next check
    got = tide.lib.tide_orthogonalize(two(*x), xt, x_ld, two(*out), out_ld, 2, rows, cols, 5, 3.4445, -4.775, 2.0315, 1e-7, 1 << 40,
                                      0, None)
    assert got == INVALID
    return tide.lib.tide_last_error()


def test_areas_against_their_bytes(tide):
    """Two matrices and their updates in a small space, against the bytes that each
    holds: refused if they share one, and only then (of different row pitches with
    gaps, if they start together)."""
    rng = random.Random(1)

    def held(p, ld, size):
        return {p + size * (r * ld + c) + k for r in range(rows) for c in range(cols) for k in range(size)}

    seen = {True: 0, False: 0}
    for _ in range(6000):
        rows, cols, xt = rng.randint(1, 4), rng.randint(1, 5), rng.randint(0, 1)
        size = 4 if xt else 2
        x_ld, out_ld = (cols + rng.choice((0, 0, 1, 3, 8)) for _ in range(2))
        if rng.random() < 0.4 and x_ld * size // 2 >= cols:
            out_ld = x_ld * size // 2  # of equal pitch in bytes
        space = rng.choice((80, 200))
        x = [4096 + size * rng.randrange(space) for _ in range(2)]
        out = [4096 + 2 * rng.randrange(2 * space) for _ in range(2)]
        hx, ho = ([held(p, ld, s) for p in at] for at, ld, s in ((x, x_ld, size), (out, out_ld, 2)))
        known = rows == 1 or x_ld == cols or out_ld == cols or x_ld * size == out_ld * 2
        shared = bool(ho[0] & ho[1]) or any(hx[i] & ho[1 - i] and (known or x[i] == out[1 - i]) for i in range(2))
        message = orthogonalize(tide, x, xt, x_ld, out, out_ld, rows, cols)
        assert (b"workspace" not in message) == shared, (rows, cols, xt, x, x_ld, out, out_ld, message)
        seen[shared] += 1
    assert min(seen.values()) > 1000
