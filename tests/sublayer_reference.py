"""64-bit references of the sublayer's operators (layer norm, the gated block,
orthogonalised updates), for the tests: numpy on the CPU, from the definitions
in include/tide.h, each with a bound of the kernels' error before the result is
rounded to its own type."""
import numpy as np

U32 = 2.0**-24  # half a step of fp32: a rounding's relative error
HALF = {"bf16": 2.0**-8, "f32": 2.0**-24, "f16": 2.0**-11}
TINY = {"bf16": 2.0**-134, "f32": 2.0**-150}  # half a step below the normal numbers


def rounded(value, err, dtype):
    """The bound after one rounding to `dtype`."""
    return err + HALF[dtype] * (np.abs(value) + err) + TINY[dtype]


def row_adds(n):
    """Additions a value of a row of n goes through: a thread's own (at most 16
    values, or n / 1024 where rows are read by loops of 1024 threads), six steps
    of a wave and at most 16 waves' sums, and two more for the division."""
    return max(16, -(-n // 1024) + 4) + 6 + 16 + 2


def layer_norm(x, w, b, eps):
    """{name: (value, bound)} of out, mean and rstd for float64 x (rows x n), w
    and b.

    The bounds are those of sums in fp32 throughout whose mean is corrected by the
    mean of what it leaves; sums in fp64 stay within them.  A mean is rounded once,
    whatever its sum lost: what is left of it, off, is taken back.  v = x - mean is
    rounded by U32 of itself, off is a mean of n of them and differs from theirs by
    K + 1 roundings of the mean magnitude, and x - mean - off is rounded again.  The
    squares' mean carries 3 + K of them, rstd half of those and four more (eps, the
    root, the division, each counted twice for routines that are off by a whole
    step).  The factor 1.01 stands for products of these errors."""
    n = x.shape[1]
    K = row_adds(n)
    mean = x.mean(-1, keepdims=True)
    d = x - mean
    var = (d * d).mean(-1, keepdims=True)
    # the mean as first rounded is off by at most this, and so are the v
    first = (K + 1) * U32 * np.abs(x).mean(-1, keepdims=True)
    v = np.abs(d) + first
    e_off = (K + 2) * U32 * v.mean(-1, keepdims=True)
    e_mean = e_off + U32 * (np.abs(mean) + e_off)
    e_num = 3 * U32 * v + e_off
    squares = (v * v).mean(-1, keepdims=True)
    e_var = (K + 4) * U32 * squares + 2 * (K + 4) * U32 * first**2 + 2 * first * e_off
    rstd = 1 / np.sqrt(var + eps)
    rel = e_var / (var + eps) / 2 * (1 + 2 * e_var / (var + eps)) + 8 * U32
    xh = d * rstd
    out = xh * w + b
    e = 1.01 * (np.abs(w) * (rstd * e_num * (1 + rel) + np.abs(xh) * (rel + 3 * U32)) + 2 * U32 * (np.abs(xh * w) + np.abs(b)))
    return {"out": (out, e), "mean": (mean[:, 0], 1.01 * e_mean[:, 0]), "rstd": (rstd[:, 0], 1.01 * (rel * rstd)[:, 0])}


def layer_norm_grad(dy, x, w, mean, rstd, old_dw=None, old_db=None):
    """{name: (value, bound)} of dx, dweight and dbias from the mean and rstd that
    are given (float64 of fp32 values).

    xh carries 2 roundings, g 1, their row sums K more; dx's four operations one
    each.  A column's sum goes through at most rows / 256 + 150 additions: a
    thread's rows (256 workgroups at least where there are that many rows), 4
    waves', a 16th of at most 2048 workgroups', 16 shares."""
    rows, n = x.shape
    K = row_adds(n)
    mean, rstd = mean[:, None], rstd[:, None]
    xh = (x - mean) * rstd
    g = dy * w
    s, sx = g.mean(-1, keepdims=True), (g * xh).mean(-1, keepdims=True)
    ma, mx = np.abs(g).mean(-1, keepdims=True), np.abs(g * xh).mean(-1, keepdims=True)
    dx = rstd * (g - s - xh * sx)
    mag = np.abs(g) + np.abs(s) + np.abs(xh * sx)
    e = rstd * (U32 * np.abs(g) + (K + 2) * U32 * ma + np.abs(xh) * (K + 6) * U32 * mx + 3 * U32 * np.abs(xh * sx) + 4 * U32 * mag)
    L = rows / 256 + 150
    dw, db = (dy * xh).sum(0), dy.sum(0)
    e_dw, e_db = (L + 4) * U32 * np.abs(dy * xh).sum(0), (L + 1) * U32 * np.abs(dy).sum(0)
    if old_dw is not None:
        dw, db = dw + old_dw, db + old_db
        e_dw, e_db = e_dw + U32 * np.abs(dw), e_db + U32 * np.abs(db)
    return {"dx": (dx, 1.01 * e), "dweight": (dw, 1.01 * e_dw), "dbias": (db, 1.01 * e_db)}

EXACT_SUM = 2.0**-23  # of the magnitudes, per addition of an adder that may truncate


def act(z, name):
    """(value, derivative, the sigmoid's argument) in float64."""
    if name == "silu":
        k, dk = z, np.ones_like(z)
    else:
        c = 2 * np.sqrt(2 / np.pi)
        k, dk = c * (z + 0.044715 * z**3), c * (1 + 3 * 0.044715 * z**2)
    e = np.exp(-np.abs(k))
    s = np.where(k >= 0, 1, e) / (1 + e)
    return z * s, s + z * dk * e / (1 + e) ** 2, k


def _activated(z, ez, name):
    """(value, bound, derivative, bound) of the activation of z that is off by ez.

    The slopes of both activations are below 1.13 and their second derivatives
    below 0.8.  The sigmoid's argument is rounded at most 7 times (GELU's cubic,
    the constant log2 e), which an exponential multiplies by |k|; the exponential,
    the reciprocal and the operations around them are off by 2^-23 each, at most
    8 of them.  Exponentials below 2^-126 may be flushed."""
    a, d, k = act(z, name)
    rel = (4 * np.abs(k) + 10) * EXACT_SUM
    s, flush = np.abs(a / np.where(z == 0, 1, z)) + (z == 0) * 0.5, 2.0**-125 * (1 + np.abs(z))
    ea = 1.13 * ez + np.abs(a) * rel + flush
    return a, ea, d, 0.8 * ez + rel * (s + np.abs(d - np.where(z == 0, 0.5, a / np.where(z == 0, 1, z)))) + flush


def _gates(x, wg, wu):
    n = (x.shape[1] + 64) * EXACT_SUM
    return x @ wg.T, n * (np.abs(x) @ np.abs(wg).T), x @ wu.T, n * (np.abs(x) @ np.abs(wu).T)


def gated_block(x, wg, wu, name):
    """{name: (value, bound)} of out and gates for float64 x, wg and wu: sums of
    hidden exact products, the activation, and one more rounding of the product."""
    g, eg, u, eu = _gates(x, wg, wu)
    a, ea, _, _ = _activated(g, eg, name)
    eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu + 2 * U32 * np.abs(a * u)
    return {"out": (a * u, eh), "gates": (np.concatenate([g, u], 1), np.concatenate([eg, eu], 1))}


def gated_block_grad(dout, x, wg, wu, name, gates=None, old=None):
    """{name: (value, bound, rms)} of dx, dw_gate and dw_up: bounds before the
    result's own rounding, and of the root mean square of the whole error of a bf16
    result.  gates: the values that were kept, which are then exact.

    dg and du are rounded to bf16 once; the sums add at most K products and 64
    partial sums.  For the root mean square those roundings and the result's are
    taken as independent and uniform in their half steps, 1.5 times, and to it the
    bound of everything else."""
    f = wg.shape[0]
    if gates is None:
        g, eg, u, eu = _gates(x, wg, wu)
    else:
        g, u = gates[:, :f], gates[:, f:]
        eg = eu = np.zeros_like(g)
    a, ea, d, ed = _activated(g, eg, name)
    dh = np.abs(dout)
    dg, du = dout * u * d, dout * a
    arith = [dh * (np.abs(u) * ed + np.abs(d) * eu + ed * eu) + 3 * U32 * np.abs(dg), dh * ea + 2 * U32 * np.abs(du)]
    err = [rounded(v, e, "bf16") for v, e in zip((dg, du), arith)]
    out = {}
    half = HALF["bf16"]

    def product(name, pairs, old=None):
        value = sum(p @ b for p, _, _, b in pairs)
        k = sum(b.shape[0] for _, _, _, b in pairs)
        sums = (k + 64) * EXACT_SUM * sum((np.abs(p) + e) @ np.abs(b) for p, e, _, b in pairs)
        var = half**2 / 3 * sum((p**2) @ (b**2) for p, _, _, b in pairs)
        rest = sum(ar @ np.abs(b) for _, _, ar, b in pairs) + sums
        bound = sum(e @ np.abs(b) for _, e, _, b in pairs) + sums
        if old is not None:
            value = value + old
            bound, rest = bound + U32 * np.abs(value), rest + U32 * np.abs(value)
        rms = 1.5 * np.sqrt((var + half**2 / 3 * value**2).sum()) + np.sqrt((rest**2).sum())
        out[name] = (value, bound, rms)

    product("dx", [(dg, err[0], arith[0], wg), (du, err[1], arith[1], wu)])
    product("dw_gate", [(dg.T, err[0].T, arith[0].T, x)], None if old is None else old[0])
    product("dw_up", [(du.T, err[1].T, arith[1].T, x)], None if old is None else old[1])
    return out


def _f16(t):
    """The value that fp16 keeps of t times 2^12."""
    with np.errstate(over="ignore"):
        return (t * 4096).astype(np.float16).astype(np.float64) / 4096


def newton_schulz(x, steps, a, b, c, eps):
    """The definition, in float64."""
    x = x / (np.sqrt((x**2).sum()) + eps)
    for _ in range(steps):
        g = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        p = b * g + c * (g @ g)
        x = a * x + (p @ x if x.shape[0] <= x.shape[1] else x @ p)
    return x


def orthogonalize(x, steps, a, b, c, eps, exact=3, f32=True):
    """(value, tolerance of the error's Frobenius norm after the rounding to bf16) of
    a float64 matrix.

    A bound that takes every rounding at its worst and in the worst direction is of
    no use here: a step multiplies by up to 3.5 what lies in the weak directions.
    The tolerance is the error of the definition with the kernels' roundings put in
    where they are (X, G and the polynomial to fp16 times 2^12; in the first `exact`
    steps a times the rest of X's rounding, to 11 bits, is added; a bf16 matrix has
    none in the first), 1.5 times, since the kernels' own fp32 sums let some
    values round the other way: as many roundings of the same sizes in other
    directions, not more or larger ones (the sums' own errors are 2^-13 of them).
    To it comes 1.5 times the root mean square of the result's rounding."""
    value = newton_schulz(x, steps, a, b, c, eps)
    tall = x.shape[0] > x.shape[1]
    y = x.T if tall else x
    y = y / (np.sqrt((y**2).sum()) + eps)
    for k in range(steps):
        h = _f16(y) if k > 0 or f32 else y
        g = _f16(h @ h.T)
        y = _f16(b * g + c * (g @ g) + a * np.eye(len(g))) @ h + (a * _f16((y - h) * 2048) / 2048 if k < exact else 0)
    err = np.linalg.norm((y.T if tall else y) - value)
    return value, 1.5 * (err + HALF["bf16"] / np.sqrt(3) * np.linalg.norm(value)) + 2.0**-20 * np.linalg.norm(value)
