"""64-bit references of the training-step operators, for the tests: numpy on
the CPU, from the definitions in include/tide.h."""
import numpy as np

BLOCK = 32
LIMIT = {"e4m3": 448.0, "int8": 127.5}
TOP = {"e4m3": 448.0, "int8": 127.0}
HIGHEST = {"e4m3": 246, "int8": 248}
LOWEST = 10


def e4m3_values():
    """The values of the codes 0..126 (127 is NaN)."""
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f * 2.0**-9, (1 + f / 8) * 2.0 ** (e - 7.0))


def pack(x, fmt):
    """(codes as uint8 bit patterns, scale bytes) of a float64 matrix."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = np.zeros((rows, nb * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, nb, BLOCK)
    amax = np.abs(v).max(-1, initial=0.0)
    finite = np.isfinite(v).all(-1)
    amax = np.where(finite, amax, 1.0)
    # the smallest exponent whose unit holds the block, found by trying all
    bytes_ = np.arange(LOWEST, HIGHEST[fmt] + 1)
    fits = amax[..., None] <= LIMIT[fmt] * 2.0 ** (bytes_ - 127.0)
    b = np.where(fits.any(-1), bytes_[np.argmax(fits, -1)], HIGHEST[fmt])
    y = np.clip(np.where(finite[..., None], v, 0.0) / 2.0 ** (b - 127.0)[..., None], -TOP[fmt], TOP[fmt])
    if fmt == "int8":
        codes = np.rint(y).astype(np.int8).view(np.uint8)
        codes = np.where(finite[..., None], codes, 0)
    else:
        table = e4m3_values()
        hi = np.searchsorted(table, np.abs(y)).clip(1, 126)
        lo = hi - 1
        dl, dh = np.abs(y) - table[lo], table[hi] - np.abs(y)
        code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        codes = code | (np.signbit(y).astype(np.int64) << 7)
        codes = np.where(finite[..., None], codes, 0x7F)
    return codes.reshape(rows, nb * BLOCK).astype(np.uint8), np.where(finite, b, 255).astype(np.uint8)


def unpack(codes, scales, fmt, cols):
    """float64 values of codes (uint8 bit patterns) and scale bytes."""
    if fmt == "int8":
        q = codes.view(np.int8).astype(np.float64)
    else:
        q = np.append(e4m3_values(), np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    u = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    rows, nb = scales.shape
    return (q.reshape(rows, nb, BLOCK) * u[..., None]).reshape(rows, nb * BLOCK)[:, :cols]


def weight_grad(dy, x, alpha=1.0, old=None):
    """(the gradient, the bound of its error before it is rounded to the
    gradient's type) of float64 dy and x.  The products are exact in fp32 and T
    of them are added, in any order and starting from 0, and at most 64 partial
    sums joined: each addition is off by at most 2^-23 of the magnitudes so
    far (2^-24 for a rounding adder, 2^-23 for one that truncates); alpha and
    the old value add one rounding each."""
    s, mag = dy.T @ x, np.abs(dy).T @ np.abs(x)
    r = alpha * s + (0.0 if old is None else old)
    err = abs(alpha) * (dy.shape[0] + 64) * 2.0**-23 * mag + 2.0**-23 * (np.abs(alpha * s) + np.abs(r))
    return r, err


def vocab_loss(h, w, targets, grad_loss=None):
    """The loss of float64 h and w and, with grad_loss, its gradients, each
    with a bound of the kernels' error before the result is rounded to its own
    type, as a dict of (value, bound) pairs.

    A logit is a sum of d exact products, each addition off by at most 2^-23 of
    the magnitudes (a truncating adder).  An exponential's argument z - m is
    rounded three times (the difference, the constant log2(e), the product) and
    the exponential itself by 2^-23; a tile's exponentials meet at most 128
    additions of 2^-24 on their way to the row's sum, and a second exponential
    joins the tile.  r is the row's range of logits.  dz's entries are
    additionally rounded to fp16 times 2^15 (2^-11 relative, or 2^-40 of the
    tile's largest) and once to bf16 (2^-8); the target's from expm1 instead."""
    tokens, vocab = h.shape[0], w.shape[0]
    keep = (targets >= 0) & (targets < vocab)
    at = np.where(keep, targets, 0)
    rows = np.arange(tokens)
    h = np.where(keep[:, None], h, 0.0)
    z = h @ w.T
    ez = (h.shape[1] + 8) * 2.0**-23 * (np.abs(h) @ np.abs(w).T)
    m = z.max(-1)
    r = m - z.min(-1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(-1))
    e_exp = 8 * 2.0**-24 * r + 2 * 2.0**-23
    e_lse = ez.max(-1) + e_exp + 128 * 2.0**-24 + 4 * 2.0**-24 * (np.abs(lse) + np.abs(m))
    zt = z[rows, at]
    loss = lse - zt
    e_loss = e_lse + ez[rows, at] + 2.0**-24 * np.abs(loss)
    out = {"loss": (np.where(keep, loss, 0.0), np.where(keep, e_loss, 0.0)),
           "lse": (np.where(keep, lse, 0.0), np.where(keep, e_lse, 0.0))}
    if grad_loss is None:
        return out
    g = np.where(keep, grad_loss, 0.0)[:, None]
    p = np.exp(z - lse[:, None])
    dz = p.copy()
    dz[rows, at] = np.expm1(zt - lse)
    # relative error of p from its exponent, and what the roundings add
    rel = ez + (e_lse + 2 * e_exp)[:, None] + 8 * 2.0**-24
    edz = p * (rel + 2.0**-11) + 2.0**-39
    edz[rows, at] = p[rows, at] * rel[rows, at] + 8 * 2.0**-24 * np.abs(dz[rows, at])
    arith, edz = edz * np.abs(g), edz + 2.0**-8 * (np.abs(dz) + edz)
    dz, edz = dz * g, edz * np.abs(g) + 2.0**-130
    adz, half = np.abs(dz) + edz, 2.0**-8
    for name, a, e, s, b, f in (("dhidden", dz, edz, adz, w, arith), ("dweight", dz.T, edz.T, adz.T, h, arith.T)):
        value = a @ b
        sums = (a.shape[1] + 64) * 2.0**-23 * (s @ np.abs(b))
        bound = e @ np.abs(b) + sums
        # Root mean square of the error with the roundings of dz and of the
        # bf16 result taken as independent and uniform in their half steps, 1.5
        # times, and to it the bound of everything else.  (That part is not
        # small everywhere: a token whose loss is 7e-6, the difference of an
        # lse and a logit near 13, has a gradient of relative error 2^-24 * 13 /
        # 7e-6 = 11% from the rounding of either to fp32.)
        rms = 1.5 * np.sqrt(((half**2 / 3) * ((a**2) @ (b**2) + value**2)).sum())
        out[name] = (value, bound, rms + np.sqrt(((f @ np.abs(b) + sums) ** 2).sum()))
    return out
