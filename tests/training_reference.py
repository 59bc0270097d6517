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
