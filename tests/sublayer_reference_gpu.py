"""The references of tests/sublayer_reference.py for sizes that take the CPU too
long: the same definitions and bounds, whose derivations stand there, in float64 on
the GPU (its library's products of float64 matrices)."""
import math

import torch

from tests.sublayer_reference import EXACT_SUM, HALF, TINY, U32


def held(t, dtype):
    """The float64 values that t's rounding to `dtype` holds."""
    return t.to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype]).double()


def close(got, value, err, dtype, what):
    """Every element within its bound after one rounding to `dtype`."""
    off = (got.double() - value).abs()
    bad = ~(off <= err + HALF[dtype] * (value.abs() + err) + TINY[dtype])
    if bool(bad.any()):
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError((what, int(bad.sum()), at, float(got[at]), float(value[at])))


def act(z, name):
    if name == "silu":
        k, dk = z, torch.ones_like(z)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        k, dk = c * (z + 0.044715 * z**3), c * (1 + 3 * 0.044715 * z**2)
    e = torch.exp(-k.abs())
    s = torch.where(k >= 0, torch.ones_like(e), e) / (1 + e)
    return z * s, s + z * dk * e / (1 + e) ** 2, k


def _activated(z, ez, name):
    a, d, k = act(z, name)
    rel = (4 * k.abs() + 10) * EXACT_SUM
    some = torch.where(z == 0, torch.ones_like(z), z)
    s, flush = (a / some).abs() + (z == 0) * 0.5, 2.0**-125 * (1 + z.abs())
    ea = 1.13 * ez + a.abs() * rel + flush
    share = torch.where(z == 0, torch.full_like(z, 0.5), a / some)
    return a, ea, d, 0.8 * ez + rel * (s + (d - share).abs()) + flush


def _gates(x, wg, wu):
    n = (x.shape[1] + 64) * EXACT_SUM
    (a, g, u) = (t.t().contiguous() for t in (x, wg, wu))
    x = a.t().contiguous()
    return x @ g, n * (x.abs() @ g.abs()), x @ u, n * (x.abs() @ u.abs())


def gated_block(x, wg, wu, name):
    g, eg, u, eu = _gates(x, wg, wu)
    a, ea, _, _ = _activated(g, eg, name)
    eh = ea * u.abs() + a.abs() * eu + ea * eu + 2 * U32 * (a * u).abs()
    return {"out": (a * u, eh), "gates": (torch.cat([g, u], 1), torch.cat([eg, eu], 1))}


def gated_block_grad(dout, x, wg, wu, name, gates=None, old=None):
    f = wg.shape[0]
    if gates is None:
        g, eg, u, eu = _gates(x, wg, wu)
    else:
        g, u = gates[:, :f].contiguous(), gates[:, f:].contiguous()
        eg = eu = torch.zeros_like(g)
    a, ea, d, ed = _activated(g, eg, name)
    dh = dout.abs()
    dg, du = dout * u * d, dout * a
    arith = [dh * (u.abs() * ed + d.abs() * eu + ed * eu) + 3 * U32 * dg.abs(), dh * ea + 2 * U32 * du.abs()]
    half = HALF["bf16"]
    err = [e + half * (v.abs() + e) + TINY["bf16"] for v, e in zip((dg, du), arith)]
    out = {}

    def product(name, pairs, old=None):
        value = sum(p @ b for p, _, _, b in pairs)
        k = sum(b.shape[0] for _, _, _, b in pairs)
        sums = (k + 64) * EXACT_SUM * sum((p.abs() + e) @ b.abs() for p, e, _, b in pairs)
        var = half**2 / 3 * sum((p**2) @ (b**2) for p, _, _, b in pairs)
        rest = sum(ar @ b.abs() for _, _, ar, b in pairs) + sums
        bound = sum(e @ b.abs() for _, e, _, b in pairs) + sums
        if old is not None:
            value = value + old
            bound, rest = bound + U32 * value.abs(), rest + U32 * value.abs()
        rms = 1.5 * float((var + half**2 / 3 * value**2).sum().sqrt()) + float((rest**2).sum().sqrt())
        out[name] = (value, bound, rms)

    def across(t):
        return t.t().contiguous()

    product("dx", [(dg, err[0], arith[0], wg), (du, err[1], arith[1], wu)])
    product("dw_gate", [(across(dg), across(err[0]), across(arith[0]), x)], None if old is None else old[0])
    product("dw_up", [(across(du), across(err[1]), across(arith[1]), x)], None if old is None else old[1])
    return out


def _f16(t):
    return (t * 4096).half().double() / 4096


def orthogonalize(x, steps, a, b, c, eps, exact=3, f32=True):
    """(value, error of the definition with the kernels' roundings put in) of a
    float64 matrix."""
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    y = z = x / (x.norm() + eps)
    one = torch.eye(len(x), dtype=x.dtype, device=x.device)
    for k in range(steps):
        g = z @ z.t().contiguous()
        z = a * z + (b * g + c * (g @ g)) @ z
        h = _f16(y) if k > 0 or f32 else y
        g = _f16(h @ h.t().contiguous())
        y = _f16(b * g + c * (g @ g) + a * one) @ h + (a * _f16((y - h) * 2048) / 2048 if k < exact else 0)
    return (z.t(), (y - z).t()) if tall else (z, y - z)
