"""The training-step operators beside the collectives, as measured cases.

Activation checkpoints held in 8 bits (packed, unpacked, and read by the
weight gradient) and the cross entropy of the output projection (the loss of
an evaluation, the loss with its gradients of a training step).  Where `own`
is false every operator is computed from elementary torch operations in 32
bits; where it is true the package's operators are called.

A packed activation holds blocks of 32 values of a row: one byte of code per
value (e4m3 or a signed integer) and one byte per block, the biased exponent
of the power of two that the block's codes are multiplied by.  A row's last
block is filled up with zero codes.
"""
import torch

own = False

BLOCK = 32
CODE_DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32}
LOWEST, HIGHEST, NOT_FINITE = 10, {"e4m3": 246, "int8": 248}, 255  # biased block exponents


def listed():
    return [
        # a short sequence's normed activations: a small call, latency counts
        dict(name="round_trip_short", op="round_trip", rows=64, cols=2048, stride=2048, dtype="bf16", fmt="e4m3"),
        # the input of a down projection over a micro-batch
        dict(name="round_trip_ffn", op="round_trip", rows=8192, cols=14336, stride=14336, dtype="bf16", fmt="int8"),
        # an fp32 residual stream held as a slice of a wider buffer
        dict(name="round_trip_strided_f32", op="round_trip", rows=4095, cols=5120, stride=5376, dtype="f32",
             fmt="e4m3"),
        # ragged rows whose last block is short
        dict(name="unpack_ragged", op="unpack", rows=333, cols=1000, dtype="bf16", fmt="int8"),
        # a wide layer's input restored for a recomputed segment
        dict(name="unpack_wide", op="unpack", rows=16384, cols=8192, dtype="bf16", fmt="e4m3"),
        # one expert's share of a batch: few tokens, an odd number
        dict(name="weight_grad_expert", op="weight_grad", tokens=509, outs=768, ins=2048, fmt="int8", grad="bf16"),
        # a square attention projection
        dict(name="weight_grad_square", op="weight_grad", tokens=4096, outs=4096, ins=4096, fmt="e4m3", grad="bf16"),
        # a down projection over a long micro-batch, into fp32 gradients
        dict(name="weight_grad_down", op="weight_grad", tokens=8192, outs=4096, ins=14336, fmt="int8", grad="f32"),
        # scoring a handful of tokens: the projection's weights are the traffic
        dict(name="loss_few_tokens", op="loss", tokens=17, hidden=2048, vocab=32000, ignored=0.0),
        # evaluation over a batch
        dict(name="loss_batch", op="loss", tokens=4096, hidden=4096, vocab=65536, ignored=0.0),
        # a padded batch, odd vocabulary
        dict(name="loss_grad_padded", op="loss_grad", tokens=1111, hidden=2048, vocab=50001, ignored=0.4, grad="bf16"),
        # a training step's head
        dict(name="loss_grad_step", op="loss_grad", tokens=4096, hidden=4096, vocab=128000, ignored=0.02,
             grad="bf16"),
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["round_trip", "unpack", "weight_grad", "loss", "loss_grad"])
    fmt = rng.choice(["e4m3", "int8"])
    if op in ("round_trip", "unpack"):
        cols = _log(rng, 100, 14336)
        rows = _log(rng, 16, 8192 * 14336 // max(cols, 3584))
        case = dict(op=op, rows=rows, cols=cols, fmt=fmt, dtype=rng.choice(["bf16", "f32"]))
        if op == "round_trip":
            case["stride"] = cols + rng.choice([0, 0, 1, 8, 256])
        return case
    if op == "weight_grad":
        return dict(op=op, tokens=_log(rng, 64, 8192), outs=_log(rng, 96, 5120), ins=_log(rng, 96, 14336), fmt=fmt,
                    grad=rng.choice(["bf16", "f32"]))
    hidden = _log(rng, 200, 4096)
    if rng.random() < 0.75:
        hidden = (hidden + 63) // 64 * 64
    return dict(op=op, tokens=_log(rng, 8, 4096), hidden=hidden, vocab=_log(rng, 1000, 128000),
                ignored=rng.choice([0.0, 0.0, 0.1, 0.5]), **({"grad": "bf16"} if op == "loss_grad" else {}))


def _blocks(cols):
    return (cols + BLOCK - 1) // BLOCK


def _ignored(case):
    return int(case["tokens"] * case["ignored"])


def _activation(rows, cols, g):
    """Activations as a layer's norm leaves them: unit scale with per-channel
    gains and a few channels of outliers."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    gain = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=g))
    gain[torch.rand(cols, device="cuda", generator=g) < 0.005] *= 20.0
    return x.mul_(gain)


def _packed(x, fmt):
    """Codes and block exponents of a float tensor, as a forward pass left
    them (any block exponent would do for the readers)."""
    rows, cols = x.shape
    nb = _blocks(cols)
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    top = 448.0 if fmt == "e4m3" else 127.0
    _, e = torch.frexp(v.abs().amax(-1).clamp_min(1e-20) / top)
    v = torch.ldexp(v, -e.unsqueeze(-1))
    codes = v.to(torch.float8_e4m3fn) if fmt == "e4m3" else v.round().to(torch.int8)
    return codes.view(rows, nb * BLOCK), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op in ("round_trip", "unpack"):
        rows, cols = case["rows"], case["cols"]
        nb = _blocks(cols)
        if op == "round_trip":
            x = torch.zeros(rows, case["stride"], dtype=FLOAT[case["dtype"]], device="cuda")
            s["x"] = x[:, :cols]
            s["x"].copy_(_activation(rows, cols, g))
            s["codes"] = torch.empty(rows, nb * BLOCK, dtype=CODE_DTYPE[case["fmt"]], device="cuda")
            s["scales"] = torch.empty(rows, nb, dtype=torch.uint8, device="cuda")
        else:
            s["codes"], s["scales"] = _packed(_activation(rows, cols, g), case["fmt"])
        s["out"] = torch.empty(rows, cols, dtype=FLOAT[case["dtype"]], device="cuda")
        return s
    if op == "weight_grad":
        tokens, outs, ins = case["tokens"], case["outs"], case["ins"]
        s["codes"], s["scales"] = _packed(_activation(tokens, ins, g), case["fmt"])
        s["dy"] = (1e-3 * torch.randn(tokens, outs, device="cuda", generator=g)).to(torch.bfloat16)
        s["dw"] = torch.empty(outs, ins, dtype=FLOAT[case["grad"]], device="cuda")
        return s
    tokens, hidden, vocab = case["tokens"], case["hidden"], case["vocab"]
    w = torch.randn(vocab, hidden, device="cuda", generator=g).mul_(hidden ** -0.5).to(torch.bfloat16)
    t = torch.randint(vocab, (tokens,), device="cuda", generator=g)
    # a trained model's states lean towards the rows of their targets, some strongly
    lean = 12.0 * torch.rand(tokens, 1, device="cuda", generator=g)
    h = torch.randn(tokens, hidden, device="cuda", generator=g) + lean * w[t].float()
    s["hidden"], s["weight"] = h.to(torch.bfloat16), w
    n = _ignored(case)
    t[torch.randperm(tokens, device="cuda", generator=g)[:n]] = -100
    s["targets"] = t
    s["loss"] = torch.empty(tokens, dtype=torch.float32, device="cuda")
    s["lse"] = torch.empty(tokens, dtype=torch.float32, device="cuda")
    if op == "loss_grad":
        s["grad_loss"] = torch.full((tokens,), 1.0 / max(tokens - n, 1), dtype=torch.float32, device="cuda")
        s["dhidden"] = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
        s["dweight"] = torch.empty(vocab, hidden, dtype=FLOAT[case["grad"]], device="cuda")
    return s


# ------------------------------------------------------------ the plain form


def _round_e4m3(y):
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(y / step) * step


def _plain_round_trip(x, fmt, dtype):
    rows, cols = x.shape
    nb = _blocks(cols)
    v = torch.zeros(rows, nb * BLOCK, dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, nb, BLOCK)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax)
    if fmt == "e4m3":
        b = e - 1 - 8 + (m > 0.875).int() + 127
    else:
        b = e - 1 - 6 + (m > 127.5 / 128).int() + 127
    b = torch.clamp(b, LOWEST, HIGHEST[fmt]).unsqueeze(-1)
    y = torch.ldexp(v, 127 - b)
    if fmt == "e4m3":
        q = _round_e4m3(torch.clamp(y, -448.0, 448.0))
    else:
        q = torch.clamp(torch.round(y), -127.0, 127.0)
    out = torch.ldexp(q, b - 127)
    out = torch.where(torch.isfinite(amax).unsqueeze(-1), out, float("nan"))
    return out.view(rows, nb * BLOCK)[:, :cols].to(dtype)


def _plain_values(codes, scales, cols):
    rows = codes.shape[0]
    q = codes.float().view(rows, -1, BLOCK)
    v = torch.ldexp(q, scales.int().unsqueeze(-1) - 127)
    v = torch.where((scales == NOT_FINITE).unsqueeze(-1), float("nan"), v)
    return v.view(rows, -1)[:, :cols]


def _plain_loss(hidden, weight, targets, grad_loss=None, grad_dtype=None):
    w = weight.float()
    keep = (targets >= 0) & (targets < weight.shape[0])
    h = torch.where(keep.unsqueeze(-1), hidden.float(), 0.0)
    z = h @ w.t()
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    at = torch.where(keep, targets, 0).unsqueeze(-1)
    below = z.gather(-1, at).squeeze(-1) - lse
    loss = torch.where(keep, -below, 0.0)
    lse = torch.where(keep, lse, 0.0)
    if grad_loss is None:
        return loss, lse
    p /= total
    p.scatter_(-1, at, torch.expm1(below).unsqueeze(-1))
    p *= torch.where(keep, grad_loss, 0.0).unsqueeze(-1)
    return loss, lse, (p @ w).to(hidden.dtype), (p.t() @ h).to(grad_dtype)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "round_trip":
        return _plain_round_trip(s["x"], case["fmt"], s["out"].dtype)
    if op == "unpack":
        return _plain_values(s["codes"], s["scales"], case["cols"]).to(s["out"].dtype)
    if op == "weight_grad":
        x = _plain_values(s["codes"], s["scales"], case["ins"])
        return (s["dy"].float().t() @ x).to(s["dw"].dtype)
    if op == "loss":
        return _plain_loss(s["hidden"], s["weight"], s["targets"])
    return _plain_loss(s["hidden"], s["weight"], s["targets"], s["grad_loss"], s["dweight"].dtype)


def _run_own(s):
    from param_collectives_amd import tide

    op = s["case"]["op"]
    if op == "round_trip":
        tide.checkpoint_pack(s["x"], s["codes"], s["scales"])
        tide.checkpoint_unpack(s["codes"], s["scales"], s["out"])
        return s["out"]
    if op == "unpack":
        tide.checkpoint_unpack(s["codes"], s["scales"], s["out"])
        return s["out"]
    if op == "weight_grad":
        tide.checkpoint_weight_grad(s["dy"], s["codes"], s["scales"], s["dw"])
        return s["dw"]
    if op == "loss":
        tide.vocab_loss(s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"])
        return s["loss"], s["lse"]
    tide.vocab_loss_grad(s["hidden"], s["weight"], s["targets"], s["grad_loss"], s["loss"], s["lse"], s["dhidden"],
                         s["dweight"])
    return s["loss"], s["lse"], s["dhidden"], s["dweight"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op in ("round_trip", "unpack"):
        n, size = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        packed = n + case["rows"] * _blocks(case["cols"])
        # a round trip writes the packed form once and reads it back once
        return {"bytes": 2 * n * size + 2 * packed, "flops": 0} if op == "round_trip" else \
            {"bytes": packed + n * size, "flops": 0}
    if op == "weight_grad":
        t, o, i = case["tokens"], case["outs"], case["ins"]
        return {"bytes": 2 * t * o + t * i + t * _blocks(i) + o * i * (2 if case["grad"] == "bf16" else 4),
                "flops": 2 * t * o * i}
    t, d, v = case["tokens"], case["hidden"], case["vocab"]
    n = t - _ignored(case)
    if op == "loss":
        return {"bytes": 2 * n * d + 2 * v * d + 8 * t + 8 * t, "flops": 2 * n * d * v}
    return {"bytes": 2 * n * d + 2 * v * d + 8 * t + 4 * n + 8 * t + 2 * t * d
            + v * d * (2 if case["grad"] == "bf16" else 4), "flops": 6 * n * d * v}


# ------------------------------------------------------------ the definition


def _exact_round_trip(x, fmt):
    rows, cols = x.shape
    out = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    if fmt == "e4m3":
        codes = torch.arange(127, device=x.device)
        e, f = codes >> 3, (codes & 7).double()
        table = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2((e - 7).double()))
    else:
        table = torch.arange(128, device=x.device).double()
    middle = (table[1:] + table[:-1]) / 2
    limit = 448.0 if fmt == "e4m3" else 127.5
    for c0 in range(0, cols, BLOCK * 64):
        c1 = min(cols, c0 + BLOCK * 64)
        v = x[:, c0:c1].double()
        n = c1 - c0
        amax = torch.stack([v[:, b:b + BLOCK].abs().amax(-1) for b in range(0, n, BLOCK)], -1)
        e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -160) / limit))
        e += (amax > limit * torch.exp2(e)).double()
        e -= (amax <= limit * torch.exp2(e - 1)).double()
        e = e.clamp(LOWEST - 127, HIGHEST[fmt] - 127)
        unit = torch.exp2(e).repeat_interleave(BLOCK, -1)[:, :n]
        a = (v.abs() / unit).contiguous()
        # the nearest code, of two equally near the one with an even number
        low = torch.searchsorted(middle, a, right=False)
        tie = (low < middle.numel()) & (middle[low.clamp(max=middle.numel() - 1)] == a)
        low = torch.where(tie & (low % 2 == 1), low + 1, low)
        out[:, c0:c1] = torch.copysign(table[low] * unit, v)
    return out


def _exact_values(codes, scales, cols):
    unit = torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)
    return (codes.to(torch.float32).double() * unit)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "round_trip":
        return _exact_round_trip(s["x"], case["fmt"])
    if op == "unpack":
        return _exact_values(s["codes"], s["scales"], case["cols"])
    if op == "weight_grad":
        x = _exact_values(s["codes"], s["scales"], case["ins"])
        return torch.matmul(s["dy"].double().t().contiguous(), x)
    tokens, hidden, vocab = case["tokens"], case["hidden"], case["vocab"]
    loss = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    rows = torch.nonzero(s["targets"] >= 0).flatten()
    t = s["targets"][rows]
    w = s["weight"].double()
    grads = op == "loss_grad"
    if grads:
        dh = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
        dw = torch.zeros(vocab, hidden, dtype=torch.float64, device="cuda")
    for r0 in range(0, rows.numel(), 1024):
        r, tt = rows[r0:r0 + 1024], t[r0:r0 + 1024]
        h = s["hidden"][r].double()
        z = torch.matmul(h, w.t())
        l = torch.logsumexp(z, -1)
        here = z[torch.arange(r.numel(), device="cuda"), tt]
        lse[r], loss[r] = l, l - here
        if grads:
            d = torch.softmax(z, -1)
            d[torch.arange(r.numel(), device="cuda"), tt] -= 1.0
            d *= s["grad_loss"][r].double().unsqueeze(-1)
            dh[r] = torch.matmul(d, w)
            dw += torch.matmul(d.t(), h)
    return (loss, lse, dh, dw) if grads else (loss, lse)
