"""The feed-forward sublayer and its update beside the collectives, as
measured cases.

Layer norm and its gradients, the gated feed-forward block (both projections,
the activation and the product) and its gradients, and the orthogonalised
update of weight matrices by Newton-Schulz products.  Where `own` is false every
operator is computed from elementary torch operations in 32 bits; where it is
true the package's operators are called.
"""
import math

import torch

own = False

FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
STEPS, COEFFICIENTS, NORM_EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7


def listed():
    return [
        # a few tokens' states before a block: a small call, latency counts
        dict(name="norm_few", op="norm", rows=5, cols=2048, x="bf16", y="bf16", affine="bf16", pad=0),
        # an fp32 residual stream into bf16 products, rows of a wider buffer
        dict(name="norm_stream", op="norm", rows=8191, cols=5120, x="f32", y="bf16", affine="f32", pad=256),
        # the backward pass over a short, odd batch
        dict(name="norm_grad_odd", op="norm_grad", rows=333, cols=1000, x="bf16", y="bf16", affine="f32", pad=0),
        # the backward pass over a long micro-batch
        dict(name="norm_grad_long", op="norm_grad", rows=16384, cols=8192, x="bf16", y="bf16", affine="bf16", pad=0),
        # one token: the weights are the traffic
        dict(name="gated_token", op="gated", tokens=1, hidden=4096, ffn=14336, act="silu", save=False),
        # a training micro-batch's forward pass, gates kept for the backward pass
        dict(name="gated_batch", op="gated", tokens=8192, hidden=4096, ffn=14336, act="silu", save=True),
        # one expert's share of a batch, gates formed again
        dict(name="gated_grad_expert", op="gated_grad", tokens=509, hidden=2048, ffn=768, act="silu", save=False),
        # a wide block from kept gates
        dict(name="gated_grad_kept", op="gated_grad", tokens=4096, hidden=5120, ffn=13824, act="gelu", save=True),
        # a micro-batch whose layer keeps its input only
        dict(name="gated_grad_again", op="gated_grad", tokens=8192, hidden=4096, ffn=14336, act="silu", save=False),
        # a key projection's update: a small matrix, latency counts
        dict(name="orthogonal_small", op="orthogonal", count=1, rows=512, cols=2048, x="bf16"),
        # a layer's experts' down projections: many tall matrices
        dict(name="orthogonal_experts", op="orthogonal", count=128, rows=2048, cols=768, x="bf16"),
        # a gate projection's update from fp32 momentum
        dict(name="orthogonal_large", op="orthogonal", count=1, rows=14336, cols=4096, x="f32"),
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated", "gated_grad", "orthogonal"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 40, 16384)
        return dict(op=op, rows=_log(rng, 1, min(65536, 16384 * 8192 // cols)), cols=cols, x=rng.choice(["bf16", "f32"]),
                    y=rng.choice(["bf16", "f32"]), affine=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 0, 1, 8, 256]))
    if op in ("gated", "gated_grad"):
        hidden, ffn = _log(rng, 64, 4096), _log(rng, 64, 14336)
        if rng.random() < 0.75:
            hidden, ffn = (hidden + 63) // 64 * 64, (ffn + 63) // 64 * 64
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=hidden, ffn=ffn, act=rng.choice(["silu", "gelu"]),
                    save=rng.choice([False, True]))
    rows, cols = _log(rng, 16, 4096), _log(rng, 16, 8192)
    if rng.random() < 0.5:
        rows, cols = (rows + 63) // 64 * 64, (cols + 63) // 64 * 64
    if rng.random() < 0.5:
        rows, cols = cols, rows
    return dict(op=op, count=_log(rng, 1, max(1, min(128, 4096 * 14336 // (rows * cols)))), rows=rows, cols=cols,
                x=rng.choice(["bf16", "f32"]))


def _stream(rows, cols, g):
    """A residual stream: unit scale with per-channel gains and offsets and a
    few channels of outliers."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    gain = torch.exp(0.5 * torch.randn(cols, device="cuda", generator=g))
    gain[torch.rand(cols, device="cuda", generator=g) < 0.005] *= 20.0
    return x.mul_(gain).add_(0.3 * torch.randn(cols, device="cuda", generator=g))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    op = case["op"]

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=g).mul_(scale)

    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        xt, yt, at = FLOAT[case["x"]], FLOAT[case["y"]], FLOAT[case["affine"]]
        x = torch.zeros(rows, cols + case["pad"], dtype=xt, device="cuda")
        s["x"] = x[:, :cols]
        s["x"].copy_(_stream(rows, cols, g))
        s["weight"] = (1.0 + 0.2 * normal(cols)).to(at)
        s["bias"] = (0.1 * normal(cols)).to(at)
        if op == "norm":
            s["out"] = empty(rows, cols, dtype=yt)
            s["mean"], s["rstd"] = empty(rows, dtype=torch.float32), empty(rows, dtype=torch.float32)
        else:
            v = s["x"].double()
            s["mean"] = v.mean(-1).float()
            s["rstd"] = torch.rsqrt(v.var(-1, unbiased=False) + EPS).float()
            s["dout"] = normal(rows, cols, scale=1e-3).to(yt)
            s["dx"] = empty(rows, cols, dtype=xt)
            s["dweight"], s["dbias"] = empty(cols, dtype=at), empty(cols, dtype=at)
        return s
    if op in ("gated", "gated_grad"):
        tokens, hidden, ffn = case["tokens"], case["hidden"], case["ffn"]
        s["x"] = normal(tokens, hidden).to(torch.bfloat16)
        s["gate"] = normal(ffn, hidden, scale=hidden ** -0.5).to(torch.bfloat16)
        s["up"] = normal(ffn, hidden, scale=hidden ** -0.5).to(torch.bfloat16)
        if op == "gated":
            s["out"] = empty(tokens, ffn)
            s["gates"] = empty(tokens, 2 * ffn) if case["save"] else None
            return s
        s["dout"] = normal(tokens, ffn, scale=1e-3).to(torch.bfloat16)
        s["gates"] = None
        if case["save"]:
            x = s["x"].float()
            s["gates"] = torch.cat([x @ s["gate"].float().t(), x @ s["up"].float().t()], -1).to(torch.bfloat16)
        s["dx"], s["dgate"], s["dup"] = empty(tokens, hidden), empty(ffn, hidden), empty(ffn, hidden)
        return s
    count, rows, cols = case["count"], case["rows"], case["cols"]
    # a momentum: a strong part of low rank and noise
    r = min(16, rows, cols)
    strength = torch.logspace(1, -1, r, device="cuda")
    m = normal(count, rows, cols)
    m.add_(torch.bmm(normal(count, rows, r).mul_(strength), normal(count, r, cols)))
    s["updates"] = list(m.mul_(1e-3).to(FLOAT[case["x"]]).unbind(0))
    s["out"] = empty(count, rows, cols)
    s["outs"] = list(s["out"].unbind(0))
    return s


# ------------------------------------------------------------ the plain form


def _plain_norm(x, weight, bias):
    x = x.float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)
    return d * rstd * weight.float() + bias.float(), mean.squeeze(-1), rstd.squeeze(-1)


def _plain_norm_grad(dout, x, weight, mean, rstd):
    dy, r = dout.float(), rstd.unsqueeze(-1)
    xh = (x.float() - mean.unsqueeze(-1)) * r
    g = dy * weight.float()
    dx = r * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def _plain_act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1.0 + g * (1.0 - s))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def _plain_gates(x, gate, up):
    x = x.float()
    return x @ gate.float().t(), x @ up.float().t()


def _plain_gated_grad(s):
    ffn = s["case"]["ffn"]
    if s["gates"] is None:
        g, u = _plain_gates(s["x"], s["gate"], s["up"])
    else:
        g, u = s["gates"][:, :ffn].float(), s["gates"][:, ffn:].float()
    a, da = _plain_act(g, s["case"]["act"])
    dh, x = s["dout"].float(), s["x"].float()
    dg, du = dh * u * da, dh * a
    return dg @ s["gate"].float() + du @ s["up"].float(), dg.t() @ x, du.t() @ x


def _plain_orthogonal(updates):
    x = torch.stack(updates).float()
    if x.shape[1] > x.shape[2]:
        x = x.transpose(1, 2).contiguous()
    a, b, c = COEFFICIENTS
    x = x / (torch.sqrt((x.double() ** 2).sum((1, 2), keepdim=True)).float() + NORM_EPS)
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    if updates[0].shape[0] > updates[0].shape[1]:
        x = x.transpose(1, 2)
    return x.to(torch.bfloat16).contiguous()


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd = _plain_norm(s["x"], s["weight"], s["bias"])
        return y.to(s["out"].dtype), mean, rstd
    if op == "norm_grad":
        dx, dw, db = _plain_norm_grad(s["dout"], s["x"], s["weight"], s["mean"], s["rstd"])
        return dx.to(s["dx"].dtype), dw.to(s["dweight"].dtype), db.to(s["dbias"].dtype)
    if op == "gated":
        g, u = _plain_gates(s["x"], s["gate"], s["up"])
        h = (_plain_act(g, case["act"])[0] * u).to(torch.bfloat16)
        return (h, torch.cat([g, u], -1).to(torch.bfloat16)) if case["save"] else (h,)
    if op == "gated_grad":
        return tuple(t.to(torch.bfloat16) for t in _plain_gated_grad(s))
    return _plain_orthogonal(s["updates"])


def _run_own(s):
    from param_collectives_amd import tide

    case = s["case"]
    op = case["op"]
    if op == "norm":
        tide.layer_norm(s["x"], s["weight"], s["bias"], s["out"], s["mean"], s["rstd"], eps=EPS)
        return s["out"], s["mean"], s["rstd"]
    if op == "norm_grad":
        tide.layer_norm_grad(s["dout"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"])
        return s["dx"], s["dweight"], s["dbias"]
    if op == "gated":
        tide.gated_block(s["x"], s["gate"], s["up"], s["out"], gates=s["gates"], activation=case["act"])
        return (s["out"], s["gates"]) if case["save"] else (s["out"],)
    if op == "gated_grad":
        tide.gated_block_grad(s["dout"], s["x"], s["gate"], s["up"], s["dx"], s["dgate"], s["dup"], gates=s["gates"],
                              activation=case["act"])
        return s["dx"], s["dgate"], s["dup"]
    tide.orthogonalize(s["updates"], s["outs"], steps=STEPS, coefficients=COEFFICIENTS, eps=NORM_EPS)
    return s["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, sx, sy = case["rows"] * case["cols"], FLOAT[case["x"]].itemsize, FLOAT[case["y"]].itemsize
        sa = FLOAT[case["affine"]].itemsize
        if op == "norm":
            return {"bytes": n * (sx + sy) + 2 * case["cols"] * sa + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": n * (2 * sx + sy) + 3 * case["cols"] * sa + 8 * case["rows"], "flops": 13 * n}
    if op in ("gated", "gated_grad"):
        t, d, f = case["tokens"], case["hidden"], case["ffn"]
        kept = 4 * t * f if case["save"] else 0
        if op == "gated":
            return {"bytes": 2 * t * d + 4 * f * d + 2 * t * f + kept, "flops": 4 * t * d * f}
        return {"bytes": 4 * t * d + 8 * f * d + 2 * t * f + kept, "flops": (8 if case["save"] else 12) * t * d * f}
    n, m = max(case["rows"], case["cols"]), min(case["rows"], case["cols"])
    # both square products are symmetric
    return {"bytes": case["count"] * m * n * (FLOAT[case["x"]].itemsize + 2),
            "flops": case["count"] * STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)}


# ------------------------------------------------------------ the definition


def _exact_act(g, act):
    if act == "silu":
        e = torch.exp(-g.abs())
        s = torch.where(g >= 0, 1 / (1 + e), e / (1 + e))
        return g * s, s + g * s * (1 - s)
    k = math.sqrt(2.0 / math.pi)
    inner = k * g * (1 + 0.044715 * g.square())
    sech = 1 / torch.cosh(inner.clamp(-300, 300))
    return g * (1 + torch.tanh(inner)) / 2, (1 + torch.tanh(inner)) / 2 + g / 2 * sech.square() * k * (
        1 + 0.134145 * g.square())


def _exact_norm(s):
    case = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, -1, correction=0)
        rstd = (var + EPS).rsqrt()
        return torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), mean, rstd
    mean, rstd = s["mean"].double(), s["rstd"].double()
    xh, dy = (x - mean[:, None]) * rstd[:, None], s["dout"].double()
    n = case["cols"]
    along = torch.stack([torch.mv(dy, w), torch.mv(dy * xh, w)], -1) / n
    dx = (dy * w - along[:, :1] - xh * along[:, 1:]) * rstd[:, None]
    return dx, torch.einsum("tc,tc->c", dy, xh), torch.mv(dy.t(), torch.ones(case["rows"], dtype=dy.dtype, device="cuda"))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s)
    if op == "orthogonal":
        outs = []
        for u in s["updates"]:
            x = u.double()
            tall = x.shape[0] > x.shape[1]
            x = x.t().contiguous() if tall else x
            x = x / (torch.linalg.vector_norm(x) + NORM_EPS)
            for _ in range(STEPS):
                a1 = torch.matmul(x, x.t().contiguous())
                a1x = torch.matmul(a1, x)
                x = COEFFICIENTS[0] * x + COEFFICIENTS[1] * a1x + COEFFICIENTS[2] * torch.matmul(a1, a1x)
            outs.append(x.t().contiguous() if tall else x)
        return torch.stack(outs)
    ffn = case["ffn"]
    x, wg, wu = s["x"].double(), s["gate"].double(), s["up"].double()
    if s["gates"] is None or op == "gated":
        g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    else:
        g, u = s["gates"].double().split(ffn, -1)
    a, da = _exact_act(g, case["act"])
    if op == "gated":
        return (a * u, torch.cat([g, u], -1)) if case["save"] else (a * u,)
    dh = s["dout"].double()
    da.mul_(dh).mul_(u)
    a.mul_(dh)
    return torch.matmul(da, wg) + torch.matmul(a, wu), torch.matmul(da.t(), x), torch.matmul(a.t(), x)
