"""GPU checks of the vocabulary loss and its gradients against 64-bit
references."""
import numpy as np
import pytest

from tests import training_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def bf16(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)


def make(rng, tokens, size, vocab, ignored=0.0, spread=1.0):
    """Host bf16 hidden states that lean towards their targets' rows, some
    strongly, weights, targets (some outside the vocabulary) and gradients."""
    w = bf16(rng.standard_normal((vocab, size)) * spread * size**-0.5)
    t = rng.integers(0, vocab, tokens)
    h = bf16(rng.standard_normal((tokens, size)) + rng.uniform(0, 12, (tokens, 1)) * w.double().numpy()[t])
    out = rng.random(tokens) < ignored
    t[out] = rng.choice([-100, -1, vocab, vocab + 3, 2**40], int(out.sum()))
    g = (rng.uniform(0.2, 2.0, tokens) / tokens).astype(np.float32)
    return h, w, t, g


class Run:
    """One call with canaries in every output."""

    def __init__(self, tide, h, w, t, g, dtype="bf16", old=None, null_lse=False, **kw):
        import torch

        self.tokens, self.size, self.vocab = h.shape[0], h.shape[1], w.shape[0]
        dev = [x.cuda() if x.device.type == "cpu" else x for x in (h, w)]
        self.loss = torch.full((self.tokens,), 77.0, device="cuda")
        self.lse = None if null_lse else torch.full((self.tokens,), 77.0, device="cuda")
        targets = torch.from_numpy(t).cuda()
        grads = None if g is None else torch.from_numpy(g).cuda()
        if kw.get("stream") is not None:
            kw["stream"].wait_stream(torch.cuda.current_stream())  # the operands and canaries
        if g is None:
            tide.vocab_loss(*dev, targets, self.loss, self.lse, **kw)
            return
        self.dh = torch.full((self.tokens, self.size), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.dw = torch.full((self.vocab, self.size), float("nan"), device="cuda",
                             dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
        if old is not None:
            self.dw.copy_(old)
        if kw.get("stream") is not None:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        tide.vocab_loss_grad(*dev, targets, grads, self.loss, self.lse, self.dh, self.dw,
                             accumulate=old is not None, **kw)

    def check(self, want, old=None):
        import torch

        half = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8}
        for name, got in (("loss", self.loss), ("lse", self.lse), ("dhidden", getattr(self, "dh", None)),
                          ("dweight", getattr(self, "dw", None))):
            if got is None or name not in want:
                continue
            value, bound = want[name][:2]
            if name == "dweight" and old is not None:
                value, bound = value + old, bound + 2.0**-23 * (np.abs(value) + np.abs(old))
            diff = np.abs(got.double().cpu().numpy() - value)
            limit = bound * (1 + half[got.dtype]) + half[got.dtype] * np.abs(value) + 2.0**-126
            bad = ~(diff <= limit)
            assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(diff / limit)))
            # the worst case of every rounding at once is far from what happens:
            # the norm of the error against what the roundings give together
            if len(want[name]) > 2 and old is None:
                assert np.sqrt((diff**2).sum()) <= want[name][2] + 2.0**-100, name


SHAPES = [(1, 8, 1), (1, 64, 2), (3, 7, 5), (17, 100, 1000), (64, 64, 64), (65, 96, 129), (100, 33, 257),
          (255, 128, 300), (257, 64, 256), (300, 200, 1111), (513, 72, 70), (700, 64, 6000)]


@pytest.mark.parametrize("tokens,size,vocab", SHAPES)
def test_loss(tide, tokens, size, vocab):
    h, w, t, _ = make(np.random.default_rng(tokens + vocab), tokens, size, vocab)
    Run(tide, h, w, t, None).check(ref.vocab_loss(h.double().numpy(), w.double().numpy(), t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ignored", [0.0, 0.4])
@pytest.mark.parametrize("tokens,size,vocab", SHAPES)
def test_gradients(tide, tokens, size, vocab, ignored, dtype):
    h, w, t, g = make(np.random.default_rng(tokens + size), tokens, size, vocab, ignored)
    Run(tide, h, w, t, g, dtype).check(ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float)))


@pytest.mark.parametrize("tokens,size,vocab", [(2900, 64, 4500), (1500, 2048, 8200)])
def test_large_tiles(tide, tokens, size, vocab):
    """Enough tiles for the large ones in every product that can take them."""
    h, w, t, g = make(np.random.default_rng(vocab), tokens, size, vocab, 0.1)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    Run(tide, h, w, t, g).check(want)
    Run(tide, h, w, t, None).check(want)


def test_large_tiles_of_the_hidden_gradient(tide):
    h, w, t, g = make(np.random.default_rng(8), 3000, 4104, 200, 0.1)
    Run(tide, h, w, t, g).check(ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float)))


@pytest.mark.parametrize("tokens", [10, 300])
def test_left_out_tokens_have_no_effect(tide, tokens):
    """NaN and infinities in the states and gradients of tokens that are left
    out reach nothing; a batch that leaves every token out gives zeros."""
    import torch

    h, w, t, g = make(np.random.default_rng(3), tokens, 72, 500, 0.5)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    out = np.nonzero((t < 0) | (t >= 500))[0]
    assert 0 < len(out) < tokens
    h[out[::2]], h[out[1::2]], g[out] = float("nan"), float("inf"), np.nan
    Run(tide, h, w, t, g).check(want)
    Run(tide, h, w, t, None).check(want)
    r = Run(tide, h, w, np.full(tokens, -100), g)
    for x in (r.loss, r.lse, r.dh, r.dw):
        assert not x.any()
    r = Run(tide, h, w, np.full(tokens, -100), None)
    assert not r.loss.any() and not r.lse.any()


def test_no_tokens(tide):
    import torch

    w = torch.zeros(30, 16, dtype=torch.bfloat16)
    h, t, g = w[:0], np.zeros(0, np.int64), np.zeros(0, np.float32)
    for dtype in ("bf16", "f32"):
        assert not Run(tide, h, w, t, g, dtype).dw.any()
        assert (Run(tide, h, w, t, g, dtype, old=torch.full((30, 16), 3.0)).dw == 3.0).all()
    Run(tide, h, w, t, None)


def test_non_finite_tokens_keep_to_their_rows(tide):
    """A counted token with a NaN state: its loss and row are NaN, and so is
    dweight (the formula's); the other tokens' losses and rows are untouched."""
    import torch

    h, w, t, g = make(np.random.default_rng(4), 100, 64, 300)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    h[42, 5] = float("nan")
    r = Run(tide, h, w, t, g)
    assert torch.isnan(r.loss[42]) and torch.isnan(r.dh[42]).all() and torch.isnan(r.dw).all()
    keep = np.arange(100) != 42
    r.loss, r.lse, r.dh = (x[torch.from_numpy(keep).cuda()] for x in (r.loss, r.lse, r.dh))
    r.check({k: (want[k][0][keep], want[k][1][keep]) for k in ("loss", "lse", "dhidden")})


def test_confident_and_hopeless_tokens(tide):
    """Targets of probability near 1 (their gradient is a difference that must
    not cancel) and near 0, and logits far below the largest."""
    rng = np.random.default_rng(6)
    size, vocab = 64, 400
    w = bf16(rng.standard_normal((vocab, size)))
    t = rng.integers(0, vocab, 64)
    gain = np.where(np.arange(64) % 2 == 0, 0.4, -0.8)[:, None] * rng.uniform(0.2, 1.0, (64, 1))
    h = bf16(gain * w.double().numpy()[t])
    g = np.ones(64, np.float32)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    assert want["loss"][0].min() < 1e-5 and want["loss"][0].max() > 50
    Run(tide, h, w, t, g, "f32").check(want)
    # one token alone: its small gradient is not hidden by the others'
    at = int(np.argmin(want["loss"][0]))
    one = ref.vocab_loss(h[at:at + 1].double().numpy(), w.double().numpy(), t[at:at + 1], np.ones(1))
    r = Run(tide, h[at:at + 1], w, t[at:at + 1], np.ones(1, np.float32), "f32")
    r.check(one)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accumulate(tide, dtype):
    import torch

    h, w, t, g = make(np.random.default_rng(9), 150, 40, 330, 0.2)
    old = torch.from_numpy(np.random.default_rng(10).standard_normal((330, 40)) * 1e-3).to(
        torch.float32 if dtype == "f32" else torch.bfloat16)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    Run(tide, h, w, t, g, dtype, old=old).check(want, old.double().numpy())


@pytest.mark.parametrize("h_at,h_ld,w_at,w_ld", [(0, 96, 0, 96), (0, 104, 0, 160), (1, 96, 0, 96), (0, 97, 8, 104),
                                                 (0, 96, 1, 96), (3, 101, 5, 99), (0, 96, 0, 97)])
def test_strided_operands(tide, h_at, h_ld, w_at, w_ld):
    import torch

    tokens, size, vocab = 120, 96, 333
    h, w, t, g = make(np.random.default_rng(w_ld), tokens, size, vocab, 0.1)

    def place(x, at, ld):
        flat = torch.full((at + x.shape[0] * ld,), float("nan"), dtype=torch.bfloat16, device="cuda")
        v = flat.as_strided(x.shape, (ld, 1), at)
        v.copy_(x)
        return v

    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    hd, wd = place(h, h_at, h_ld), place(w, w_at, w_ld)
    Run(tide, hd, wd, t, g).check(want)
    Run(tide, hd, wd, t, None, null_lse=True).check(want)
    Run(tide, hd, wd, t, g, null_lse=True).check(want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,ignored", [(600, 0.0), (600, 0.5), (1100, 0.2)])
def test_pieces(tide, tokens, ignored, dtype):
    """More tokens than one piece holds (2 GiB of exponentials: 512 tokens of a
    vocabulary of 2^21), the last pieces short or, with tokens left out, empty;
    against the same sums in 64 bits on the GPU."""
    import torch

    size, vocab = 8, 1 << 21
    rng = np.random.default_rng(12)
    h, w, t, g = make(rng, tokens, size, vocab, ignored)
    r = Run(tide, h, w, t, g, dtype)
    H, Wd = h.double().cuda(), w.double().cuda()
    keep = np.nonzero((t >= 0) & (t < vocab))[0]
    dw, dh = torch.zeros_like(Wd), torch.zeros_like(H)
    loss = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    for k0 in range(0, len(keep), 128):
        k = torch.from_numpy(keep[k0:k0 + 128]).cuda()
        tt, gg = torch.from_numpy(t[keep[k0:k0 + 128]]).cuda(), torch.from_numpy(g).double().cuda()[k]
        z = H[k] @ Wd.t()
        lse = torch.logsumexp(z, -1)
        i = torch.arange(len(k), device="cuda")
        loss[k] = lse - z[i, tt]
        p = torch.exp(z - lse[:, None])
        p[i, tt] -= 1.0
        p *= gg[:, None]
        dh[k] = p @ Wd
        dw += p.t().contiguous() @ H[k]
    # a logit of 8 products and at most 2^14 roundings of 2^-24 on the way to lse
    assert (r.loss.double() - loss).abs().max() < 2.0**-10
    # dz rounded by 2^-8 at most (2^-8 / sqrt(3) in the mean square), the bf16 results once more
    for got, want in ((r.dh, dh), (r.dw, dw)):
        assert float((got.double() - want).norm() / want.norm()) < 2.0**-8 * (2 / 3) ** 0.5 * 1.2
    assert not r.dh[torch.from_numpy(np.setdiff1d(np.arange(tokens), keep)).cuda()].any()


def test_a_training_step(tide):
    """The head of a step as it is used: the last layer's input packed, the
    loss and its gradients, the layer's weight gradient from the checkpoint, and
    the reduce-scatter of both; eagerly on a stream and as a captured graph
    replayed with new inputs."""
    import torch

    rng = np.random.default_rng(14)
    tokens, ins, size, vocab, W = 300, 64, 72, 515, 2
    x = torch.empty(tokens, ins, dtype=torch.bfloat16, device="cuda")
    layer = torch.empty(size, ins, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(tokens, size, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(vocab, size, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(tokens, dtype=torch.int64, device="cuda")
    g = torch.empty(tokens, device="cuda")
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    dh = torch.empty_like(h)
    shapes = [(vocab, size), (size, ins)]
    grads = [[torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in shapes] for _ in range(W)]
    plan = tide.Plan(W, shapes)
    shards = [torch.zeros(plan.shard_elems, device="cuda") for _ in range(W)]
    c, s = tide.checkpoint_layout(ins)
    codes = torch.empty(tokens, c, dtype=torch.int8, device="cuda")
    scales = torch.empty(tokens, s, dtype=torch.uint8, device="cuda")
    calls = [tide.checkpoint_pack_call(x, codes, scales),
             tide.vocab_loss_grad_call(h, w, t, g, loss, lse, dh, grads[0][0]),
             tide.checkpoint_weight_grad_call(dh, codes, scales, grads[0][1]),
             tide.reduce_scatter_call(plan, grads, shards)]
    side = torch.cuda.Stream()

    def fill():
        x.copy_(torch.from_numpy(rng.standard_normal((tokens, ins))))
        layer.copy_(torch.from_numpy(rng.standard_normal((size, ins)) * ins**-0.5))
        hh, ww, tt, gg = make(rng, tokens, size, vocab, rng.choice([0.0, 0.3]))
        h.copy_(hh)
        w.copy_(ww)
        t.copy_(torch.from_numpy(tt))
        g.copy_(torch.from_numpy(gg))
        torch.cuda.synchronize()

    def check():
        torch.cuda.synchronize()
        want = ref.vocab_loss(h.double().cpu().numpy(), w.double().cpu().numpy(), t.cpu().numpy(),
                              g.double().cpu().numpy())
        r = Run.__new__(Run)
        r.loss, r.lse, r.dh, r.dw = loss, lse, dh, grads[0][0]
        r.check(want)
        back = ref.unpack(*ref.pack(x.double().cpu().numpy(), "int8"), "int8", ins)
        value, bound = ref.weight_grad(dh.double().cpu().numpy(), back)
        diff = np.abs(grads[0][1].double().cpu().numpy() - value)
        assert (diff <= bound * 1.01 + 2.0**-8 * np.abs(value)).all()
        for r in range(W):
            for p, (o, n) in enumerate(zip(plan.shard_offset, plan.n_real[r])):
                lo = r * int(plan.rows_per_rank[p]) * shapes[p][1]
                part = grads[0][p].flatten()[lo:lo + n].float() + grads[1][p].flatten()[lo:lo + n].float()
                assert torch.equal(shards[r][o:o + n], part)

    fill()
    for call in calls:
        call(side)
    check()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        for call in calls:
            call()
    for _ in range(4):
        fill()
        for out in (loss, lse, dh, grads[0][0], grads[0][1], codes, scales, *shards):
            out.zero_()
        graph.replay()
        check()


def test_two_calls_at_once(tide):
    import torch

    jobs = []
    for k in range(2):
        h, w, t, g = make(np.random.default_rng(20 + k), 400, 64, 3000 + k, 0.1)
        want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
        jobs.append((h.cuda(), w.cuda(), t, g, torch.cuda.Stream(), want))
    torch.cuda.synchronize()
    runs = []
    for _ in range(5):
        for h, w, t, g, stream, want in jobs:
            runs.append((Run.__new__(Run), want))
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                runs[-1][0].__init__(tide, h, w, t, g)
    torch.cuda.synchronize()
    for r, want in runs:
        r.check(want)


def test_results_repeat_bit_for_bit(tide):
    import torch

    h, w, t, g = make(np.random.default_rng(30), 500, 128, 5000, 0.2)
    need = tide.vocab_loss_workspace(h.cuda(), w.cuda(), torch.empty(5000, 128, device="cuda"))
    runs = []
    for k in range(3):
        ws = torch.full((need,), 255 * (k & 1), dtype=torch.uint8, device="cuda")
        runs.append(Run(tide, h, w, t, g, "f32", workspace=ws))
    for r in runs[1:]:
        for name in ("loss", "lse", "dh", "dw"):
            assert torch.equal(getattr(r, name), getattr(runs[0], name))


def test_binding_refusals(tide):
    import torch

    def tensors(**change):
        a = dict(h=torch.zeros(4, 16, dtype=torch.bfloat16), w=torch.zeros(9, 16, dtype=torch.bfloat16),
                 t=torch.zeros(4, dtype=torch.int64), g=torch.zeros(4), loss=torch.zeros(4), lse=torch.zeros(4),
                 dh=torch.zeros(4, 16, dtype=torch.bfloat16), dw=torch.zeros(9, 16))
        a.update(change)
        return [x.cuda() for x in a.values()]  # one that is on the GPU keeps its strides

    bad = [dict(h=torch.zeros(4, 16)), dict(w=torch.zeros(9, 15, dtype=torch.bfloat16)),
           dict(t=torch.zeros(4, dtype=torch.int32)), dict(t=torch.zeros(5, dtype=torch.int64)), dict(g=torch.zeros(3)),
           dict(loss=torch.zeros(4, dtype=torch.bfloat16)), dict(lse=torch.zeros(2)),
           dict(dh=torch.zeros(4, 16)), dict(dh=torch.zeros(4, 24, dtype=torch.bfloat16, device="cuda")[:, :16]),
           dict(dw=torch.zeros(8, 16)), dict(dw=torch.zeros(9, 16, dtype=torch.float16)),
           dict(h=torch.zeros(16, 4, dtype=torch.bfloat16).t())]
    for change in bad:
        with pytest.raises((TypeError, ValueError)):
            tide.vocab_loss_grad(*tensors(**change))
    h, w, t, g, loss, lse, dh, dw = tensors()
    with pytest.raises(tide.TideError):
        tide.vocab_loss_grad(h, w, t, g, loss, lse, dh, dw, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tide.TideError):
        tide.vocab_loss(h, w[:0], t, loss)
