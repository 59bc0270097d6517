"""GPU checks of how the training-step operators' products are cut: whole rounds
of tiles with the rest split along k, several rounds of tiles in resident
workgroups, the few-token kernel's blocks, and streams that hold only some of
the CUs; against 64-bit references, the large ones computed on the GPU."""
import numpy as np
import pytest

from tests import training_reference as ref
from tests.test_gpu_vocab_loss import Run, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


# tokens, out features, in features: 272 large tiles, the 16 beyond a round
# split in 4; 384, split in 2; a round of small tiles split many times; a
# token count that ends inside a split's last step
CUTS = [(4096, 4096, 4352), (4500, 6144, 4096), (5000, 200, 300), (4097, 130, 4000), (2081, 512, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("tokens,outs,ins", CUTS)
def test_weight_grad_cuts(tide, tokens, outs, ins, fmt, dtype):
    import torch

    g = torch.Generator(device="cuda").manual_seed(tokens)
    dy = (torch.randn(tokens, outs, device="cuda", generator=g) * 1e-2).bfloat16()
    x = torch.randn(tokens, ins, device="cuda", generator=g)
    c, s = tide.checkpoint_layout(ins)
    codes = torch.empty(tokens, c, dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(tokens, s, dtype=torch.uint8, device="cuda")
    back = torch.empty_like(x)
    tide.checkpoint_pack(x, codes, scales)
    tide.checkpoint_unpack(codes, scales, back)
    dw = torch.full((outs, ins), float("nan"), dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    tide.checkpoint_weight_grad(dy, codes, scales, dw)
    y, X = dy.double(), back.double()
    want = torch.matmul(y.t().contiguous(), X)
    # the exact products' sum in any order, each addition off by 2^-23 at most (a truncating adder)
    bound = (tokens + 64) * 2.0**-23 * torch.matmul(y.abs().t().contiguous(), X.abs())
    half = 2.0**-24 if dtype == "f32" else 2.0**-8
    diff = (dw.double() - want).abs()
    assert (diff <= bound * (1 + half) + half * want.abs()).all()
    # and together far closer: 2^-23 of the magnitudes' root mean square per addition
    mean = torch.sqrt(torch.matmul((y * y).t().contiguous(), X * X))
    assert float(diff.norm()) <= float((mean * tokens**0.5 * 2.0**-23).norm() + half * want.norm())


def loss_on_gpu(h, w, t, g):
    """loss, dhidden, dweight in 64 bits, the tokens 1024 at a time."""
    import torch

    H, Wd = h.double().cuda(), w.double().cuda()
    keep = np.nonzero((t >= 0) & (t < w.shape[0]))[0]
    loss = torch.zeros(h.shape[0], dtype=torch.float64, device="cuda")
    dh, dw = torch.zeros_like(H), torch.zeros_like(Wd)
    for k0 in range(0, len(keep), 1024):
        k = torch.from_numpy(keep[k0:k0 + 1024]).cuda()
        tt, gg = torch.from_numpy(t[keep[k0:k0 + 1024]]).cuda(), torch.from_numpy(g).double().cuda()[k]
        z = H[k] @ Wd.t().contiguous()
        lse = torch.logsumexp(z, -1)
        i = torch.arange(len(k), device="cuda")
        loss[k] = lse - z[i, tt]
        p = torch.exp(z - lse[:, None])
        p[i, tt] -= 1.0
        p *= gg[:, None]
        dh[k] = p @ Wd
        dw += p.t().contiguous() @ H[k]
    return loss, dh, dw


# tokens, hidden, vocabulary, left out: 432 and 1044 large tiles of logits with
# a hidden size that ends inside a step; 548 large tiles of dW; 272 of dH, the
# rest split; 24 of dH split many times; 512-slot rounds of small tiles
ROUNDS = [(2900, 100, 9000, 0.0), (7400, 72, 9100, 0.3), (300, 512, 70000, 0.1), (4352, 4096, 4200, 0.0),
          (700, 2048, 50000, 0.4), (400, 64, 30000, 0.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,size,vocab,ignored", ROUNDS)
def test_vocab_loss_rounds(tide, tokens, size, vocab, ignored, dtype):
    h, w, t, g = make(np.random.default_rng(tokens), tokens, size, vocab, ignored)
    loss, dh, dw = loss_on_gpu(h, w, t, g)
    r = Run(tide, h, w, t, g, dtype)
    only = Run(tide, h, w, t, None)
    # a logit's products and the row's exponentials in fp32: sums of up to 4096
    # terms of magnitude up to ~20, 2^-23 each with truncation, far below 2^-9
    for x in (r, only):
        assert float((x.loss.double() - loss).abs().max()) < 2.0**-9
    # dz rounded by 2^-8 at most (2^-8 / sqrt(3) in the mean square), the bf16 results once more
    for got, want in ((r.dh, dh), (r.dw, dw)):
        assert float((got.double() - want).norm() / want.norm()) < 2.0**-8 * (2 / 3) ** 0.5 * 1.2
        # no tile is off by itself
        rows = (got.double() - want).norm(dim=1) / (want.norm(dim=1) + want.norm() * 1e-3)
        assert float(rows.max()) < 2.0**-5


@pytest.mark.parametrize("tokens", [5, 16, 33, 48, 64])
@pytest.mark.parametrize("size", [8, 248, 256, 512, 776, 1024, 1300])
def test_few_tokens(tide, tokens, size):
    """One to four fragments of tokens, none to five blocks of 256 k with and
    without a rest, vocabularies that end inside a wave's rows."""
    h, w, t, g = make(np.random.default_rng(size + tokens), tokens, size, 333, 0.2)
    want = ref.vocab_loss(h.double().numpy(), w.double().numpy(), t, g.astype(float))
    Run(tide, h, w, t, None).check(want)
    Run(tide, h, w, t, g).check(want)


def test_streams_that_hold_some_cus(tide):
    """On a stream masked to 24 CUs the results are those of the whole GPU."""
    import torch

    h, w, t, g = make(np.random.default_rng(1), 2000, 128, 9000, 0.1)
    whole = Run(tide, h, w, t, g, "f32")
    dy = torch.randn(3000, 300, device="cuda").bfloat16()
    c, s = tide.checkpoint_layout(500)
    codes = torch.randint(-127, 128, (3000, c), dtype=torch.int8, device="cuda")
    scales = torch.full((3000, s), 121, dtype=torch.uint8, device="cuda")
    dw = [torch.full((300, 500), float("nan"), device="cuda") for _ in range(2)]
    tide.checkpoint_weight_grad(dy, codes, scales, dw[0])
    torch.cuda.synchronize()
    stream = tide.Stream(cus=range(24))
    some = Run(tide, h.cuda(), w.cuda(), t, g, "f32", stream=stream.torch)
    tide.checkpoint_weight_grad(dy, codes, scales, dw[1], stream=stream.torch)
    torch.cuda.synchronize()
    for name in ("loss", "lse", "dh", "dw"):
        assert torch.equal(getattr(some, name), getattr(whole, name)), name
    assert torch.equal(dw[0], dw[1])
    stream.destroy()


def test_weight_grad_pieces_in_rounds(tide):
    """160 large tiles, split in 3: 480 pieces, two rounds."""
    for fmt, dtype in (("e4m3", "bf16"), ("int8", "f32")):
        test_weight_grad_cuts(tide, 21999, 2560, 4090, fmt, dtype)


def test_vocab_loss_pieces_in_rounds(tide):
    """The same for dH; the tokens that count decide it."""
    test_vocab_loss_rounds(tide, 2560, 4096, 22001, 0.0, "bf16")
    test_vocab_loss_rounds(tide, 2900, 4096, 22001, 0.12, "f32")
