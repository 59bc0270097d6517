"""GPU checks of the training-step operators at the largest sizes a launch's
32-bit thread count and a grid's limits could be passed at."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def test_no_tokens_and_a_gradient_above_16_gib(tide):
    """No tokens: dweight is set to 0 throughout, and nothing behind it."""
    import torch

    vocab, size = (1 << 21) + 3, 4099
    dw = torch.ones(vocab * size + 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, device="cuda")
    tide.vocab_loss_grad(torch.empty(0, size, dtype=torch.bfloat16, device="cuda"),
                         torch.empty(vocab, size, dtype=torch.bfloat16, device="cuda"),
                         torch.empty(0, dtype=torch.int64, device="cuda"), none, none, None,
                         torch.empty(0, size, dtype=torch.bfloat16, device="cuda"), dw[:vocab * size].view(vocab, size))
    torch.cuda.synchronize()
    for part in dw[:vocab * size].split(1 << 30):
        assert not bool(part.view(torch.int16).any())
    assert bool((dw[vocab * size:] == 1).all())


def test_the_most_tokens_of_a_small_vocabulary(tide):
    """2^24 tokens, a workgroup for each row of a piece."""
    import torch

    tokens, size, vocab = 1 << 24, 8, 5
    gen = torch.Generator("cuda").manual_seed(24)
    h = torch.randn(tokens, size, generator=gen, device="cuda").bfloat16()
    w = torch.randn(vocab, size, generator=gen, device="cuda").bfloat16()
    t = torch.randint(-1, vocab, (tokens,), generator=gen, device="cuda")
    g = torch.rand(tokens, generator=gen, device="cuda")
    loss, lse = (torch.full((tokens,), float("nan"), device="cuda") for _ in range(2))
    dh = torch.full((tokens, size), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((vocab, size), float("nan"), device="cuda")
    tide.vocab_loss_grad(h, w, t, g, loss, lse, dh, dw)
    torch.cuda.synchronize()
    counts = t >= 0
    z = h.double() @ w.double().t().contiguous()
    want = torch.logsumexp(z, -1)
    tt = t.clamp(min=0)[:, None]
    p = torch.exp(z - want[:, None]).scatter_add(1, tt, torch.full((tokens, 1), -1.0, dtype=torch.float64, device="cuda"))
    p *= (g.double() * counts)[:, None]
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    want_loss = torch.where(counts, want - z.gather(1, tt)[:, 0], zero)
    # sums of 8 products and 5 exponentials in fp32, of magnitudes below 64
    assert float((lse.double() - torch.where(counts, want, zero)).abs().max()) < 2.0**-14
    assert float((loss.double() - want_loss).abs().max()) < 2.0**-14
    # dz rounded by at most 2^-8 of each of its 5 terms, then the result by 2^-9 of
    # itself (2^-8 counts for both halves), and a term's own fp32 error
    terms = p.abs() @ w.double().abs()
    err = (dh.double() - p @ w.double()).abs()
    assert float((err - terms * 2.0**-7 - 2.0**-14).max()) < 0
    # 2^19 steps of 32 tokens, each partial sum (at most the sum of the magnitudes)
    # rounded in fp32, 2^-23 with truncation: 2^-4 at the very worst
    terms = p.abs().t().contiguous() @ h.double().abs()
    assert bool(((dw.double() - p.t().contiguous() @ h.double()).abs() < terms * 2.0**-4).all())
