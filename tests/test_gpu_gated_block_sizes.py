"""GPU check of the gated block at an out of more than 2^33 elements, whose gates
would have more than 2^34 and are not asked for."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def test_more_than_2_33_elements(tide):
    import torch

    from tests import sublayer_reference_gpu as ref

    tokens, hidden, ffn = 530_003, 40, 16392
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").bfloat16()
    wg, wu = ((torch.randn(ffn, hidden, generator=gen, device="cuda") * hidden**-0.5).bfloat16() for _ in range(2))
    out = torch.full((tokens, ffn), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert tokens * ffn > 2**33 and 2 * tokens * ffn > 2**34
    tide.gated_block(x, wg, wu, out)
    # the first rows, those around 2^32 and 2^33 elements, the last
    for first in (0, 2**32 // ffn - 20, 2**33 // ffn - 20, tokens - 40):
        rows = slice(first, first + 40)
        want = ref.gated_block(x[rows].double(), wg.double(), wu.double(), "silu")
        ref.close(out[rows], *want["out"], "bf16", first)
    for first in range(0, tokens, 50_000):
        assert bool(out[first:first + 50_000].isfinite().all())
