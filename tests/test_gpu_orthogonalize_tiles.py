"""GPU checks of the orthogonalized updates at sizes and counts whose products go
to the largest tiles, and whose lists go in unequal pieces; against 64-bit
references on the GPU with the kernels' roundings put in."""
import math

import pytest

pytestmark = pytest.mark.gpu

ABC, EPS = (3.4445, -4.7750, 2.0315), 1e-7

# count, rows, columns.  G and its polynomial by one round of tiles of 256, both orientations; by more than one, split; X's
# product split; X's product in two rounds of short tiles; a list in two pieces, of which the last is smaller and takes
# other tiles
SIZES = [(24, 1030, 780), (16, 1030, 1040), (4, 3027, 3124), (4, 3089, 2986), (2, 2264, 4049), (2, 3724, 2444), (40, 389, 1218),
         (32, 1544, 388), (51, 1075, 801), (37, 878, 1708), (69, 1459, 524)]


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


def matrix(gen, rows, cols, kind):
    """fp64; of the strong kind a few directions hold most of it."""
    import torch

    def rand(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64, device="cuda")

    x = rand(rows, cols)
    if kind == "strong":
        x += (rand(rows, 6) * torch.logspace(2, 0, 6, dtype=torch.float64, device="cuda")) @ rand(6, cols)
    return x * 1e-3


def check(out, x, dtype, what):
    """The error's norm within 1.5 times that of the kernels' roundings (the rule of
    tests/sublayer_reference.py) and of the result's own; of every 16 rows and columns,
    which have a sixteen-th of their number of its square on the average, within 4
    times their share."""
    from tests import sublayer_reference_gpu as ref

    value, error = ref.orthogonalize(x, 5, *ABC, EPS, f32=dtype == "f32")
    off = out.double() - value
    norm = float(value.norm())
    expected = float(error.norm()) + 2.0**-8 / math.sqrt(3) * norm
    assert float(off.norm()) <= 1.5 * expected + 2.0**-20 * norm, (what, float(off.norm()), expected, norm)
    for side in range(2):
        n = value.shape[side]
        for first in range(0, n, 16):
            band = off.narrow(side, first, min(16, n - first))
            share = math.sqrt(band.shape[side] / n)
            own = 2.0**-8 / math.sqrt(3) * float(value.narrow(side, first, band.shape[side]).norm())
            assert float(band.norm()) <= 4 * (share * float(error.norm()) + own) + 2.0**-20 * norm, (what, side, first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("count,rows,cols", SIZES)
def test_sizes(tide, count, rows, cols, dtype):
    import torch

    from tests.sublayer_reference_gpu import held

    gen = torch.Generator("cuda").manual_seed(rows)
    xs = [held(matrix(gen, rows, cols, "strong" if i % 2 else "noise"), dtype) for i in range(count)]
    own = torch.bfloat16 if dtype == "bf16" else torch.float32
    outs = [torch.full((rows, cols), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in xs]
    tide.orthogonalize([x.to(own) for x in xs], outs)
    # both ends of the list and of its halves
    for i in sorted({0, 1, (count - 1) // 2, (count + 1) // 2, count - 2, count - 1}):
        check(outs[i], xs[i], dtype, i)
    assert all(bool(o.isfinite().all()) for o in outs)
