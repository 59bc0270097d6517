"""GPU checks of layer norm on rows at the end of bf16's range: their sums leave
it, their means do not."""
import numpy as np
import pytest

from tests import sublayer_reference as ref
from tests.test_gpu_checkpoint import device
from tests.test_gpu_layer_norm import EPS, close, nan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from param_collectives_amd import tide

    return tide


# columns that 16 lanes, a wave and workgroups of 256 and 512 share, that loops read; powers of two have an exact mean
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [2, 3, 40, 128, 200, 700, 1024, 2048, 3000, 4096, 6200, 8192, 9000, 16384, 16385, 20000])
def test_rows_of_one_large_value(tide, cols, xt):
    """bf16 and fp32 rows of numbers near 2^127 come out by the formula: no deviation,
    the mean exact."""
    x = np.repeat(np.array([[2.0**127], [-(2.0**127)], [1.9921875 * 2.0**127], [2.0**126], [-1.5 * 2.0**123], [1.0]]), cols, 1)
    w, b = np.ones(cols), np.random.default_rng(cols).standard_normal(cols).astype(np.float32).astype(np.float64)
    out, mean, rstd = nan(x.shape, "f32"), nan((len(x),), "f32"), nan((len(x),), "f32")
    tide.layer_norm(device(x, xt), device(w, "f32"), device(b, "f32"), out, mean, rstd, eps=EPS)
    want = ref.layer_norm(x, w, b, EPS)
    assert (mean.double().cpu().numpy() == x[:, 0]).all()
    assert (abs(rstd.double().cpu().numpy() * EPS**0.5 - 1) < 8 * 2.0**-24).all()
    close(out, want["out"], "f32", "out")
    if cols & (cols - 1) == 0:
        assert (out.double().cpu().numpy() == b).all()
