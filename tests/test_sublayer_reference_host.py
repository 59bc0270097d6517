"""The references for large sizes against those for small ones (no GPU)."""
import numpy as np
import pytest
import torch

from tests import sublayer_reference as ref, sublayer_reference_gpu as large


def same(a, b):
    assert np.allclose(np.asarray(a), np.asarray(b), rtol=1e-9, atol=1e-300)


@pytest.mark.parametrize("old", [False, True])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_block(name, old):
    rng = np.random.default_rng(3)
    x, wg, wu, dout = (rng.standard_normal(s) for s in ((5, 7), (6, 7), (6, 7), (5, 6)))
    x[2] = 0.0  # gates of zero
    had = [rng.standard_normal((6, 7)) for _ in range(2)] if old else None
    t = [torch.from_numpy(a) for a in (x, wg, wu, dout)]
    a, b = ref.gated_block(x, wg, wu, name), large.gated_block(*t[:3], name)
    for key in ("out", "gates"):
        same(a[key][0], b[key][0])
        same(a[key][1], b[key][1])
    for gates in (None, a["gates"][0]):
        p = ref.gated_block_grad(dout, x, wg, wu, name, gates, had)
        q = large.gated_block_grad(t[3], *t[:3], name, None if gates is None else torch.from_numpy(gates),
                                   had and [torch.from_numpy(h) for h in had])
        for key in p:
            for v, w in zip(p[key], q[key]):
                same(v, w)


@pytest.mark.parametrize("rows,cols", [(5, 9), (9, 5), (20, 20)])
@pytest.mark.parametrize("f32", [False, True])
def test_orthogonalize(rows, cols, f32):
    x = np.random.default_rng(rows).standard_normal((rows, cols))
    abc, eps = (3.4445, -4.7750, 2.0315), 1e-7
    value, tolerance = ref.orthogonalize(x, 5, *abc, eps, f32=f32)
    got, error = large.orthogonalize(torch.from_numpy(x), 5, *abc, eps, f32=f32)
    assert np.allclose(got.numpy(), value, rtol=1e-9, atol=1e-12)
    norm = np.linalg.norm(value)
    assert tolerance == pytest.approx(1.5 * (float(error.norm()) + ref.HALF["bf16"] / np.sqrt(3) * norm) + 2.0**-20 * norm, rel=1e-6)


def test_an_element_out_of_its_bound():
    value, err = torch.ones(3, 4, dtype=torch.float64), torch.full((3, 4), 1e-9, dtype=torch.float64)
    good = value.bfloat16()
    large.close(good, value, err, "bf16", "good")
    bad = good.clone()
    bad[2, 1] = 1.0 + 2.0**-6
    for wrong in (bad, torch.full_like(good, float("nan"))):
        with pytest.raises(AssertionError, match="wrong"):
            large.close(wrong, value, err, "bf16", "wrong")
