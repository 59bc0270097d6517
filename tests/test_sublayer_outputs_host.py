"""Calls whose outputs are the same memory are refused (no GPU: nothing is
launched)."""
import pytest

P = 0x7F0000000000


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


def test_mean_and_rstd(tide):
    Q = P + (1 << 20)
    got = tide.lib.tide_layer_norm(P, 0, 64, 10, 64, None, None, 1, 1e-5, Q, 0, 64, P, P, None)
    assert got == -1 and b"same vector" in tide.lib.tide_last_error()


def test_dweight_and_dbias(tide):
    got = tide.lib.tide_layer_norm_grad(P, 0, 64, P, 0, 64, 10, 64, P, 1, P, P, P, 64, P, P, 0, P, 1 << 30, None)
    assert got == -1 and b"same vector" in tide.lib.tide_last_error()


@pytest.mark.parametrize("tokens", [5, 300])
def test_the_weights_gradients(tide, tokens):
    got = tide.lib.tide_gated_block_grad(P, 96, P, 64, P, 64, P, 64, tokens, 64, 96, 0, None, 192, P, 64, P, P, 0, 0, P,
                                         1 << 40, None)
    assert got == -1 and b"same matrix" in tide.lib.tide_last_error()


def test_updates(tide):
    import ctypes

    two = (ctypes.c_void_p * 2)
    got = tide.lib.tide_orthogonalize(two(P, P + 4096), 0, 64, two(P + 8192, P + 8192), 64, 2, 8, 64, 5, 3.4445, -4.775,
                                      2.0315, 1e-7, P, 1 << 40, None)
    assert got == -1 and b"same matrix" in tide.lib.tide_last_error()
