"""The largest sizes of the gated block (no GPU: nothing is launched)."""
import ctypes

import pytest

RANGE = -2
P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


def workspace(tide, tokens, ffn, grad, gates):
    need = ctypes.c_int64(-1)
    st = tide.lib.tide_gated_block_workspace(P, 64, P, 64, P, 64, tokens, 64, ffn, grad, gates, ctypes.byref(need))
    return need.value if st == 0 else st


def test_the_limit_is_that_of_the_matrices_there_are(tide):
    """out of up to 2^34 elements; gates, or the dg and du that the gradients keep in
    their workspace, have twice as many."""
    for tokens, ffn in ((1 << 20, 1 << 14), ((1 << 20) - 5, (1 << 14) - 3), (600_000, 16384)):
        assert workspace(tide, tokens, ffn, 0, None) >= 0
        for grad, gates in ((0, P), (1, None), (1, P)):
            assert workspace(tide, tokens, ffn, grad, gates) == RANGE
    assert workspace(tide, 1 << 19, 1 << 14, 0, P) >= 0 and workspace(tide, 1 << 19, 1 << 14, 1, P) > 0
    assert workspace(tide, (1 << 20) + 1, 1 << 14, 0, None) == RANGE
