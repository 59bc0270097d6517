"""Host-side checks of the gated block (no GPU): every refusal, made before any
device work (the addresses passed here are not device memory), its workspace,
and the 64-bit reference against differences."""
import ctypes

import numpy as np
import pytest

from tests import sublayer_reference as ref

INVALID, RANGE, ALIGN = -1, -2, -3
P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


CALL = dict(x=P, x_ld=64, g=P, g_ld=64, u=P, u_ld=64, tokens=300, size=64, ffn=96, act=0, out=P, out_ld=96, gates=P,
            gates_ld=192, ws=P, ws_bytes=1 << 40)
WIDE = (1 << 22) + 1
REFUSED = [
    (dict(x=0), INVALID), (dict(g=0), INVALID), (dict(u=0), INVALID), (dict(tokens=-1), INVALID),
    (dict(size=0, x_ld=0, g_ld=0, u_ld=0), INVALID), (dict(ffn=0), INVALID), (dict(ffn=-1), INVALID),
    (dict(x_ld=63), INVALID), (dict(g_ld=63), INVALID), (dict(u_ld=63), INVALID), (dict(gates_ld=191), INVALID),
    (dict(act=2), INVALID), (dict(act=-1), INVALID), (dict(tokens=1 << 31), RANGE),
    (dict(size=WIDE, x_ld=WIDE, g_ld=WIDE, u_ld=WIDE), RANGE), (dict(u_ld=WIDE), RANGE),
    (dict(ffn=(1 << 21) + 1, out_ld=1 << 22, gates_ld=1 << 22, y_ld=1 << 22), RANGE),
    (dict(tokens=1 << 29, y_ld=96), RANGE), (dict(x=P + 1), ALIGN), (dict(g=P + 1), ALIGN), (dict(u=P + 1), ALIGN),
    (dict(gates=P + 1), ALIGN),
]
FORWARD = REFUSED + [(dict(out=0), INVALID), (dict(out_ld=95), INVALID), (dict(out=P + 1), ALIGN)]
GRAD = dict(CALL, dy=P, y_ld=96, dx=P, dx_ld=64, dg=P, du=P, dtype=0, acc=0)
BACKWARD = REFUSED + [
    (dict(dy=0), INVALID), (dict(dx=0), INVALID), (dict(dg=0), INVALID), (dict(du=0), INVALID), (dict(y_ld=95), INVALID),
    (dict(dx_ld=63), INVALID), (dict(dtype=2), INVALID), (dict(acc=2), INVALID), (dict(ws=0), INVALID),
    (dict(ws_bytes=64), INVALID), (dict(ws=P + 64), ALIGN), (dict(dy=P + 1), ALIGN), (dict(dx=P + 1), ALIGN),
    (dict(dg=P + 1), ALIGN), (dict(du=P + 2, dtype=1), ALIGN),
]


def forward(tide, a):
    return tide.lib.tide_gated_block(a["x"] or None, a["x_ld"], a["g"] or None, a["g_ld"], a["u"] or None, a["u_ld"],
                                     a["tokens"], a["size"], a["ffn"], a["act"], a["out"] or None, a["out_ld"],
                                     a["gates"] or None, a["gates_ld"], a["ws"] or None, a["ws_bytes"], None)


def backward(tide, a):
    return tide.lib.tide_gated_block_grad(a["dy"] or None, a["y_ld"], a["x"] or None, a["x_ld"], a["g"] or None, a["g_ld"],
                                          a["u"] or None, a["u_ld"], a["tokens"], a["size"], a["ffn"], a["act"],
                                          a["gates"] or None, a["gates_ld"], a["dx"] or None, a["dx_ld"], a["dg"] or None,
                                          a["du"] or None, a["dtype"], a["acc"], a["ws"] or None, a["ws_bytes"], None)


@pytest.mark.parametrize("change,status", FORWARD)
def test_refusals(tide, change, status):
    assert forward(tide, {**CALL, **change}) == status and tide.lib.tide_last_error()


@pytest.mark.parametrize("change,status", BACKWARD)
def test_gradient_refusals(tide, change, status):
    assert backward(tide, {**GRAD, **change}) == status and tide.lib.tide_last_error()


def test_no_tokens(tide):
    # nothing to do: no pointers are needed (but the gradients', which stay)
    none = dict(tokens=0, x=0, g=0, u=0, out=0, gates=0, ws=0, dy=0, dx=0, acc=1)
    assert forward(tide, {**CALL, **none}) == 0
    assert backward(tide, {**GRAD, **none}) == 0


def test_workspace(tide):
    need = ctypes.c_int64(-1)

    def size(tokens=8192, hidden=4096, ffn=14336, grad=0, gates=P, ld=None, gate=P, up_ld=None):
        ld = ld or hidden
        st = tide.lib.tide_gated_block_workspace(P, ld, gate, hidden, P, up_ld or hidden, tokens, hidden, ffn, grad,
                                                 gates, ctypes.byref(need))
        return need.value if st == 0 else st

    assert size(grad=2) == INVALID and size(ld=100) == INVALID and size(ffn=0) == INVALID
    queues = 3 * 8 * 64 * 4
    assert size() == queues
    dgates = 8192 * 2 * 14336 * 2
    # dg and du, and at most three rounds of 256 partial tiles
    assert dgates <= size(grad=1) <= dgates + queues + 3 * 256 * 65536 * 4
    assert size(grad=1) == size(grad=1, gates=None)
    # copies of rows that are not on 16 bytes
    assert size(ld=4097) - size() == 8192 * 4096 * 2
    assert size(gate=P + 2) - size() == size(up_ld=4104) - size() == 2 * 14336 * 4096 * 2
    assert size(ffn=14337, grad=1) > 2 * 14368 * 4096 * 2
    # up to 16 tokens the forward pass takes none, wherever the rows start
    assert size(tokens=16, ld=4097, gate=P + 2) == 0
    assert size(tokens=0) == size(tokens=0, grad=1) == 0


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_reference_gradients_against_differences(name):
    rng = np.random.default_rng(5)
    x, wg, wu = rng.standard_normal((3, 5)), rng.standard_normal((4, 5)), rng.standard_normal((4, 5))
    dy = rng.standard_normal((3, 4))
    got = ref.gated_block_grad(dy, x, wg, wu, name)
    kept = ref.gated_block_grad(dy, x, wg, wu, name, ref.gated_block(x, wg, wu, name)["gates"][0])

    def f(x, wg, wu):
        return (ref.gated_block(x, wg, wu, name)["out"][0] * dy).sum()

    for key, t, at in (("dx", x, lambda d: f(x + d, wg, wu) - f(x - d, wg, wu)),
                       ("dw_gate", wg, lambda d: f(x, wg + d, wu) - f(x, wg - d, wu)),
                       ("dw_up", wu, lambda d: f(x, wg, wu + d) - f(x, wg, wu - d))):
        assert np.allclose(got[key][0], kept[key][0], rtol=1e-12, atol=1e-14)
        for i in np.ndindex(t.shape):
            d = np.zeros_like(t)
            d[i] = 1e-5
            assert abs(at(d) / 2e-5 - got[key][0][i]) < 1e-8


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_reference_activation(name):
    """Against torch's, and its derivative against differences."""
    import torch

    z = np.linspace(-30, 30, 4001)
    t = torch.from_numpy(z)
    want = torch.nn.functional.silu(t) if name == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    a, d, _ = ref.act(z, name)
    assert np.allclose(a, want.numpy(), rtol=1e-9, atol=1e-13)
    assert np.allclose((ref.act(z + 1e-6, name)[0] - ref.act(z - 1e-6, name)[0]) / 2e-6, d, atol=1e-7)
