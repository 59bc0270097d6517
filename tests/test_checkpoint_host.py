"""Host-side checks of the 8-bit activation checkpoints (no GPU): the layout,
and every refusal, made before any device work (the addresses passed here are
not device memory)."""
import ctypes

import numpy as np
import pytest

from tests import training_reference as ref

INVALID, RANGE, ALIGN = -1, -2, -3
P = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def tide():
    from param_collectives_amd import tide

    return tide


@pytest.mark.parametrize("cols,want", [(0, (0, 0)), (1, (32, 1)), (32, (32, 1)), (33, (64, 2)), (1000, (1024, 32)),
                                       (1 << 22, (1 << 22, 1 << 17))])
def test_layout(tide, cols, want):
    assert tide.checkpoint_layout(cols) == want


def test_layout_refusals(tide):
    for cols, status in ((-1, INVALID), ((1 << 22) + 1, RANGE)):
        with pytest.raises(tide.TideError) as e:
            tide.checkpoint_layout(cols)
        assert e.value.status == status
    assert tide.lib.tide_checkpoint_layout(33, None, None) == 0


PACK = dict(x=P, dtype=1, rows=4, cols=64, stride=64, fmt=0, codes=P, scales=P)
PACK_REFUSED = [
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(fmt=2), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=-1), INVALID), (dict(stride=63), INVALID), (dict(rows=1 << 31), RANGE),
    (dict(cols=(1 << 22) + 1, stride=(1 << 22) + 1), RANGE), (dict(stride=(1 << 22) + 1), RANGE),
    (dict(rows=1 << 20, cols=1 << 15, stride=1 << 15), RANGE), (dict(x=0), INVALID), (dict(codes=0), INVALID),
    (dict(scales=0), INVALID), (dict(x=P + 2), ALIGN), (dict(x=P + 1, dtype=0), ALIGN), (dict(codes=P + 8), ALIGN),
]


@pytest.mark.parametrize("change,status", PACK_REFUSED)
def test_pack_and_unpack_refusals(tide, change, status):
    a = {**PACK, **change}
    got = tide.lib.tide_checkpoint_pack(a["x"] or None, a["dtype"], a["rows"], a["cols"], a["stride"], a["fmt"],
                                        a["codes"] or None, a["scales"] or None, None)
    assert got == status and tide.lib.tide_last_error()
    got = tide.lib.tide_checkpoint_unpack(a["codes"] or None, a["scales"] or None, a["fmt"], a["rows"], a["cols"],
                                          a["x"] or None, a["dtype"], a["stride"], None)
    assert got == status and tide.lib.tide_last_error()


def test_short_rows_count_with_their_filling(tide):
    # 2^31 - 1 rows of one value take 32 codes each, and 64 elements in an aligned copy
    for rows, status in (((1 << 31) - 1, RANGE), ((1 << 28) + 1, RANGE), (1 << 28, INVALID)):
        assert tide.lib.tide_checkpoint_pack(None, 1, rows, 1, 1, 0, P, P, None) == status
        assert tide.lib.tide_checkpoint_unpack(P, P, 0, rows, 1, None, 1, 1, None) == status
        need = ctypes.c_int64()
        assert tide.lib.tide_checkpoint_weight_grad_workspace(None, rows, 1, 1, 64, ctypes.byref(need)) == status


def test_empty_matrices_need_no_pointers(tide):
    for rows, cols in ((0, 64), (4, 0), (0, 0)):
        assert tide.lib.tide_checkpoint_pack(None, 1, rows, cols, cols, 0, None, None, None) == 0
        assert tide.lib.tide_checkpoint_unpack(None, None, 0, rows, cols, None, 1, cols, None) == 0
    assert tide.lib.tide_checkpoint_weight_grad(None, 4, 0, 0, None, None, 0, 8, None, 1, 1.0, 0, None, 0, None) == 0
    assert tide.lib.tide_checkpoint_weight_grad(None, 4, 8, 8, None, None, 0, 0, None, 1, 1.0, 0, None, 0, None) == 0


# dy's rows are not aligned, so every call that is not refused earlier needs a workspace
GRAD = dict(dy=P, rows=1000, outs=64, stride=65, codes=P, scales=P, fmt=0, ins=64, dw=P, dtype=1, acc=0, ws=P,
            ws_bytes=1 << 30)
GRAD_REFUSED = [
    (dict(fmt=7), INVALID), (dict(dtype=3), INVALID), (dict(acc=2), INVALID), (dict(rows=-1), INVALID),
    (dict(outs=-1), INVALID), (dict(ins=-1), INVALID), (dict(stride=10), INVALID), (dict(rows=1 << 31), RANGE),
    (dict(ins=(1 << 22) + 1), RANGE), (dict(outs=1 << 18, stride=1 << 18, ins=1 << 17, rows=1), RANGE),
    (dict(dy=0), INVALID), (dict(dw=0), INVALID), (dict(codes=0), INVALID), (dict(scales=0), INVALID),
    (dict(dy=P + 1), ALIGN), (dict(dw=P + 2), ALIGN), (dict(codes=P + 4), ALIGN), (dict(ws=0), INVALID),
    (dict(ws=P + 128), ALIGN), (dict(ws_bytes=1), INVALID),
]


@pytest.mark.parametrize("change,status", GRAD_REFUSED)
def test_weight_grad_refusals(tide, change, status):
    a = {**GRAD, **change}
    got = tide.lib.tide_checkpoint_weight_grad(
        a["dy"] or None, a["rows"], a["outs"], a["stride"], a["codes"] or None, a["scales"] or None, a["fmt"],
        a["ins"], a["dw"] or None, a["dtype"], 1.0, a["acc"], a["ws"] or None, a["ws_bytes"], None)
    assert got == status and tide.lib.tide_last_error()


def test_weight_grad_workspace(tide):
    need = ctypes.c_int64(-1)
    fn = tide.lib.tide_checkpoint_weight_grad_workspace
    assert fn(P, 100, 64, 64, 64, None) == INVALID
    assert fn(P, 100, 64, 10, 64, ctypes.byref(need)) == INVALID and need.value == -1
    # one tile row of few tokens: neither splits nor a copy of dy
    assert fn(P, 100, 64, 64, 64, ctypes.byref(need)) == 0 and need.value == 0
    # dy's rows do not all start on 16 bytes: a copy of pitch 64 (a multiple of 64)
    assert fn(P, 100, 63, 63, 64, ctypes.byref(need)) == 0 and need.value == 100 * 64 * 2
    assert fn(P + 2, 100, 64, 64, 64, ctypes.byref(need)) == 0 and need.value == 100 * 64 * 2
    # many tokens, one tile: split, each split with an fp32 matrix
    assert fn(P, 64 * 64, 64, 64, 64, ctypes.byref(need)) == 0
    assert need.value > 0 and need.value % (64 * 64 * 4) == 0


def test_binding_refuses_host_tensors(tide):
    import torch

    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        tide.checkpoint_pack(x, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        tide.checkpoint_unpack(None, None, x.numpy())


def test_reference_round_trip_bounds():
    """The reference keeps the header's bounds: 2^-4 of the value or 2^-10
    units (e4m3), half a unit (int8)."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 320)) * 10.0 ** rng.uniform(-3, 3, (64, 320))
    for fmt in ("e4m3", "int8"):
        codes, scales = ref.pack(x, fmt)
        y = ref.unpack(codes, scales, fmt, 320)
        u = np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1)
        bound = u / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0**-4, u * 2.0**-10)
        assert (np.abs(x - y) <= bound).all()
