"""Registered calls of the operators with a workspace (no GPU: the library's
launches and the device's parts of the binding are replaced)."""
import os
import subprocess
import sys
import types

import pytest


@pytest.fixture
def tide(monkeypatch):
    from param_collectives_amd import tide

    monkeypatch.setattr(tide, "_on_device", lambda t, what: None)
    monkeypatch.setattr(tide, "_current_device", lambda: 0, raising=False)
    return tide


def registered(tide, name, workspace=None):
    """A registered call on host tensors that needs a workspace."""
    import torch

    tokens, size, vocab = 300, 40, 70
    h, w = torch.zeros(tokens, size, dtype=torch.bfloat16), torch.zeros(vocab, size, dtype=torch.bfloat16)
    t, loss = torch.zeros(tokens, dtype=torch.int64), torch.zeros(tokens)
    if name == "tide_vocab_loss":
        return tide.vocab_loss_call(h, w, t, loss, workspace=workspace)
    if name == "tide_vocab_loss_grad":
        return tide.vocab_loss_grad_call(h, w, t, torch.zeros(tokens), loss, None, torch.zeros_like(h),
                                         torch.zeros_like(w), workspace=workspace)
    c, s = tide.checkpoint_layout(size)
    return tide.checkpoint_weight_grad_call(torch.zeros(tokens, 7, dtype=torch.bfloat16),
                                            torch.zeros(tokens, c, dtype=torch.int8),
                                            torch.zeros(tokens, s, dtype=torch.uint8), torch.zeros(7, size),
                                            workspace=workspace)


CALLS = ["tide_checkpoint_weight_grad", "tide_vocab_loss", "tide_vocab_loss_grad"]


@pytest.mark.parametrize("name", CALLS)
def test_a_launch_takes_its_workspace_on_its_own_stream(tide, monkeypatch, name):
    """Not when the call is made, on whichever stream is current then: freed, it
    would go back to that stream while a launch on another still uses it."""
    import torch

    taken, launched = [], []

    def workspace(nbytes, given, stream):
        assert given is None and nbytes > 0
        t = torch.empty(nbytes, dtype=torch.uint8)
        taken.append((stream, t.data_ptr()))
        return t.data_ptr(), nbytes, t

    monkeypatch.setattr(tide, "_workspace", workspace)
    monkeypatch.setattr(tide.lib, name, lambda *a: launched.append(a[-3:]) or 0)
    call = registered(tide, name)
    assert not taken
    streams = [types.SimpleNamespace(cuda_stream=0x1000 * (k + 1)) for k in range(2)]
    for s in (*streams, streams[0]):
        call(s)
    assert [s for s, _ in taken] == [*streams, streams[0]]
    for (s, at), (ws, _, handle) in zip(taken, launched):
        assert ws == at and getattr(handle, "value", handle) == s.cuda_stream


@pytest.mark.parametrize("name", CALLS)
def test_the_callers_workspace_serves_every_launch(tide, monkeypatch, name):
    import torch

    launched = []
    monkeypatch.setattr(tide.lib, name, lambda *a: launched.append(a[-3:-1]) or 0)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    call = registered(tide, name, ws)
    for _ in range(2):
        call(types.SimpleNamespace(cuda_stream=0x1000))
    assert launched == [(ws.data_ptr(), 1 << 20)] * 2
    with pytest.raises(TypeError):
        registered(tide, name, ws.view(torch.int32))


ALL_CALLS = ["tide_checkpoint_pack", "tide_checkpoint_unpack", *CALLS]


@pytest.mark.parametrize("name", ALL_CALLS)
def test_launches_on_another_device_are_refused(tide, monkeypatch, name):
    """The tensors are checked when the call is made; a launch would take its
    stream from the device that is current then."""
    import torch

    launched = []
    monkeypatch.setattr(tide.lib, name, lambda *a: launched.append(a) or 0)
    x, codes, scales = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    here = types.SimpleNamespace(cuda_stream=0x1000, device_index=0)
    there = types.SimpleNamespace(cuda_stream=0x2000, device_index=1)
    if name == "tide_checkpoint_pack":
        call = tide.checkpoint_pack_call(x, codes, scales)
        once = lambda s: tide.checkpoint_pack(x, codes, scales, stream=s)
    elif name == "tide_checkpoint_unpack":
        call = tide.checkpoint_unpack_call(codes, scales, x)
        once = lambda s: tide.checkpoint_unpack(codes, scales, x, stream=s)
    else:
        call = once = registered(tide, name, ws)
    call(here)
    once(here)
    assert len(launched) == 2
    for launch in (call, once):
        with pytest.raises(ValueError, match="device"):
            launch(there)
    monkeypatch.setattr(tide, "_current_device", lambda: 1)
    for stream in (here, there):
        with pytest.raises(ValueError, match="device"):
            call(stream)
    assert len(launched) == 2


def test_public_torch_calls_where_the_private_ones_are_missing():
    code = """
import types
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    delattr(torch._C, name)
from param_collectives_amd import tide
assert tide._current_device is torch.cuda.current_device
torch.cuda.current_device = lambda: 0
torch.cuda.current_stream = lambda device: types.SimpleNamespace(cuda_stream=0x5000 + device)
assert tide._stream_handle(None) == 0x5000
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)


def test_the_layouts_kept_are_bounded():
    from param_collectives_amd import tide

    for cols in range(2000):
        blocks = -(-cols // 32)
        assert tide.checkpoint_layout(cols) == (32 * blocks, blocks)
    assert tide.checkpoint_layout.cache_info().currsize <= 256
