"""Registered calls of layer norm, the gated block and the orthogonalized updates
(no GPU: the library's launches and the device's parts of the binding are
replaced)."""
import types

import pytest


@pytest.fixture
def tide(monkeypatch):
    from param_collectives_amd import tide

    monkeypatch.setattr(tide, "_on_device", lambda t, what: None)
    monkeypatch.setattr(tide, "_current_device", lambda: 0, raising=False)
    return tide


def arguments(name):
    """(name of the binding's function, its arguments) on host tensors; those with a
    workspace need one."""
    import torch

    b = torch.bfloat16
    rows, n, f = 300, 40, 72
    x, v, s = torch.zeros(rows, n, dtype=b), torch.zeros(n), torch.zeros(rows)
    w, h = torch.zeros(f, n, dtype=b), torch.zeros(rows, f, dtype=b)
    return {
        "tide_layer_norm": ("layer_norm", (x, v, v, torch.zeros_like(x), s, s)),
        "tide_layer_norm_grad": ("layer_norm_grad", (x, x, v, s, s, torch.zeros_like(x), torch.zeros(n), torch.zeros(n))),
        # a row of x that ends off 16 bytes needs a copy
        "tide_gated_block": ("gated_block", (x[:, :39], w[:, :39], w[:, :39], h)),
        "tide_gated_block_grad": ("gated_block_grad", (h, x, w, w, torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(w))),
        "tide_orthogonalize": ("orthogonalize", ([w, w], [torch.zeros_like(w), torch.zeros_like(w)])),
    }[name]


CALLS = ["tide_layer_norm_grad", "tide_gated_block", "tide_gated_block_grad", "tide_orthogonalize"]


def registered(tide, name, workspace=None):
    function, args = arguments(name)
    more = {} if name == "tide_layer_norm" else {"workspace": workspace}
    return getattr(tide, function + "_call")(*args, **more)


@pytest.mark.parametrize("name", CALLS)
def test_a_launch_takes_its_workspace_on_its_own_stream(tide, monkeypatch, name):
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


@pytest.mark.parametrize("name", ["tide_layer_norm", *CALLS])
def test_launches_on_another_device_are_refused(tide, monkeypatch, name):
    import torch

    launched = []
    monkeypatch.setattr(tide.lib, name, lambda *a: launched.append(a) or 0)
    here = types.SimpleNamespace(cuda_stream=0x1000, device_index=0)
    there = types.SimpleNamespace(cuda_stream=0x2000, device_index=1)
    function, args = arguments(name)
    more = {} if name == "tide_layer_norm" else {"workspace": torch.empty(1 << 20, dtype=torch.uint8)}
    call = registered(tide, name, more.get("workspace"))
    once = lambda s: getattr(tide, function)(*args, **more, stream=s)
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
