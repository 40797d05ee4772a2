"""CPU: which device and stream a call names, for tensors that are not on the current device.

No device is touched: the library's entry points and torch's queries of the current device and
stream are stand-ins that record what they are asked.
"""
import contextlib
import types

import pytest
import torch

from sequence_exact_attention_ring_b200 import api


@pytest.fixture
def devices(monkeypatch):
    """Device 0 is current; a device's current stream is 1000 + its index."""
    now = [0]

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d.index
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(
        cuda_stream=1000 + (now[0] if d is None else d.index)))
    monkeypatch.setattr(api, "_current_raw_stream", lambda index: 1000 + index)
    return now


@pytest.mark.parametrize("index", [0, 1])
def test_status_waits_for_its_workspaces_device(devices, monkeypatch, index):
    asked = []
    monkeypatch.setattr(api._b, "ring_attn_status", lambda ws, stream: asked.append((ws, stream, devices[0])) or 0)
    ws = types.SimpleNamespace(device=torch.device("cuda", index), data_ptr=lambda: 77)
    assert api.status(ws) == 0
    assert api.status(ws, stream=types.SimpleNamespace(cuda_stream=5)) == 0
    assert asked == [(77, 1000 + index, index), (77, 5, index)]
    assert devices == [0]
