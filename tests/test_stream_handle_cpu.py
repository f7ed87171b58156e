"""The binding's handle of the current stream, with and without torch's
short way to it."""
import types

import pytest
import torch

import optimizer_step_amd as osa


def test_current_stream_without_the_raw_handle(monkeypatch):
    """A torch without the private accessor gives the handle by its public one."""
    asked = []
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: asked.append(dev) or types.SimpleNamespace(cuda_stream=77))
    assert osa._stream(None) == 77 and osa._raw_stream(None, 2) == 77
    assert asked == [3, 2]


def test_current_stream_by_the_raw_handle(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert osa._stream(None) == 103 and osa._raw_stream(None, 2) == 102


def test_given_streams():
    assert osa._stream(5) == 5 and osa._raw_stream(5, 0) == 5
    assert osa._stream(types.SimpleNamespace(cuda_stream=9)) == 9


def test_streams_of_another_device_are_refused():
    """A launch runs on its stream's device, where the tensors' addresses may mean nothing."""
    assert osa._raw_stream(types.SimpleNamespace(cuda_stream=9, device_index=1), 1) == 9
    with pytest.raises(ValueError, match="device 1"):
        osa._raw_stream(types.SimpleNamespace(cuda_stream=9, device_index=1), 0)
