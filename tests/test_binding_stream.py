"""Which stream the binding takes: the current one where none is given, with or without torch's
unpublished names for it; a handle; a Stream."""
import types

import pytest
import torch

import rotated_bit_linear_amd as rbl


@pytest.mark.parametrize("missing", ["_raw_stream", "_raw_device"])
def test_torch_without_the_unpublished_names(monkeypatch, missing):
    monkeypatch.setattr(rbl, missing, None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0x1230))
    assert rbl._stream(None) == 0x1230


def test_current_stream_of_the_current_device(monkeypatch):
    monkeypatch.setattr(rbl, "_raw_device", lambda: 3)
    monkeypatch.setattr(rbl, "_raw_stream", lambda device: 0x100 + device)
    assert rbl._stream(None) == 0x103


def test_given_streams():
    assert rbl._stream(0) == 0 and rbl._stream(77) == 77
    assert rbl._stream(types.SimpleNamespace(cuda_stream=0x55)) == 0x55


@pytest.mark.gpu
def test_same_handle_as_the_public_way():
    assert rbl._stream(None) == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert rbl._stream(None) == side.cuda_stream
