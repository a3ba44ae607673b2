"""The stream a call takes when it is given none: the handle alone where torch offers it,
the stream object otherwise (no GPU needed)."""
import types

import pytest
import torch

import rank_compressed_kv_star_b200 as S


@pytest.fixture
def current(monkeypatch):
    """A current stream with handle 4321, known to torch's public functions."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=4321))


def test_given_streams_are_taken_as_they_are():
    assert S._stream(77) == 77 and S._stream(0) == 0
    assert S._stream(types.SimpleNamespace(cuda_stream=99)) == 99


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_a_torch_without_the_raw_handle(monkeypatch, current, missing):
    monkeypatch.delattr(torch._C, missing, raising=False)
    assert S._stream(None) == 4321


def test_the_raw_handle_is_preferred(monkeypatch, current):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    assert S._stream(None) == 1003


def test_before_cuda_is_initialised(monkeypatch, current):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    assert S._stream(None) == 4321
