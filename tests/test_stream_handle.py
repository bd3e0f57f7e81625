"""Where the binding takes the current stream's handle from."""
import types

import pytest
import torch

from bit_expert_ffn_fp32_b200 import native


@pytest.fixture
def fresh():
    """The binding's view of torch, to be looked up anew before and after the test."""
    def forget():
        native._Types.code, native._Types.device, native._Types.raw_stream = {}, None, None
    forget()
    yield
    forget()


def test_without_torchs_raw_handle(fresh, monkeypatch):
    """torch's function for the bare handle is not part of its public interface."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(cuda_stream=70 + dev))
    assert native.stream_handle() == 73


@pytest.mark.gpu
def test_handles_are_the_same(fresh, monkeypatch):
    side = torch.cuda.Stream()
    with_raw = native.stream_handle()
    with torch.cuda.stream(side):
        side_raw = native.stream_handle()
    native._Types.device = None
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    with torch.cuda.stream(side):
        assert native.stream_handle() == side_raw == native.stream_handle(side) == side.cuda_stream
    assert native.stream_handle() == with_raw
