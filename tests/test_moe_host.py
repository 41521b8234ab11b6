"""What the expert layer's Python calls keep between calls, on the CPU: the
caches are filled with CPU tensors and the device's answers are given."""
import pytest
import torch

from communication_overlap_gb300 import fo, moe


@pytest.fixture
def device(monkeypatch):
    """A device whose stream is 7, and whether it is being captured."""
    dev, capturing = torch.device("cpu"), [False]
    monkeypatch.setattr(moe, "_workspaces", {})
    monkeypatch.setattr(moe, "_status", {})
    monkeypatch.setattr(moe, "_stream", lambda d: 7)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: dev.index)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    return dev, capturing


def test_a_captured_call_has_a_workspace_of_its_own(device):
    """Whether or not the stream has one already: a graph keeps the address,
    and a later, larger call would give the stream's back."""
    dev, capturing = device
    eager = moe._workspace("few", dev, 100)
    capturing[0] = True
    captured = moe._workspace("few", dev, 100)
    assert captured.data_ptr() != eager.data_ptr() and not captured.any()
    assert moe._workspace("few", dev, 100).data_ptr() != captured.data_ptr()
    capturing[0] = False
    assert moe._workspace("few", dev, 100) is eager
    larger = moe._workspace("few", dev, 200)
    assert larger.numel() >= 200 and moe._workspace("few", dev, 100) is larger
