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


@pytest.mark.parametrize("status", [fo.FO_ERR_TIMEOUT, fo.FO_ERR_ARG])
def test_clearing_an_error_gives_the_workspaces_up(device, monkeypatch, status):
    """A wait that ran out leaves a workspace's counters anywhere; the status
    keeps the first error only, so one of another kind may stand before it."""
    dev = torch.device("cuda", 0)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d=None: None)
    other = torch.device("cuda", 1)
    ws = torch.ones(100, dtype=torch.uint8)
    moe._status[dev] = torch.tensor([status], dtype=torch.int32)
    moe._workspaces[("few", dev, 7)] = moe._workspaces[("few", other, 7)] = ws
    assert moe.device_status(dev) == status and ("few", dev, 7) in moe._workspaces
    assert moe.device_status(dev, clear=True) == status
    assert ("few", dev, 7) not in moe._workspaces and ("few", other, 7) in moe._workspaces
    moe._workspaces[("few", dev, 7)] = ws
    assert moe.device_status(dev, clear=True) == fo.FO_OK
    assert moe._workspaces[("few", dev, 7)] is ws


def test_gathering_from_a_matrix_without_rows_is_no_bad_argument():
    """(Without a GPU the call gets as far as asking for the device.)"""
    args = dict(src=0, type=0, batch=1, batch_stride=0, rows=8, cols=64, row_stride=64,
                transpose=0, row_index=64, src_rows=0, codes=64, scales=64, stream=0)
    if torch.cuda.is_available():
        pytest.skip("these addresses are not to be launched on")
    with pytest.raises(fo.FoError) as e:
        fo.fo_mx_quantize(*args.values())
    assert e.value.status != fo.FO_ERR_ARG
    with pytest.raises(fo.FoError) as e:
        fo.fo_mx_quantize(*{**args, "src_rows": 1}.values())
    assert e.value.status == fo.FO_ERR_ARG


def test_calls_that_would_lose_a_gradient_are_refused():
    x, w = torch.zeros((4, 8)), torch.zeros((4, 2))
    ids = torch.zeros((4, 2), dtype=torch.int32)
    tracked = lambda t: t.clone().requires_grad_()
    for call in (lambda: moe.route(tracked(x), 2),
                 lambda: moe.route_backward(tracked(x), ids, w, w),
                 lambda: moe.route_backward(x, ids, tracked(w), w),
                 lambda: moe.route_backward(x, ids, w, tracked(w))):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
            call()


def test_the_status_word_is_set_before_any_other_stream_can_use_it(device, monkeypatch):
    """It is zeroed on one stream and used on all: once when it is made, and when
    an error is cleared, its zero is waited for."""
    dev, _ = device
    waits = []
    stream = lambda d: type("Stream", (), {"synchronize": lambda self: waits.append(d)})()
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d=None: waits.append(d))
    moe._status_word(dev)
    assert waits == [dev]
    moe._status_word(dev)
    assert waits == [dev]
    gpu = torch.device("cuda", 0)
    moe._status[gpu] = torch.tensor([fo.FO_ERR_ARG], dtype=torch.int32)
    assert moe.device_status(gpu, clear=True) == fo.FO_ERR_ARG
    assert waits == [dev, gpu, gpu]
