"""The `stream` of a layer call: it belongs to the tensors' device, whichever device is current."""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import layer


class Elsewhere(torch.Tensor):
    """A host tensor that says it lies on the second GPU."""
    device = torch.device("cuda:1")


def elsewhere(*shape):
    return torch.zeros(*shape).as_subclass(Elsewhere)


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle
        self.device = torch.device("cuda:0" if device is None else device)


@pytest.fixture
def used(monkeypatch):
    """The streams that calls make current, and stand-ins for the calls into the library."""
    streams = []

    class Context:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            streams.append(self.stream)

        def __exit__(self, *_):
            pass

    class Native:
        def norm_forward(self, x, *_):
            return x, None, None, None

        def norm_backward(self, *_):
            return None, None

    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(layer, "_native", Native)
    return streams


def test_a_handle_becomes_a_stream_of_the_tensors_device(used):
    layer.norm_forward(elsewhere(2, 64), elsewhere(64), stream=1234)
    layer.norm_backward(dy=elsewhere(2, 64), r=elsewhere(2, 64), weight=elsewhere(64), stream=1234)
    assert [(s.cuda_stream, s.device) for s in used] == [(1234, torch.device("cuda:1"))] * 2


def test_a_stream_of_the_tensors_device_is_taken(used):
    mine = FakeStream(7, "cuda:1")
    layer.norm_forward(elsewhere(2, 64), elsewhere(64), stream=mine)
    assert used == [mine]


def test_a_stream_of_another_device_is_refused(used):
    with pytest.raises(ValueError, match="stream"):
        layer.norm_forward(elsewhere(2, 64), elsewhere(64), stream=FakeStream(7, "cuda:0"))
    assert not used


def test_no_stream_is_the_current_one(used):
    layer.norm_forward(elsewhere(2, 64), elsewhere(64))
    assert not used


def test_host_tensors_are_refused_with_a_stream_too():
    with pytest.raises(ValueError, match="device tensor"):
        layer.norm_forward(torch.zeros(2, 64), torch.zeros(64), stream=1234)


@pytest.mark.gpu
def test_a_handle_is_the_stream_the_kernels_run_on():
    side = torch.cuda.Stream()
    x, w = torch.randn(64, 256, device="cuda"), torch.ones(256, device="cuda")
    want = layer.norm_forward(x, w)[0]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)                # tens of milliseconds ahead of the call on that stream alone
    done = torch.cuda.Event()
    y = layer.norm_forward(x, w, stream=side.cuda_stream)[0]
    done.record(side)
    assert not done.query()
    done.synchronize()
    assert torch.equal(y, want)
