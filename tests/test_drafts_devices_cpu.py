"""Which device a call on drafted tokens is launched on, without a GPU: torch's stream functions are stood in for."""
import contextlib

import pytest
import torch

from hybrid_gated_deltanet_q4k_gb300 import lib as gl


class Cuda:
    """The current device, the devices' streams, and a C entry point that notes where it was called."""

    def __init__(self, monkeypatch, current, cached):
        self.current, self.calls = current, []
        raw, here = (lambda device: 100 + device), (lambda: self.current)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", raw, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", here, raising=False)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(gl, "_raw_stream", raw if cached else None)
        monkeypatch.setattr(gl, "_current_device", here if cached else None)

    @contextlib.contextmanager
    def device(self, device):
        before, self.current = self.current, device
        yield
        self.current = before

    def entry(self, *args):
        self.calls.append((self.current, *args))
        return 0


class Stream:
    def __init__(self, device, handle):
        self.device_index, self.cuda_stream = device, handle


def call(cuda, device, stream, *args):
    """As the wrappers call the library."""
    return gl.entry(cuda.entry, device, stream)(*args, gl.stream_on(device, stream))


@pytest.mark.parametrize("cached", [False, True])
def test_memory_of_another_device_is_refused(monkeypatch, cached):
    """In a process's first call as in any later one."""
    c = Cuda(monkeypatch, 0, cached)
    for stream in (None, Stream(0, 7), Stream(0, 0)):
        with pytest.raises(ValueError, match="cuda:1"):
            call(c, 1, stream, 5)
    assert not c.calls
    assert call(c, 0, None, 5) == 0 and c.calls == [(0, 5, 100)]


@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("handle", [0, 7])
def test_a_stream_of_another_device_is_called_on_that_device(monkeypatch, cached, handle):
    """The handle of a default stream (0) would stand for the current device's."""
    c = Cuda(monkeypatch, 0, cached)
    call(c, 1, Stream(1, handle), 5, 6)
    call(c, 0, Stream(0, handle), 5, 6)
    assert c.calls == [(1, 5, 6, handle), (0, 5, 6, handle)] and c.current == 0


@pytest.mark.parametrize("cached", [False, True])
def test_the_stream_s_device_is_compared(monkeypatch, cached):
    Cuda(monkeypatch, 0, cached)
    with pytest.raises(ValueError, match="cuda:1"):
        gl.stream_on(1)
    assert gl.stream_on(0) == 100
