"""The expert-layer binding on the host: what it takes from torch, and in which order."""
import contextlib
from types import SimpleNamespace

import pytest

capi = pytest.importorskip("muon_optimizer_step_gb300.capi",
                           reason="libmuon.so not built (run __graft_entry__.build())")
torch = pytest.importorskip("torch")


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


@pytest.fixture()
def torch_with_streams(monkeypatch):
    """A stand-in for torch whose allocations note the stream that is current then."""
    current = [Stream(0x500)]
    taken = []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def empty(n, dtype, device):
        taken.append(current[-1].cuda_stream)
        return SimpleNamespace(data_ptr=lambda: 0x10008, record_stream=lambda s: None)

    cuda = SimpleNamespace(Stream=Stream, stream=stream, default_stream=lambda device: Stream(0),
                           ExternalStream=lambda handle, device: Stream(handle))
    monkeypatch.setattr(capi, "_torch", SimpleNamespace(cuda=cuda, empty=empty, uint8=None))
    return taken


@pytest.mark.parametrize("stream,handle", [
    (None, 0x500), (Stream(0x700), 0x700), (0x900, 0x900),
    (0, 0), (1, 0),       # the default stream, by either of its handles
])
def test_workspace_comes_from_the_stream_that_uses_it(torch_with_streams, stream, handle):
    """A block freed on the current stream may still be in use there: only work behind it on the same
    stream may have it."""
    ptr, nbytes, owner = capi._workspace(None, 100, 1024, SimpleNamespace(device="cuda:0"), stream)
    assert torch_with_streams == [handle]
    assert ptr % 1024 == 0 and 0 <= ptr - 0x10008 < 1024 and nbytes == 100 and owner is not None
