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


class OnDevice:
    """A tensor's attributes, on a GPU that this machine need not have."""

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.is_cuda, self.device = device >= 0, "cuda:%d" % device

    def get_device(self):
        return self.index

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1


H, F, I = torch.bfloat16, torch.float32, torch.int64
CALLS = {
    "muon_grouped_mm": (dict(x=((4, 16), H), w=((2, 16, 8), H), offsets=((3,), I), y=((4, 8), H)), ()),
    "muon_grouped_wgrad": (dict(a=((4, 16), H), b=((4, 8), H), offsets=((3,), I), dw=((2, 16, 8), F)), ()),
    "muon_swiglu": (dict(gate=((4, 8), H), up=((4, 8), H), out=((4, 8), H), row_weight=((4,), F)), ()),
    "muon_swiglu_grad": (dict(dout=((4, 8), H), gate=((4, 8), H), up=((4, 8), H), dgate=((4, 8), H),
                              dup=((4, 8), H), row_weight=((4,), F), d_row_weight=((4,), F)), ()),
    "muon_grad_norm": (dict(grads=((4, 8), H), norm=((2,), F)), ("grads",)),
    "muon_clip_grads": (dict(grads=((4, 8), H), outs=((4, 8), H), norm=((2,), F)), ("grads", "outs")),
}
WITH_WORKSPACE = [c for c in CALLS if "swiglu" not in c]


@pytest.fixture()
def no_launch(monkeypatch):
    """Calls that get through the binding's checks end at the library, which launches nothing."""
    class Reached(Exception):
        pass

    def reached(*args):
        raise Reached

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    monkeypatch.setattr(capi, "lib", SimpleNamespace(**{name: reached for name in CALLS}))
    return Reached


def _call(name, elsewhere=None, device=1, workspace=None):
    spec, lists = CALLS[name]
    args = {}
    for k, (shape, dtype) in spec.items():
        t = OnDevice(shape, dtype, device if elsewhere in (k, "all") else 0)
        args[k] = [t] if k in lists else t
    if "norm" in spec:
        args["max_norm"] = 1.0
        workspace = workspace or OnDevice((64,), torch.uint8)
    return getattr(capi, name)(**args, **({"workspace": workspace} if workspace is not None else {}))


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_device_goes_through(no_launch, name):
    with pytest.raises(no_launch):
        _call(name)


@pytest.mark.parametrize("device", [1, -1])
@pytest.mark.parametrize("name,arg", [(n, a) for n, (spec, _) in CALLS.items() for a in [*spec, "all"]])
def test_tensors_of_other_devices_are_refused(no_launch, name, arg, device):
    """The library launches on the current device: a pointer of another is not to get there."""
    with pytest.raises(ValueError, match="cuda|CUDA"):
        _call(name, arg, device)


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspaces_that_the_gpu_cannot_use_are_refused(no_launch, name):
    with pytest.raises(no_launch):
        _call(name, workspace=OnDevice((64,), torch.uint8))
    for device in (1, -1):
        with pytest.raises(ValueError, match="workspace"):
            _call(name, workspace=OnDevice((64,), torch.uint8, device))
    expanded = OnDevice((64,), torch.uint8)
    expanded.is_contiguous = lambda: False
    with pytest.raises(ValueError, match="workspace"):
        _call(name, workspace=expanded)


def test_a_scale_of_another_device_is_refused(no_launch):
    for device in (1, -1):
        with pytest.raises(ValueError, match="grad_scale"):
            capi.muon_step_scaled([], [], [], None, 0, [], OnDevice((1,), F, device))
