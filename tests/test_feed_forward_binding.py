"""The feed-forward binding on the host: tensors of another device, type or shape are refused before the
library is called."""
from types import SimpleNamespace

import pytest

capi = pytest.importorskip("muon_optimizer_step_gb300.capi",
                           reason="libmuon.so not built (run __graft_entry__.build())")
torch = pytest.importorskip("torch")

H, G, F, I, Q = torch.bfloat16, torch.float16, torch.float32, torch.int64, torch.float8_e4m3fn


class OnDevice:
    """A tensor's attributes, on a GPU that this machine need not have."""

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.device = "cuda:%d" % device

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


CALLS = {
    "muon_layer_norm": dict(x=((4, 16), H), weight=((16,), F), bias=((16,), F), y=((4, 16), H), mean=((4,), F),
                            rstd=((4,), F)),
    "muon_layer_norm_grad": dict(dy=((4, 16), H), x=((4, 16), H), weight=((16,), F), mean=((4,), F), rstd=((4,), F),
                                 dx=((4, 16), H), dweight=((16,), F), dbias=((16,), F)),
    "muon_gated_mm": dict(x=((4, 16), H), w_gate=((2, 16, 8), H), w_up=((2, 16, 8), H), offsets=((3,), I),
                          out=((4, 8), H), gate=((4, 8), H), up=((4, 8), H), row_weight=((4,), F)),
    "muon_gated_mm_grad": dict(dy=((4, 16), H), w=((2, 16, 8), H), offsets=((3,), I), gate=((4, 8), H),
                               up=((4, 8), H), dgate=((4, 8), H), dup=((4, 8), H), out=((4, 8), H),
                               row_weight=((4,), F), d_row_weight=((4,), F)),
    "muon_grouped_mm_sum": dict(x1=((4, 16), H), w1=((2, 16, 8), H), x2=((4, 16), H), w2=((2, 16, 8), H),
                                offsets=((3,), I), y=((4, 8), H)),
    "muon_quantize_rows": dict(x=((4, 200), H), q=((4, 200), Q), scale=((2, 4), F)),
    "muon_quantize_weights": dict(w=((3, 200, 16), H), q=((3, 200, 16), Q), scale=((3, 2, 1), F)),
    "muon_grouped_mm_fp8": dict(x=((4, 208), Q), x_scale=((2, 4), F), w=((2, 16, 208), Q), w_scale=((2, 1, 2), F),
                                offsets=((3,), I), y=((4, 16), H)),
}
OPTIONAL = {"muon_layer_norm": ("weight", "bias", "mean", "rstd"),
            "muon_layer_norm_grad": ("weight", "dweight", "dbias"),
            "muon_gated_mm": ("gate", "up", "row_weight"), "muon_gated_mm_grad": ("out", "row_weight", "d_row_weight")}
WITH_WORKSPACE = ["muon_layer_norm_grad", "muon_gated_mm", "muon_gated_mm_grad", "muon_grouped_mm_sum"]


@pytest.fixture()
def no_launch(monkeypatch):
    """Calls that get through the binding's checks end at the library, which launches nothing."""
    class Reached(Exception):
        pass

    def reached(*args):
        raise Reached

    def query(*args):
        return capi.MUON_OK

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    names = {name: reached for name in CALLS}
    names.update({name + "_workspace_bytes": query for name in WITH_WORKSPACE})
    monkeypatch.setattr(capi, "lib", SimpleNamespace(**names))
    return Reached


def _call(name, workspace=None, **changes):
    args = {k: OnDevice(shape, dtype) for k, (shape, dtype) in CALLS[name].items()}
    args.update(changes)
    if name in WITH_WORKSPACE:
        args["workspace"] = workspace or OnDevice((64,), torch.uint8)
    return getattr(capi, name)(**args)


@pytest.mark.parametrize("name", CALLS)
def test_calls_go_through(no_launch, name):
    with pytest.raises(no_launch):
        _call(name)
    for arg in OPTIONAL.get(name, ()):
        with pytest.raises(no_launch):
            _call(name, **{arg: None})
    if "offsets" in CALLS[name]:
        with pytest.raises(ValueError, match="offsets"):
            _call(name, offsets=None)


@pytest.mark.parametrize("device", [1, -1])
@pytest.mark.parametrize("name,arg", [(n, a) for n, spec in CALLS.items() for a in spec])
def test_tensors_of_other_devices_are_refused(no_launch, name, arg, device):
    shape, dtype = CALLS[name][arg]
    with pytest.raises(ValueError, match="cuda|CUDA"):
        _call(name, **{arg: OnDevice(shape, dtype, device)})


@pytest.mark.parametrize("name,arg", [(n, a) for n, spec in CALLS.items() for a in spec])
def test_other_types_and_shapes_are_refused(no_launch, name, arg):
    shape, dtype = CALLS[name][arg]
    wrong = {H: G, F: H, I: torch.int32, Q: torch.uint8}[dtype]
    alone = {"muon_quantize_rows": ("x",), "muon_quantize_weights": ("w",), "muon_grouped_mm_fp8": ("y",)}
    if arg not in alone.get(name, ()):     # (those take any type)
        with pytest.raises(ValueError):
            _call(name, **{arg: OnDevice(shape, wrong)})
    with pytest.raises(ValueError):
        _call(name, **{arg: OnDevice(shape, torch.float64)})
    for other in ((*shape[:-1], shape[-1] + 1), (*shape, 1), (shape[0] + 1, *shape[1:])):
        with pytest.raises(ValueError):
            _call(name, **{arg: OnDevice(other, dtype)})


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspaces_that_the_gpu_cannot_use_are_refused(no_launch, name):
    for device in (1, -1):
        with pytest.raises(ValueError, match="workspace"):
            _call(name, workspace=OnDevice((64,), torch.uint8, device))
    expanded = OnDevice((64,), torch.uint8)
    expanded.is_contiguous = lambda: False
    with pytest.raises(ValueError, match="workspace"):
        _call(name, workspace=expanded)


def test_mixed_matrices_are_refused(no_launch):
    """The gradient needs the forward pass's statistics; host tensors never pass."""
    with pytest.raises(ValueError, match="mean"):
        _call("muon_layer_norm_grad", mean=None)
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        capi.muon_layer_norm(x, None, None, x)
