"""ctypes binding of libmuon.so: the C entry points under the same names.

Only argument marshalling happens here (torch tensors -> device pointers, Python
lists -> host pointer arrays, a torch stream -> cudaStream_t); every step of the
optimizer runs in the library's CUDA kernels.  Importing this module loads the library
and raises if it has not been built: there is no other code path.
"""
from __future__ import annotations

import array
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# MUON_LIB may name another build of the library (e.g. libmuon_debug.so, whose kernels
# range-check every table entry they use); the default is the in-tree libmuon.so.
LIB_PATH = os.environ.get("MUON_LIB") or os.path.join(_HERE, "libmuon.so")

MUON_OK = 0
MUON_ERR_INVALID_ARG = 1
MUON_ERR_ALIGNMENT = 2
MUON_ERR_CUDA = 3
MUON_ERR_TIMEOUT = 4
MUON_ERR_OOM = 5
MUON_ERR_UNSUPPORTED = 6
MUON_ERR_DEVICE_CHECK = 7
MUON_ERR_ROW_OFFSETS = 8
MUON_NS_BF16 = 0
MUON_NS_FP32 = 1
MUON_NS_SPLIT_FP32 = 2
MUON_DTYPE_F32 = 0
MUON_DTYPE_BF16 = 1
MUON_DTYPE_F16 = 2
MUON_MAX_SHARDS = 128
MUON_MAX_EXPERTS = 1024
WORKSPACE_ALIGN = 1024

_STATUS_NAMES = {0: "MUON_OK", 1: "MUON_ERR_INVALID_ARG", 2: "MUON_ERR_ALIGNMENT",
                 3: "MUON_ERR_CUDA", 4: "MUON_ERR_TIMEOUT", 5: "MUON_ERR_OOM",
                 6: "MUON_ERR_UNSUPPORTED", 7: "MUON_ERR_DEVICE_CHECK",
                 8: "MUON_ERR_ROW_OFFSETS"}

# (name, restype, argtypes) of every entry point declared in include/muon.h.
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F = ctypes.c_float
_PP = ctypes.POINTER(ctypes.c_void_p)


class GroupHparams(ctypes.Structure):
    """muon_group_hparams: one optimizer group's hyper-parameters."""
    _fields_ = [("lr", ctypes.c_float), ("wd", ctypes.c_float), ("mu", ctypes.c_float),
                ("nesterov", ctypes.c_int32)]

_SZ = ctypes.c_size_t

SIGNATURES = [
    ("muon_abi_version", _I32, []),
    ("muon_last_error", ctypes.c_char_p, []),
    ("muon_layout_create", _I32, [ctypes.POINTER(_I64), ctypes.POINTER(ctypes.c_uint8), _I32,
                                  _I32, _I32, ctypes.POINTER(_P)]),
    ("muon_layout_destroy", _I32, [_P]),
    ("muon_layout_numel", _I32, [_P, ctypes.POINTER(_I64)]),
    ("muon_layout_shard_len", _I32, [_P, ctypes.POINTER(_I64)]),
    ("muon_layout_workspace_bytes", _I32, [_P, ctypes.POINTER(ctypes.c_size_t)]),
    ("muon_layout_full_numel", _I32, [_P, ctypes.POINTER(_I64)]),
    ("muon_full_offsets", _I32, [_P, ctypes.POINTER(_I64)]),
    ("muon_step", _I32, [_PP, _PP, _PP, _P, _P, _F, _F, _F, _I32, _I32, _P]),
    ("muon_compute_momentum_inputs", _I32, [_PP, _PP, _P, _P, _F, _I32, _P]),
    ("muon_orthogonalize_updates", _I32, [_P, _P, _I32, _P]),
    ("muon_apply_local_updates", _I32, [_PP, _P, _P, _F, _F, _I32, _P]),
    ("muon_orthogonalize_apply", _I32, [_PP, _P, _P, _F, _F, _I32, _P]),
    ("muon_layout_set_groups", _I32, [_P, ctypes.POINTER(_I32), _I32]),
    ("muon_step_grouped", _I32, [_PP, _PP, _PP, _P, _P, ctypes.POINTER(GroupHparams), _I32, _P]),
    ("muon_assign_owners", _I32, [_P, _I32, ctypes.POINTER(_I32), ctypes.POINTER(ctypes.c_double)]),
    ("muon_exchange_plan", _I32, [_P, ctypes.POINTER(_I32), _I32, _P, ctypes.POINTER(_I64), _P,
                                  ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                                  ctypes.POINTER(_I64)]),
    ("muon_gather_full", _I32, [_P, _PP, _P, _P]),
    ("muon_scatter_updates", _I32, [_P, _P, _PP, _P]),
    ("muon_orthogonalize_full", _I32, [_P, _P, _P, _P, _I32, _P]),
    ("muon_export_input", _I32, [_P, _P, _P, _P]),
    ("muon_export_update", _I32, [_P, _P, _I32, _P, _P]),
    ("muon_orthogonalize_full_noalloc", _I32, [_P, _P, _P, _I32, _P]),
    ("muon_check", _I32, [_P]),
    ("muon_selftest_wait_timeout", _I32, [_I64, _P]),
    ("muon_debug_build", _I32, []),
    ("muon_selftest_device_check", _I32, [_P]),
    ("muon_layout_ns_kernel", _I32, [_P, ctypes.POINTER(_I32), ctypes.POINTER(_I32),
                                     ctypes.POINTER(_I32)]),
    ("muon_layout_fused_apply", _I32, [_P, ctypes.POINTER(_I32)]),
    ("muon_step_scaled", _I32, [_PP, _PP, _PP, _P, _P, ctypes.POINTER(GroupHparams), _I32, _P,
                                _P]),
    ("muon_grouped_mm", _I32, [_P, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _I32, _I32, _I32,
                               _I32, _I32, _I32, _P, _SZ, _P]),
    ("muon_grouped_mm_workspace_bytes", _I32, [_P, _I64, _P, _I64, _I64, _I64, _I32, _I32, _I32,
                                               _I32, ctypes.POINTER(_SZ)]),
    ("muon_grouped_wgrad", _I32, [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _I32, _I32, _I32,
                                  _I32, _I32, _P, _SZ, _P]),
    ("muon_grouped_wgrad_workspace_bytes", _I32, [_P, _I64, _P, _I64, _I64, _I32, _I32,
                                                  ctypes.POINTER(_SZ)]),
    ("muon_swiglu", _I32, [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _I32, _I32, _P]),
    ("muon_swiglu_grad", _I32, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64,
                                _I32, _I32, _P]),
    ("muon_grad_norm", _I32, [_P, _I32, _F, _P, _P, _SZ, _P]),
    ("muon_clip_grads", _I32, [_P, _P, _I32, _F, _P, _P, _SZ, _P]),
    ("muon_clip_workspace_bytes", _I32, [_P, _I32, ctypes.POINTER(_SZ)]),
    ("muon_layer_norm", _I32, [_P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _I32, _F, _I32, _P]),
    ("muon_layer_norm_grad", _I32, [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _I64, _I32,
                                    _I32, _I32, _P, _SZ, _P]),
    ("muon_layer_norm_grad_workspace_bytes", _I32, [_I64, _I32, ctypes.POINTER(_SZ)]),
    ("muon_gated_mm", _I32, [_P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _P, _I64,
                             _P, _I64, _I64, _I32, _I32, _I32, _I32, _I32, _P, _SZ, _P]),
    ("muon_gated_mm_workspace_bytes", _I32, [_P, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _I32,
                                             _I32, _I32, _I32, ctypes.POINTER(_SZ)]),
    ("muon_gated_mm_grad", _I32, [_P, _I64, _P, _I64, _I64, _P, _P, _I64, _P, _I64, _P, _P, _I64, _P,
                                  _I64, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _SZ,
                                  _P]),
    ("muon_gated_mm_grad_workspace_bytes", _I32, [_P, _I64, _P, _I64, _I64, _I64, _I32, _I32, _I32,
                                                  _I32, _I32, ctypes.POINTER(_SZ)]),
    ("muon_grouped_mm_sum", _I32, [_P, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _I64, _P, _P, _I64,
                                   _I64, _I32, _I32, _I32, _I32, _I32, _I32, _P, _SZ, _P]),
    ("muon_grouped_mm_sum_workspace_bytes", _I32, [_P, _I64, _P, _I64, _I64, _P, _I64, _P, _I64,
                                                   _I64, _I64, _I32, _I32, _I32, _I32,
                                                   ctypes.POINTER(_SZ)]),
    ("muon_quantize_rows", _I32, [_P, _I64, _P, _I64, _P, _I64, _I64, _I32, _I32, _P]),
    ("muon_quantize_weights", _I32, [_P, _I64, _I64, _P, _I64, _I64, _P, _I32, _I32, _I32, _I32, _I32,
                                     _P]),
    ("muon_grouped_mm_fp8", _I32, [_P, _I64, _P, _I64, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _I32,
                                   _I32, _I32, _I32, _P]),
]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; "
            "g.build()'); this package has no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class MuonError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib.muon_last_error().decode(errors="replace")
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status: int, where: str):
    if status != MUON_OK:
        raise MuonError(status, where)


# ------------------------------------------------------------------ marshalling helpers
def _stream_handle(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _shard_array(layout, shards, name):
    """A host array of n_shards device pointers from a tensor or a list of tensors."""
    if not isinstance(shards, (list, tuple)):
        shards = [shards]
    if len(shards) != layout.n_shards:
        raise ValueError(f"{name}: expected {layout.n_shards} shard(s), got {len(shards)}")
    for s in shards:
        if isinstance(s, int):
            continue
        import torch
        if s.dtype != torch.float32 or not s.is_contiguous() or s.device.type != "cuda":
            raise ValueError(f"{name}: shards must be contiguous float32 CUDA tensors")
        if s.numel() < layout.shard_len:
            raise ValueError(f"{name}: shard has {s.numel()} elements, layout needs {layout.shard_len}")
    arr = (ctypes.c_void_p * max(1, len(shards)))()
    for i, s in enumerate(shards):
        arr[i] = s if isinstance(s, int) else s.data_ptr()
    return arr


class Layout:
    """Owns a muon_layout handle (see muon_layout_create)."""

    def __init__(self, handle, shapes, is_matrix, n_shards, ns_dtype):
        self.handle = handle
        self.shapes = shapes
        self.is_matrix = is_matrix
        self.n_shards = n_shards
        self.ns_dtype = ns_dtype
        v = _I64()
        _check(lib.muon_layout_numel(handle, ctypes.byref(v)), "muon_layout_numel")
        self.numel = v.value
        _check(lib.muon_layout_shard_len(handle, ctypes.byref(v)), "muon_layout_shard_len")
        self.shard_len = v.value
        _check(lib.muon_layout_full_numel(handle, ctypes.byref(v)), "muon_layout_full_numel")
        self.full_numel = v.value
        b = ctypes.c_size_t()
        _check(lib.muon_layout_workspace_bytes(handle, ctypes.byref(b)),
               "muon_layout_workspace_bytes")
        self.workspace_bytes = b.value
        offs = (_I64 * max(1, len(shapes)))()
        _check(lib.muon_full_offsets(handle, offs), "muon_full_offsets")
        self.full_offsets = [offs[i] for i in range(len(shapes))]

    def close(self):
        if self.handle:
            lib.muon_layout_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def _as_parameter_(self):
        return self.handle


def muon_layout_create(shapes, n_shards=1, ns_dtype=MUON_NS_BF16, is_matrix=None) -> Layout:
    shapes = [(int(r), int(c)) for r, c in shapes]
    n = len(shapes)
    flat = (_I64 * max(1, 2 * n))(*[v for rc in shapes for v in rc])
    flags = None
    if is_matrix is not None:
        is_matrix = [1 if f else 0 for f in is_matrix]
        if len(is_matrix) != n:
            raise ValueError("is_matrix must have one flag per shape")
        flags = (ctypes.c_uint8 * max(1, n))(*is_matrix)
    if isinstance(ns_dtype, str):
        ns_dtype = {"bf16": MUON_NS_BF16, "fp32": MUON_NS_FP32, "split": MUON_NS_SPLIT_FP32}[ns_dtype]
    h = ctypes.c_void_p()
    _check(lib.muon_layout_create(flat, flags, n, int(n_shards), int(ns_dtype), ctypes.byref(h)),
           "muon_layout_create")
    return Layout(h, shapes, is_matrix, int(n_shards), int(ns_dtype))


def workspace_tensor(layout: Layout, device="cuda"):
    """A uint8 CUDA tensor of layout.workspace_bytes whose data_ptr is 1024-byte aligned."""
    import torch
    raw = torch.empty(layout.workspace_bytes + WORKSPACE_ALIGN, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % WORKSPACE_ALIGN
    ws = raw[off: off + layout.workspace_bytes]
    ws._muon_base = raw  # keep the allocation alive with the view
    return ws


def muon_step(flat_params, flat_grads, flat_momentum, layout, workspace, lr, wd, mu,
              nesterov=True, ns_steps=5, stream=None):
    _check(lib.muon_step(_shard_array(layout, flat_params, "flat_params"),
                         _shard_array(layout, flat_grads, "flat_grads"),
                         _shard_array(layout, flat_momentum, "flat_momentum"),
                         layout.handle, _ptr(workspace), float(lr), float(wd), float(mu),
                         1 if nesterov else 0, int(ns_steps), _stream_handle(stream)),
           "muon_step")


def muon_layout_set_groups(layout, group_of, n_groups):
    arr = (_I32 * max(1, len(group_of)))(*[int(g) for g in group_of])
    _check(lib.muon_layout_set_groups(layout.handle, arr, int(n_groups)), "muon_layout_set_groups")
    layout.n_groups = int(n_groups)


def muon_step_grouped(flat_params, flat_grads, flat_momentum, layout, workspace, groups,
                      ns_steps=5, stream=None):
    """groups: a sequence of (lr, wd, mu, nesterov), one per optimizer group."""
    arr = (GroupHparams * max(1, len(groups)))(
        *[GroupHparams(float(lr), float(wd), float(mu), 1 if nest else 0)
          for lr, wd, mu, nest in groups])
    _check(lib.muon_step_grouped(_shard_array(layout, flat_params, "flat_params"),
                                 _shard_array(layout, flat_grads, "flat_grads"),
                                 _shard_array(layout, flat_momentum, "flat_momentum"),
                                 layout.handle, _ptr(workspace), arr, int(ns_steps),
                                 _stream_handle(stream)), "muon_step_grouped")


def muon_step_scaled(flat_params, flat_grads, flat_momentum, layout, workspace, groups,
                     grad_scale, ns_steps=5, stream=None):
    """muon_step_grouped with the gradients multiplied by grad_scale, a CUDA tensor of one
    float32 (norm[1:] of muon_grad_norm: the step then clips by the global norm)."""
    if not isinstance(grad_scale, int):
        _device_of(grad_scale, "grad_scale")
        if grad_scale.numel() < 1 or _kind(grad_scale, "grad_scale") != MUON_DTYPE_F32:
            raise ValueError("grad_scale: must be a float32 value")
    arr = (GroupHparams * max(1, len(groups)))(
        *[GroupHparams(float(lr), float(wd), float(mu), 1 if nest else 0)
          for lr, wd, mu, nest in groups])
    if len(groups) < getattr(layout, "n_groups", 1):
        raise ValueError(f"groups: expected {getattr(layout, 'n_groups', 1)}, got {len(groups)}")
    _check(lib.muon_step_scaled(_shard_array(layout, flat_params, "flat_params"),
                                _shard_array(layout, flat_grads, "flat_grads"),
                                _shard_array(layout, flat_momentum, "flat_momentum"),
                                layout.handle, _ptr(workspace), arr, int(ns_steps),
                                _ptr(grad_scale), _stream_handle(stream)), "muon_step_scaled")


def muon_compute_momentum_inputs(flat_grads, flat_momentum, layout, workspace, mu,
                                 nesterov=True, stream=None):
    _check(lib.muon_compute_momentum_inputs(
        _shard_array(layout, flat_grads, "flat_grads"),
        _shard_array(layout, flat_momentum, "flat_momentum"), layout.handle, _ptr(workspace),
        float(mu), 1 if nesterov else 0, _stream_handle(stream)), "muon_compute_momentum_inputs")


def muon_orthogonalize_updates(layout, workspace, ns_steps=5, stream=None):
    _check(lib.muon_orthogonalize_updates(layout.handle, _ptr(workspace), int(ns_steps),
                                          _stream_handle(stream)), "muon_orthogonalize_updates")


def muon_apply_local_updates(flat_params, layout, workspace, lr, wd, ns_steps=5, stream=None):
    _check(lib.muon_apply_local_updates(_shard_array(layout, flat_params, "flat_params"),
                                        layout.handle, _ptr(workspace), float(lr), float(wd),
                                        int(ns_steps), _stream_handle(stream)),
           "muon_apply_local_updates")


def muon_orthogonalize_apply(flat_params, layout, workspace, lr, wd, ns_steps=5, stream=None):
    _check(lib.muon_orthogonalize_apply(_shard_array(layout, flat_params, "flat_params"),
                                        layout.handle, _ptr(workspace), float(lr), float(wd),
                                        int(ns_steps), _stream_handle(stream)),
           "muon_orthogonalize_apply")


def muon_assign_owners(layout, ns_steps=5):
    """(owner per parameter, flop total per rank) for one rank per shard."""
    owner = (_I32 * max(1, len(layout.shapes)))()
    cost = (ctypes.c_double * max(1, layout.n_shards))()
    _check(lib.muon_assign_owners(layout.handle, int(ns_steps), owner, cost), "muon_assign_owners")
    return [owner[i] for i in range(len(layout.shapes))], [cost[s] for s in range(layout.n_shards)]


class Xfer(ctypes.Structure):
    """muon_xfer: one run of a matrix's flat elements moved between a shard and its
    owner's packed buffer."""
    _fields_ = [("param", ctypes.c_int32), ("src_rank", ctypes.c_int32),
                ("dst_rank", ctypes.c_int32), ("pad_", ctypes.c_int32),
                ("shard_off", ctypes.c_int64), ("owner_off", ctypes.c_int64),
                ("len", ctypes.c_int64)]


def muon_exchange_plan(layout, owner, rank):
    """(sends, recvs, owned_numel, owned_offsets) of the owner exchange for `rank`: sends
    and recvs are lists of dicts with the muon_xfer fields."""
    n = len(layout.shapes)
    own = (_I32 * max(1, n))(*[int(o) for o in owner])
    ns, nr, owned = _I64(0), _I64(0), _I64(0)
    _check(lib.muon_exchange_plan(layout.handle, own, int(rank), None, ctypes.byref(ns), None,
                                  ctypes.byref(nr), ctypes.byref(owned), None),
           "muon_exchange_plan")
    snd = (Xfer * max(1, ns.value))()
    rcv = (Xfer * max(1, nr.value))()
    offs = (_I64 * max(1, n))()
    _check(lib.muon_exchange_plan(layout.handle, own, int(rank), snd, ctypes.byref(ns), rcv,
                                  ctypes.byref(nr), ctypes.byref(owned), offs),
           "muon_exchange_plan")

    def rows(arr, k):
        return [{f: getattr(arr[i], f) for f, _ in Xfer._fields_ if f != "pad_"}
                for i in range(k)]
    return rows(snd, ns.value), rows(rcv, nr.value), owned.value, [offs[i] for i in range(n)]


def muon_gather_full(layout, shards, full, stream=None):
    _check(lib.muon_gather_full(layout.handle, _shard_array(layout, shards, "shards"), _ptr(full),
                                _stream_handle(stream)), "muon_gather_full")


def muon_scatter_updates(layout, full, shards, stream=None):
    _check(lib.muon_scatter_updates(layout.handle, _ptr(full), _shard_array(layout, shards, "shards"),
                                    _stream_handle(stream)), "muon_scatter_updates")


def muon_orthogonalize_full(layout, workspace, full_in, full_out, ns_steps=5, stream=None):
    _check(lib.muon_orthogonalize_full(layout.handle, _ptr(workspace), _ptr(full_in),
                                       _ptr(full_out), int(ns_steps), _stream_handle(stream)),
           "muon_orthogonalize_full")


def muon_orthogonalize_full_noalloc(layout, full_in, full_out, ns_steps=5, stream=None):
    """Like muon_orthogonalize_full, but with no workspace argument and no device
    allocation: for callers that cannot allocate device memory where they orthogonalize
    (fp32 layouts up to 32 MiB of tables plus workspace; see include/muon.h)."""
    _check(lib.muon_orthogonalize_full_noalloc(layout.handle, _ptr(full_in), _ptr(full_out),
                                               int(ns_steps), _stream_handle(stream)),
           "muon_orthogonalize_full_noalloc")


def muon_export_input(layout, workspace, full_out, stream=None):
    _check(lib.muon_export_input(layout.handle, _ptr(workspace), _ptr(full_out),
                                 _stream_handle(stream)), "muon_export_input")


def muon_export_update(layout, workspace, ns_steps, full_out, stream=None):
    _check(lib.muon_export_update(layout.handle, _ptr(workspace), int(ns_steps), _ptr(full_out),
                                  _stream_handle(stream)), "muon_export_update")


# ------------------------------------------------------------------ expert layers
# These calls are short, so their checks are: one look at each tensor's attributes, and torch's
# stream handle instead of a stream object.
_KINDS = {}   # torch dtype -> muon_dtype
_torch = None  # the module, once a tensor has come


def _kinds():
    global _torch
    import torch
    _torch = torch
    _KINDS.update({torch.float32: MUON_DTYPE_F32, torch.bfloat16: MUON_DTYPE_BF16,
                   torch.float16: MUON_DTYPE_F16})
    return _KINDS


def _kind(t, name):
    """t's muon_dtype."""
    k = _KINDS.get(t.dtype)
    if k is None:
        k = _kinds().get(t.dtype)
        if k is None:
            raise ValueError(f"{name}: type {t.dtype}; float32, bfloat16 or float16 is needed")
    return k


def _device_of(t, name):
    """The device that a call's tensors all have to be on: that of t, which has to be the current
    one, where the library launches."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if _torch is None:
        _kinds()
    if device != _torch.cuda.current_device():
        raise ValueError(f"{name}: on cuda:{device}, but cuda:{_torch.cuda.current_device()} is current")
    return device


def _on(t, name, device):
    if t.get_device() != device:
        raise ValueError(f"{name}: must be a CUDA tensor on cuda:{device}, as the call's others")


def _matrix(t, name, device, shape=None):
    """(pointer, row pitch, muon_dtype) of a 2-D tensor with contiguous rows.  Strides of
    dimensions of length 1 mean nothing."""
    size = t.shape
    _on(t, name, device)
    if len(size) != 2 or (shape is not None and size != shape):
        raise ValueError(f"{name}: shape {tuple(size)}, expected "
                         f"{'two dimensions' if shape is None else tuple(shape)}")
    pitch, step = t.stride()
    if step != 1 and size[1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), pitch if size[0] > 1 else max(size[1], 1), _kind(t, name)


def _matrices(t, name, device):
    """(pointer, pitch, distance between matrices, muon_dtype) of a 3-D tensor."""
    size = t.shape
    _on(t, name, device)
    if len(size) != 3:
        raise ValueError(f"{name}: must have three dimensions")
    apart, pitch, step = t.stride()
    if step != 1 and size[2] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return (t.data_ptr(), pitch if size[1] > 1 else max(size[2], 1),
            apart if size[0] > 1 else max(size[1] * size[2], 1), _kind(t, name))


def _row_floats(t, rows, name, device):
    """Pointer of a contiguous float32 vector of `rows` elements (None stays None)."""
    if t is None:
        return None
    _on(t, name, device)
    if t.shape != (rows,) or not t.is_contiguous() \
            or _kind(t, name) != MUON_DTYPE_F32:
        raise ValueError(f"{name}: must be {rows} contiguous float32 values")
    return t.data_ptr()


def _offsets(t, n_experts, device):
    _on(t, "offsets", device)
    if t.dtype != _torch.int64 or t.shape != (n_experts + 1,) or not t.is_contiguous():
        raise ValueError(f"offsets: must be {n_experts + 1} contiguous int64 values")
    return t.data_ptr()


def _stream_of(stream, device):
    """The handle of `stream`, or of the device's current stream."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _torch_stream(stream, device):
    """`stream` as torch's stream object (a handle of 0 or 1 is the default stream)."""
    if isinstance(stream, _torch.cuda.Stream):
        return stream
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    return (_torch.cuda.default_stream(device) if handle in (0, 1)
            else _torch.cuda.ExternalStream(handle, device=device))


def _workspace(workspace, nbytes, align, like, stream):
    """(pointer, bytes, owner) of the caller's workspace, or of one from torch's allocator: a block of
    `stream` itself, so that nothing pending elsewhere still uses it and work behind this call
    may have it next."""
    if workspace is not None:
        _on(workspace, "workspace", like.get_device())
        if not workspace.is_contiguous():
            raise ValueError("workspace: must be contiguous")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if nbytes == 0:
        return None, 0, None
    if stream is None:
        raw = _torch.empty(nbytes + align, dtype=_torch.uint8, device=like.device)
    else:
        with _torch.cuda.stream(_torch_stream(stream, like.device)):
            raw = _torch.empty(nbytes + align, dtype=_torch.uint8, device=like.device)
    at = raw.data_ptr()
    return at + (-at) % align, nbytes, raw


def muon_grouped_mm(x, w, offsets, y, trans_w=False, workspace=None, stream=None):
    """y[r] = x[r] @ w[e] (or @ w[e].T with trans_w) for the rows offsets[e]..offsets[e+1]-1 of
    every expert e; rows of no expert get zeros.

    x (rows, k) and w (experts, k, n) (trans_w: (experts, n, k)) are bfloat16 or float16, y
    (rows, n) is of their type or float32, offsets holds experts + 1 int64 values on the GPU.
    Any strides with a contiguous last dimension; operands whose rows do not start on 16 bytes
    are copied to the workspace first (allocated when None is given)."""
    device = _device_of(w, "w")
    wp, ldw, apart, dtype = _matrices(w, "w", device)
    e, k, n = w.shape
    if trans_w:
        k, n = n, k
    rows = x.shape[0]
    xp, ldx, xkind = _matrix(x, "x", device, (rows, k))
    yp, ldy, out = _matrix(y, "y", device, (rows, n))
    if xkind != dtype or dtype == MUON_DTYPE_F32 or out not in (dtype, MUON_DTYPE_F32):
        raise ValueError("x and w must both be bfloat16 or both float16, y of their type or float32")
    nbytes = 0
    if (xp | wp) & 15 or (ldx | ldw | apart) & 7:
        need = _SZ()
        _check(lib.muon_grouped_mm_workspace_bytes(xp, ldx, wp, ldw, apart, rows, e, k, n,
                                                   1 if trans_w else 0, ctypes.byref(need)),
               "muon_grouped_mm_workspace_bytes")
        nbytes = need.value
    ws, nbytes, owner = _workspace(workspace, nbytes, WORKSPACE_ALIGN, x, stream)
    st = lib.muon_grouped_mm(xp, ldx, wp, ldw, apart, _offsets(offsets, e, device), yp, ldy, rows, e, k,
                             n, 1 if trans_w else 0, dtype, out, ws, nbytes,
                             _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_grouped_mm")


def muon_grouped_wgrad(a, b, offsets, dw, accumulate=False, workspace=None, stream=None):
    """dw[e] = a[rows of e].T @ b[rows of e] in float32 for every expert e, or with accumulate
    dw[e] += that.  a (rows, m) and b (rows, n) are bfloat16 or float16; dw (experts, m, n) is
    float32 with any strides of its first two dimensions, e.g. a view of the flat gradient
    buffer."""
    device = _device_of(dw, "dw")
    dp, lddw, apart, out = _matrices(dw, "dw", device)
    e, m, n = dw.shape
    rows = a.shape[0]
    ap, lda, dtype = _matrix(a, "a", device, (rows, m))
    bp, ldb, bkind = _matrix(b, "b", device, (rows, n))
    if bkind != dtype or dtype == MUON_DTYPE_F32 or out != MUON_DTYPE_F32:
        raise ValueError("a and b must both be bfloat16 or both float16, and dw float32")
    nbytes = 0
    if (ap | bp) & 15 or (lda | ldb) & 7:
        need = _SZ()
        _check(lib.muon_grouped_wgrad_workspace_bytes(ap, lda, bp, ldb, rows, m, n,
                                                      ctypes.byref(need)),
               "muon_grouped_wgrad_workspace_bytes")
        nbytes = need.value
    ws, nbytes, owner = _workspace(workspace, nbytes, WORKSPACE_ALIGN, a, stream)
    st = lib.muon_grouped_wgrad(ap, lda, bp, ldb, _offsets(offsets, e, device), dp, lddw, apart, rows, e,
                                m, n, 1 if accumulate else 0, dtype, ws, nbytes,
                                _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_grouped_wgrad")


def muon_swiglu(gate, up, out, row_weight=None, stream=None):
    """out = row_weight[:, None] * silu(gate) * up, row by row; all (rows, cols) of one type."""
    device = _device_of(gate, "gate")
    g, ldg, dtype = _matrix(gate, "gate", device)
    shape = gate.shape
    u, ldu, ukind = _matrix(up, "up", device, shape)
    o, ldo, okind = _matrix(out, "out", device, shape)
    if ukind != dtype or okind != dtype:
        raise ValueError("gate, up and out must have the same type")
    st = lib.muon_swiglu(g, ldg, u, ldu, _row_floats(row_weight, shape[0], "row_weight", device), o, ldo,
                         shape[0], shape[1], dtype, _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_swiglu")


def muon_swiglu_grad(dout, gate, up, dgate, dup, row_weight=None, d_row_weight=None, stream=None):
    """The gradient of muon_swiglu: writes dgate, dup and, where given, d_row_weight."""
    device = _device_of(gate, "gate")
    g, ldg, dtype = _matrix(gate, "gate", device)
    shape = gate.shape
    d, ldd, dkind = _matrix(dout, "dout", device, shape)
    u, ldu, ukind = _matrix(up, "up", device, shape)
    dg, lddg, dgkind = _matrix(dgate, "dgate", device, shape)
    du, lddu, dukind = _matrix(dup, "dup", device, shape)
    if not dtype == dkind == ukind == dgkind == dukind:
        raise ValueError("dout, gate, up, dgate and dup must have the same type")
    st = lib.muon_swiglu_grad(d, ldd, g, ldg, u, ldu,
                              _row_floats(row_weight, shape[0], "row_weight", device), dg, lddg, du, lddu,
                              _row_floats(d_row_weight, shape[0], "d_row_weight", device), shape[0],
                              shape[1], dtype, _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_swiglu_grad")


# ------------------------------------------------------------------ gradient norm, clipping
def _tensor_list(tensors, name, device):
    """(array that owns it, address) of muon_tensor records (pointer, length, type as three
    64-bit words; the machine is little-endian) of contiguous tensors."""
    kinds = _KINDS or _kinds()
    try:
        flat = [v for t in tensors for v in (t.data_ptr(), t.numel(), kinds[t.dtype])]
    except KeyError as e:
        raise ValueError(f"{name}: type {e.args[0]}; float32, bfloat16 or float16 is needed") from None
    if not all([t.get_device() == device and t.is_contiguous() for t in tensors]):
        raise ValueError(f"{name}: must be contiguous CUDA tensors on cuda:{device}, as norm")
    words = array.array("Q", flat)
    return words, words.buffer_info()[0]


def _clip_call(grads, norm, workspace, stream):
    """(grads' records and their owner, norm's pointer, workspace pointer, bytes and owner,
    stream)."""
    device = _device_of(norm, "norm")
    np = _row_floats(norm, 2, "norm", device)
    words, g = _tensor_list(grads, "grads", device)
    nbytes = 0
    if workspace is None:
        need = _SZ()
        _check(lib.muon_clip_workspace_bytes(g, len(grads), ctypes.byref(need)),
               "muon_clip_workspace_bytes")
        nbytes = need.value
    ws, nbytes, owner = _workspace(workspace, nbytes, 8, norm, stream)
    return g, words, np, ws, nbytes, owner, _stream_of(stream, device)


def muon_grad_norm(grads, max_norm, norm, workspace=None, stream=None):
    """norm[0] = the 2-norm of all gradients together, norm[1] = min(1, max_norm / (norm[0] +
    1e-6)).  grads: a sequence of contiguous CUDA tensors; norm: 2 float32 on the GPU."""
    g, words, np, ws, nbytes, owner, st = _clip_call(grads, norm, workspace, stream)
    _check(lib.muon_grad_norm(g, len(grads), max_norm, np, ws, nbytes, st), "muon_grad_norm")


def muon_clip_grads(grads, outs, max_norm, norm, workspace=None, stream=None):
    """muon_grad_norm, and outs[i] = norm[1] * grads[i].  outs[i] is grads[i] itself or a tensor
    of its length and of its type or float32."""
    if len(outs) != len(grads):
        raise ValueError(f"outs: {len(outs)} tensors for {len(grads)} gradients")
    out_words, o = _tensor_list(outs, "outs", _device_of(norm, "norm"))
    g, words, np, ws, nbytes, owner, st = _clip_call(grads, norm, workspace, stream)
    _check(lib.muon_clip_grads(g, o, len(grads), max_norm, np, ws, nbytes, st), "muon_clip_grads")


def layout_grads(layout, flat_grads):
    """The shards of a flat buffer without the padding behind the last one: what
    muon_grad_norm sums over for the global norm of a layout's gradients."""
    if not isinstance(flat_grads, (list, tuple)):
        flat_grads = [flat_grads]
    return [g[:max(0, min(layout.shard_len, layout.numel - s * layout.shard_len))]
            for s, g in enumerate(flat_grads)]


# ------------------------------------------------------------------ feed-forward operators
def muon_layer_norm(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, stream=None):
    """y = (x - mean) * rstd * weight + bias, row by row; x and y (rows, cols) of one type.

    weight and bias: cols float32 values (None: 1 and 0); mean and rstd: None, or rows float32
    values that the gradient will take."""
    device = _device_of(x, "x")
    xp, ldx, dtype = _matrix(x, "x", device)
    rows, cols = x.shape
    yp, ldy, ykind = _matrix(y, "y", device, x.shape)
    if ykind != dtype:
        raise ValueError("x and y must have the same type")
    st = lib.muon_layer_norm(xp, ldx, _row_floats(weight, cols, "weight", device),
                             _row_floats(bias, cols, "bias", device), yp, ldy,
                             _row_floats(mean, rows, "mean", device),
                             _row_floats(rstd, rows, "rstd", device), rows, cols, eps, dtype,
                             _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_layer_norm")


def muon_layer_norm_grad(dy, x, weight, mean, rstd, dx, dweight, dbias, accumulate=False,
                         workspace=None, stream=None):
    """The gradient of muon_layer_norm: writes dx, and dweight and dbias (float32, None: not wanted),
    or with accumulate adds to those two."""
    device = _device_of(x, "x")
    xp, ldx, dtype = _matrix(x, "x", device)
    rows, cols = x.shape
    dyp, lddy, dykind = _matrix(dy, "dy", device, x.shape)
    dxp, lddx, dxkind = _matrix(dx, "dx", device, x.shape)
    if not dtype == dykind == dxkind:
        raise ValueError("dy, x and dx must have the same type")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd: the forward pass's are needed")
    nbytes = 0
    if workspace is None and (dweight is not None or dbias is not None):
        need = _SZ()
        _check(lib.muon_layer_norm_grad_workspace_bytes(rows, cols, ctypes.byref(need)),
               "muon_layer_norm_grad_workspace_bytes")
        nbytes = need.value
    ws, nbytes, owner = _workspace(workspace, nbytes, 16, x, stream)
    st = lib.muon_layer_norm_grad(dyp, lddy, xp, ldx, _row_floats(weight, cols, "weight", device),
                                  _row_floats(mean, rows, "mean", device),
                                  _row_floats(rstd, rows, "rstd", device), dxp, lddx,
                                  _row_floats(dweight, cols, "dweight", device),
                                  _row_floats(dbias, cols, "dbias", device), rows, cols,
                                  1 if accumulate else 0, dtype, ws, nbytes,
                                  _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_layer_norm_grad")


def _product_offsets(offsets, n_experts, device):
    """The row offsets' pointer; None: one expert owns every row."""
    if offsets is None:
        if n_experts != 1:
            raise ValueError(f"offsets: needed for {n_experts} experts")
        return None
    return _offsets(offsets, n_experts, device)


def _same_shape(w, other, name):
    if other.shape != w.shape:
        raise ValueError(f"{name}: shape {tuple(other.shape)}, expected {tuple(w.shape)}")


def _optional_matrix(t, name, device, shape, dtype):
    """(pointer, pitch) of a matrix of the call's type, or of None."""
    if t is None:
        return None, 0
    p, ld, kind = _matrix(t, name, device, shape)
    if kind != dtype:
        raise ValueError(f"{name}: must have the type of the call's other matrices")
    return p, ld


def _need(call, *args):
    """The bytes of workspace that a query reports."""
    need = _SZ()
    _check(getattr(lib, call)(*args, ctypes.byref(need)), call)
    return need.value


def muon_gated_mm(x, w_gate, w_up, offsets, out, gate=None, up=None, row_weight=None, trans_w=False,
                  workspace=None, stream=None):
    """out[r] = row_weight[r] * silu(x[r] @ w_gate[e]) * (x[r] @ w_up[e]) in one kernel (trans_w:
    w.T) for the rows offsets[e]..offsets[e+1]-1 of every expert e; rows of no expert get zeros.

    x (rows, k), both weights (experts, k, n) (trans_w: (experts, n, k)) and out (rows, n) are all
    bfloat16 or all float16.  offsets: experts + 1 int64 values on the GPU, or None for one expert
    that owns every row.  gate and up: None, or receive the two products for muon_gated_mm_grad."""
    device = _device_of(w_gate, "w_gate")
    wp, ldw, apart, dtype = _matrices(w_gate, "w_gate", device)
    _same_shape(w_gate, w_up, "w_up")
    up_p, ldw_up, up_apart, up_kind = _matrices(w_up, "w_up", device)
    e, k, n = w_gate.shape
    if trans_w:
        k, n = n, k
    rows = x.shape[0]
    xp, ldx, xkind = _matrix(x, "x", device, (rows, k))
    op, ldo, okind = _matrix(out, "out", device, (rows, n))
    if not dtype == up_kind == xkind == okind or dtype == MUON_DTYPE_F32:
        raise ValueError("x, w_gate, w_up and out must all be bfloat16 or all float16")
    gp, ldg = _optional_matrix(gate, "gate", device, (rows, n), dtype)
    upp, ldu = _optional_matrix(up, "up", device, (rows, n), dtype)
    trans = 1 if trans_w else 0
    nbytes = 0
    if (xp | wp | up_p) & 15 or (ldx | ldw | apart | ldw_up | up_apart) & 7:
        nbytes = _need("muon_gated_mm_workspace_bytes", xp, ldx, wp, ldw, apart, up_p, ldw_up, up_apart,
                       rows, e, k, n, trans)
    ws, nbytes, owner = _workspace(workspace, nbytes, WORKSPACE_ALIGN, x, stream)
    st = lib.muon_gated_mm(xp, ldx, wp, ldw, apart, up_p, ldw_up, up_apart,
                           _product_offsets(offsets, e, device),
                           _row_floats(row_weight, rows, "row_weight", device), op, ldo, gp, ldg, upp,
                           ldu, rows, e, k, n, trans, dtype, ws, nbytes, _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_gated_mm")


def muon_gated_mm_grad(dy, w, offsets, gate, up, dgate, dup, out=None, row_weight=None,
                       d_row_weight=None, trans_w=False, workspace=None, stream=None):
    """Backward through a gated block's second product and its activation in one kernel: from dh =
    dy @ w[e] (trans_w: w[e].T, which a down projection stored (inner, hidden) takes), which is never
    stored, and the forward pass's gate and up, writes dgate and dup and, where given, out (the
    activation, for the second product's weight gradient) and d_row_weight.

    dy (rows, k), gate, up, dgate, dup and out (rows, n) and w are all bfloat16 or all float16."""
    device = _device_of(w, "w")
    wp, ldw, apart, dtype = _matrices(w, "w", device)
    e, k, n = w.shape
    if trans_w:
        k, n = n, k
    rows = dy.shape[0]
    yp, ldy, ykind = _matrix(dy, "dy", device, (rows, k))
    g, ldg, gkind = _matrix(gate, "gate", device, (rows, n))
    u, ldu, ukind = _matrix(up, "up", device, (rows, n))
    dg, lddg, dgkind = _matrix(dgate, "dgate", device, (rows, n))
    du, lddu, dukind = _matrix(dup, "dup", device, (rows, n))
    if not dtype == ykind == gkind == ukind == dgkind == dukind or dtype == MUON_DTYPE_F32:
        raise ValueError("dy, w, gate, up, dgate and dup must all be bfloat16 or all float16")
    op, ldo = _optional_matrix(out, "out", device, (rows, n), dtype)
    trans = 1 if trans_w else 0
    nbytes = 0
    if d_row_weight is not None or (yp | wp) & 15 or (ldy | ldw | apart) & 7:
        nbytes = _need("muon_gated_mm_grad_workspace_bytes", yp, ldy, wp, ldw, apart, rows, e, k, n,
                       trans, 0 if d_row_weight is None else 1)
    ws, nbytes, owner = _workspace(workspace, nbytes, WORKSPACE_ALIGN, dy, stream)
    st = lib.muon_gated_mm_grad(yp, ldy, wp, ldw, apart, _product_offsets(offsets, e, device), g, ldg, u,
                                ldu, _row_floats(row_weight, rows, "row_weight", device), dg, lddg, du,
                                lddu, op, ldo, _row_floats(d_row_weight, rows, "d_row_weight", device),
                                rows, e, k, n, trans, dtype, ws, nbytes, _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_gated_mm_grad")


def muon_grouped_mm_sum(x1, w1, x2, w2, offsets, y, trans_w=False, workspace=None, stream=None):
    """y[r] = x1[r] @ w1[e] + x2[r] @ w2[e] (trans_w: w.T), summed before the one rounding, for the
    rows offsets[e]..offsets[e+1]-1 of every expert e (offsets None: one expert owns every row).

    x1 and x2 (rows, k), w1 and w2 (experts, k, n) (trans_w: (experts, n, k)) are all bfloat16 or
    all float16, y (rows, n) is of their type or float32."""
    device = _device_of(w1, "w1")
    p1, ldw1, apart1, dtype = _matrices(w1, "w1", device)
    _same_shape(w1, w2, "w2")
    p2, ldw2, apart2, kind2 = _matrices(w2, "w2", device)
    e, k, n = w1.shape
    if trans_w:
        k, n = n, k
    rows = x1.shape[0]
    a, lda, akind = _matrix(x1, "x1", device, (rows, k))
    b, ldb, bkind = _matrix(x2, "x2", device, (rows, k))
    yp, ldy, out = _matrix(y, "y", device, (rows, n))
    if not dtype == kind2 == akind == bkind or dtype == MUON_DTYPE_F32 or out not in (dtype, MUON_DTYPE_F32):
        raise ValueError("x1, w1, x2 and w2 must all be bfloat16 or all float16, y of their type or float32")
    trans = 1 if trans_w else 0
    nbytes = 0
    if (a | b | p1 | p2) & 15 or (lda | ldb | ldw1 | apart1 | ldw2 | apart2) & 7:
        nbytes = _need("muon_grouped_mm_sum_workspace_bytes", a, lda, p1, ldw1, apart1, b, ldb, p2, ldw2,
                       apart2, rows, e, k, n, trans)
    ws, nbytes, owner = _workspace(workspace, nbytes, WORKSPACE_ALIGN, x1, stream)
    st = lib.muon_grouped_mm_sum(a, lda, p1, ldw1, apart1, b, ldb, p2, ldw2, apart2,
                                 _product_offsets(offsets, e, device), yp, ldy, rows, e, k, n, trans,
                                 dtype, out, ws, nbytes, _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_grouped_mm_sum")


FP8_BLOCK = 128   # elements (of a row), or rows and columns (of a weight), that share a scale


def _fp8_blocks(n):
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def _fp8(t, name, device, dims):
    """(pointer, strides) of an e4m3 tensor with contiguous rows; a single row's (or matrix's) stride
    means nothing and counts as the least that works."""
    _on(t, name, device)
    size, step = t.shape, t.stride()
    if t.dtype != _torch.float8_e4m3fn or len(size) != dims:
        raise ValueError(f"{name}: must be a float8_e4m3fn tensor of {dims} dimensions")
    if step[-1] != 1 and size[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    pitch = step[-2] if size[-2] > 1 else max(size[-1], 1)
    if dims == 2:
        return t.data_ptr(), pitch
    return t.data_ptr(), pitch, step[0] if size[0] > 1 else max(size[1], 1) * pitch


def muon_quantize_rows(x, q, scale, stream=None):
    """x (rows, cols; any type) to q (rows, cols) in float8_e4m3fn, with scale (blocks of 128 columns,
    rows) in float32: q * scale is x but for the rounding to e4m3."""
    device = _device_of(x, "x")
    xp, ldx, dtype = _matrix(x, "x", device)
    rows, cols = x.shape
    qp, ldq = _fp8(q, "q", device, 2)
    if q.shape != x.shape:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected {tuple(x.shape)}")
    sp, ld_scale, kind = _matrix(scale, "scale", device, (_fp8_blocks(cols), rows))
    if kind != MUON_DTYPE_F32:
        raise ValueError("scale: must be float32")
    st = lib.muon_quantize_rows(xp, ldx, qp, ldq, sp, ld_scale, rows, cols, dtype,
                                _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_quantize_rows")


def muon_quantize_weights(w, q, scale, transpose=False, stream=None):
    """w (n, rows, cols; any type) to q in float8_e4m3fn, (n, rows, cols) or with transpose (n, cols,
    rows), with a float32 scale for each 128 x 128 block in q's order (n, blocks, blocks; contiguous)."""
    device = _device_of(w, "w")
    wp, ldw, apart, dtype = _matrices(w, "w", device)
    n, rows, cols = w.shape
    want = (n, cols, rows) if transpose else (n, rows, cols)
    qp, ldq, q_apart = _fp8(q, "q", device, 3)
    if q.shape != want:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected {want}")
    _on(scale, "scale", device)
    blocks = (n, _fp8_blocks(want[1]), _fp8_blocks(want[2]))
    if scale.shape != blocks or not scale.is_contiguous() or _kind(scale, "scale") != MUON_DTYPE_F32:
        raise ValueError(f"scale: must be {blocks} contiguous float32 values")
    st = lib.muon_quantize_weights(wp, ldw, apart, qp, ldq, q_apart, scale.data_ptr(), n, rows, cols,
                                   1 if transpose else 0, dtype, _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_quantize_weights")


def muon_grouped_mm_fp8(x, x_scale, w, w_scale, offsets, y, stream=None):
    """y[r] = x[r] @ w[e].T for the rows offsets[e]..offsets[e+1]-1 of every expert e (offsets None: one
    expert owns every row), from e4m3 values and the scales of muon_quantize_rows and
    muon_quantize_weights.

    x (rows, k) and w (experts, n, k) are float8_e4m3fn with rows that start on 16 bytes, y (rows, n) is
    bfloat16, float16 or float32."""
    device = _device_of(w, "w")
    wp, ldw, apart = _fp8(w, "w", device, 3)
    e, n, k = w.shape
    rows = x.shape[0]
    xp, ldx = _fp8(x, "x", device, 2)
    if x.shape[1] != k:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected {(rows, k)}")
    blocks = _fp8_blocks(k)
    xs, ld_xs, xs_kind = _matrix(x_scale, "x_scale", device, (blocks, rows))
    _on(w_scale, "w_scale", device)
    if xs_kind != MUON_DTYPE_F32 or _kind(w_scale, "w_scale") != MUON_DTYPE_F32 \
            or w_scale.shape != (e, _fp8_blocks(n), blocks) or not w_scale.is_contiguous():
        raise ValueError(f"x_scale and w_scale: must be {(blocks, rows)} and contiguous "
                         f"{(e, _fp8_blocks(n), blocks)} float32 values")
    yp, ldy, out = _matrix(y, "y", device, (rows, n))
    st = lib.muon_grouped_mm_fp8(xp, ldx, xs, ld_xs, wp, ldw, apart, w_scale.data_ptr(),
                                 _product_offsets(offsets, e, device), yp, ldy, rows, e, k, n, out,
                                 _stream_of(stream, device))
    if st != MUON_OK:
        raise MuonError(st, "muon_grouped_mm_fp8")


def muon_check(stream=None):
    _check(lib.muon_check(_stream_handle(stream)), "muon_check")


def muon_check_status(stream=None) -> int:
    """Like muon_check but returns the status instead of raising."""
    return lib.muon_check(_stream_handle(stream))


def muon_selftest_wait_timeout(budget_cycles, stream=None):
    _check(lib.muon_selftest_wait_timeout(int(budget_cycles), _stream_handle(stream)),
           "muon_selftest_wait_timeout")


def muon_debug_build() -> bool:
    """Whether the loaded library was built with device-side range checks."""
    return bool(lib.muon_debug_build())


def muon_selftest_device_check(stream=None):
    _check(lib.muon_selftest_device_check(_stream_handle(stream)), "muon_selftest_device_check")


def muon_layout_ns_kernel(layout) -> dict:
    """The Newton-Schulz kernel `layout` runs on the current device:
    {"tile_shape": 1 single CTA | 2 CTA pair | 3 CTA pair with 256x512 tiles (0: none),
     "units": int, "persistent": bool}."""
    shape, units, pers = _I32(), _I32(), _I32()
    _check(lib.muon_layout_ns_kernel(layout.handle, ctypes.byref(shape), ctypes.byref(units),
                                     ctypes.byref(pers)), "muon_layout_ns_kernel")
    return {"tile_shape": int(shape.value), "units": int(units.value),
            "persistent": bool(pers.value)}


def muon_layout_fused_apply(layout) -> bool:
    """True when muon_step / muon_orthogonalize_apply apply the update to W inside the last
    Newton-Schulz Update on the current device, False when a separate apply pass runs."""
    f = _I32()
    _check(lib.muon_layout_fused_apply(layout.handle, ctypes.byref(f)), "muon_layout_fused_apply")
    return bool(f.value)


def muon_last_error() -> str:
    return lib.muon_last_error().decode(errors="replace")


def muon_abi_version() -> int:
    return lib.muon_abi_version()
