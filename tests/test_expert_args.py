"""Argument checks of the expert-layer entry points, on the host: every refusal comes back as a
status with a message before anything is launched.  The pointers are made up; no call here
passes its checks."""
import ctypes

import pytest

capi = pytest.importorskip("muon_optimizer_step_gb300.capi",
                           reason="libmuon.so not built (run __graft_entry__.build())")
torch = pytest.importorskip("torch")

INV, ALIGN = capi.MUON_ERR_INVALID_ARG, capi.MUON_ERR_ALIGNMENT
BF16, F16, F32 = capi.MUON_DTYPE_BF16, capi.MUON_DTYPE_F16, capi.MUON_DTYPE_F32

MM = dict(x=0x10000, ldx=64, w=0x20000, ldw=32, w_stride=2048, off=0x30000, y=0x40000, ldy=32, rows=10,
          experts=4, k=64, n=32, trans=0, dtype=BF16, out=BF16, ws=None, ws_bytes=0, stream=None)
WG = dict(a=0x10000, lda=64, b=0x20000, ldb=32, off=0x30000, dw=0x40000, lddw=32, stride=2048, rows=10,
          experts=4, m=64, n=32, acc=0, dtype=BF16, ws=None, ws_bytes=0, stream=None)
SW = dict(g=0x10000, ldg=8, u=0x20000, ldu=8, p=None, o=0x30000, ldo=8, rows=4, cols=8, dtype=BF16,
          stream=None)
SG = dict(d=0x10000, ldd=8, g=0x20000, ldg=8, u=0x30000, ldu=8, p=None, dg=0x40000, lddg=8, du=0x50000,
          lddu=8, dp=None, rows=4, cols=8, dtype=BF16, stream=None)


@pytest.mark.parametrize("base,call,bad,status", [
    (MM, "muon_grouped_mm", bad, status) for bad, status in [
        (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(off=None), INV),
        (dict(x=0x10001), ALIGN), (dict(w=0x20001), ALIGN), (dict(y=0x40001), ALIGN),
        (dict(off=0x30004), ALIGN), (dict(out=F32, y=0x40002), ALIGN), (dict(ldx=63), INV),
        (dict(ldw=31), INV), (dict(trans=1, ldw=63), INV), (dict(ldy=31), INV), (dict(w_stride=0), INV),
        (dict(w_stride=-2048), INV), (dict(ldx=1 << 40), INV), (dict(rows=-1), INV),
        (dict(rows=1 << 31), INV), (dict(experts=0), INV), (dict(experts=1025), INV), (dict(k=0), INV),
        (dict(n=-3), INV), (dict(dtype=F32), INV), (dict(dtype=3), INV), (dict(out=F16), INV),
        (dict(rows=(1 << 31) - 1, n=(1 << 31) - 1, ldw=1 << 31, ldy=1 << 31), capi.MUON_ERR_UNSUPPORTED),
        (dict(x=0x10002), INV),                           # needs a workspace
        (dict(ldx=65, ws=0x50000, ws_bytes=16), INV),     # too small
        (dict(ldx=65, ws=0x50010, ws_bytes=1 << 20), ALIGN),
    ]] + [
    (WG, "muon_grouped_wgrad", bad, status) for bad, status in [
        (dict(a=None), INV), (dict(b=None), INV), (dict(dw=None), INV), (dict(dw=0x40002), ALIGN),
        (dict(off=None), INV), (dict(lda=63), INV), (dict(ldb=31), INV), (dict(lddw=31), INV),
        (dict(stride=31), INV), (dict(rows=-1), INV), (dict(experts=0), INV), (dict(m=0), INV),
        (dict(n=0), INV), (dict(dtype=F32), INV), (dict(ldb=33), INV),
        (dict(m=1 << 30, lda=1 << 30, n=1 << 30, ldb=1 << 30, lddw=1 << 30, stride=1 << 31),
         capi.MUON_ERR_UNSUPPORTED),
    ]] + [
    (SW, "muon_swiglu", bad, status) for bad, status in [
        (dict(g=None), INV), (dict(u=0x20001), ALIGN), (dict(o=None), INV), (dict(ldg=7), INV),
        (dict(cols=0), INV), (dict(rows=-1), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV),
        (dict(p=0x60002), ALIGN), (dict(dtype=F32, g=0x10002), ALIGN),
    ]] + [
    (SG, "muon_swiglu_grad", bad, status) for bad, status in [
        (dict(d=None), INV), (dict(dg=None), INV), (dict(du=0x50001), ALIGN), (dict(lddu=7), INV),
        (dict(dp=0x60002), ALIGN), (dict(rows=1 << 31), INV), (dict(cols=-1), INV),
    ]])
def test_refusals(base, call, bad, status):
    args = {**base, **bad}
    assert getattr(capi.lib, call)(*args.values()) == status
    assert capi.muon_last_error()


def _list(*records):
    words = [v for r in records for v in r]
    return (ctypes.c_uint64 * max(3, len(words)))(*words)


@pytest.mark.parametrize("grads,outs,n,max_norm,norm,status", [
    (None, None, 1, 1.0, 0x9000, INV),
    (_list((0x1000, 4, F32)), None, -1, 1.0, 0x9000, INV),
    (_list((0x1000, 4, 3)), _list((0x1000, 4, 3)), 1, 1.0, 0x9000, INV),
    (_list((0, 4, F32)), _list((0x1000, 4, F32)), 1, 1.0, 0x9000, INV),
    (_list((0x1002, 4, F32)), _list((0x1000, 4, F32)), 1, 1.0, 0x9000, ALIGN),
    (_list((0x1000, 4, F32)), _list((0x1000, 5, F32)), 1, 1.0, 0x9000, INV),
    (_list((0x1000, 4, F32)), _list((0x1000, 4, BF16)), 1, 1.0, 0x9000, INV),
    (_list((0x1000, 4, BF16)), _list((0x1000, 4, F16)), 1, 1.0, 0x9000, INV),
    (_list((0x1000, 4, BF16)), _list((0x1000, 4, F32)), 1, 1.0, 0x9000, INV),   # in place, wider
    (_list((0x1000, (1 << 64) - 4, F32)), _list((0x1000, (1 << 64) - 4, F32)), 1, 1.0, 0x9000, INV),
    (_list((0x1000, 4, F32)), _list((0x1000, 4, F32)), 1, -0.5, 0x9000, INV),
    (_list((0x1000, 4, F32)), _list((0x1000, 4, F32)), 1, float("nan"), 0x9000, INV),
    (_list((0x1000, 4, F32)), _list((0x1000, 4, F32)), 1, float("inf"), 0x9000, INV),
    (_list((0x1000, 4, F32)), _list((0x1000, 4, F32)), 1, 1.0, None, INV),
    (_list((0x1000, 4, F32)), _list((0x1000, 4, F32)), 1, 1.0, 0x9002, ALIGN),
])
def test_clip_refusals(grads, outs, n, max_norm, norm, status):
    assert capi.lib.muon_clip_grads(grads, outs, n, max_norm, norm, None, 0, None) == status
    assert capi.muon_last_error()


def test_scaled_step_refusals():
    lay = capi.muon_layout_create([(8, 8)], 1, 0)
    shards = (ctypes.c_void_p * 1)(0x1000)
    groups = (capi.GroupHparams * 1)(capi.GroupHparams(0.1, 0.0, 0.9, 1))

    def call(scale, layout=lay.handle, ws=0x10000, g=groups):
        return capi.lib.muon_step_scaled(shards, shards, shards, layout, ws, g, 5, scale, None)

    assert call(None) == INV
    assert call(0x2002) == ALIGN
    assert call(0x2000, layout=None) == INV
    assert call(0x2000, ws=0x10010) == ALIGN
    assert call(0x2000, g=None) == INV


def test_workspace_sizes():
    """Nothing for operands whose rows start on 16 bytes; else whole copies, rows on 16 or 128 bytes."""
    def mm(x=0x1000, ldx=64, w=0x2000, ldw=32, stride=2048, rows=10, e=4, k=64, n=32, trans=0):
        v = ctypes.c_size_t()
        assert capi.lib.muon_grouped_mm_workspace_bytes(x, ldx, w, ldw, stride, rows, e, k, n, trans,
                                                        ctypes.byref(v)) == capi.MUON_OK
        return v.value

    assert mm() == 0
    assert mm(rows=0, x=None, w=None, ldx=65) == 0
    assert mm(ldx=72, ldw=40, stride=4096) == 0
    assert 10 * 64 * 2 <= mm(ldx=65) <= 10 * 64 * 2 + 1024
    assert mm(rows=1, ldx=65) == 0 and mm(rows=1, x=0x1002) > 0
    assert 10 * 128 * 2 <= mm(k=65, ldx=65) <= 10 * 128 * 2 + 1024      # whole 128-byte lines
    assert 10 * 64 * 2 <= mm(x=0x1002) <= 10 * 64 * 2 + 1024
    assert 4 * 64 * 32 * 2 <= mm(ldw=33) <= 4 * 64 * 32 * 2 + 1024
    assert 4 * 64 * 32 * 2 <= mm(stride=2049) <= 4 * 64 * 32 * 2 + 1024
    assert mm(stride=2049, e=1) == 0
    assert 4 * 5 * 128 * 2 <= mm(trans=1, n=5, k=65, ldw=65, ldx=72, stride=512) <= 4 * 5 * 128 * 2 + 1024
    v = ctypes.c_size_t()
    assert capi.lib.muon_grouped_wgrad_workspace_bytes(0x1000, 65, 0x2002, 32, 10, 64, 32,
                                                       ctypes.byref(v)) == capi.MUON_OK
    assert 10 * 96 * 2 <= v.value <= 10 * 96 * 2 + 2048
    assert capi.lib.muon_grouped_mm_workspace_bytes(0x1000, 64, 0x2000, 32, 2048, 10, 4, 64, 32, 0,
                                                    None) == INV
    assert capi.lib.muon_clip_workspace_bytes(None, 0, None) == INV


def test_layout_grads_leaves_out_the_padding():
    lay = capi.muon_layout_create([(5, 5), (3, 1)], 3, 0, [True, False])   # 28 elements, shards of 10
    shards = [torch.zeros(12) for _ in range(3)]
    assert [t.numel() for t in capi.layout_grads(lay, shards)] == [10, 10, 8]
    lay = capi.muon_layout_create([(1, 2)], 4, 0)                          # shards without elements
    assert [t.numel() for t in capi.layout_grads(lay, [torch.zeros(1)] * 4)] == [1, 1, 0, 0]


def test_binding_refuses_host_tensors():
    x, w, y = torch.zeros(4, 8).bfloat16(), torch.zeros(2, 8, 8).bfloat16(), torch.zeros(4, 8).bfloat16()
    off = torch.tensor([0, 2, 4])
    with pytest.raises(ValueError):
        capi.muon_grouped_mm(x, w, off, y)
    with pytest.raises(ValueError):
        capi.muon_grouped_wgrad(x, y, off, w.float())
    with pytest.raises(ValueError):
        capi.muon_swiglu(x, x, x)
    with pytest.raises(ValueError):
        capi.muon_swiglu_grad(x, x, x, x, x)
    with pytest.raises(ValueError):
        capi.muon_grad_norm([x], 1.0, torch.zeros(2))
