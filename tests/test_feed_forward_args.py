"""Argument checks of the feed-forward entry points, on the host: every refusal comes back as a
status with a message before anything is launched.  The pointers are made up; no call here passes
its checks."""
import ctypes

import pytest

capi = pytest.importorskip("muon_optimizer_step_gb300.capi",
                           reason="libmuon.so not built (run __graft_entry__.build())")
torch = pytest.importorskip("torch")

INV, ALIGN = capi.MUON_ERR_INVALID_ARG, capi.MUON_ERR_ALIGNMENT
BF16, F16, F32 = capi.MUON_DTYPE_BF16, capi.MUON_DTYPE_F16, capi.MUON_DTYPE_F32

LN = dict(x=0x10000, ldx=64, w=0x20000, b=0x30000, y=0x40000, ldy=64, mean=None, rstd=None, rows=4, cols=64,
          eps=1e-5, dtype=BF16, stream=None)
LG = dict(dy=0x10000, lddy=64, x=0x20000, ldx=64, w=0x30000, mean=0x40000, rstd=0x50000, dx=0x60000, lddx=64,
          dw=0x70000, db=0x80000, rows=4, cols=64, acc=0, dtype=BF16, ws=0x90000, ws_bytes=1 << 20, stream=None)
CASES = [
    (LN, "muon_layer_norm", bad, status) for bad, status in [
        (dict(x=None), INV), (dict(y=None), INV), (dict(x=0x10001), ALIGN), (dict(y=0x40001), ALIGN),
        (dict(dtype=F32, x=0x10002), ALIGN), (dict(w=0x20002), ALIGN), (dict(b=0x30001), ALIGN),
        (dict(mean=0x50002), ALIGN), (dict(rstd=0x50002), ALIGN), (dict(ldx=63), INV), (dict(ldy=63), INV),
        (dict(ldx=1 << 36), INV), (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(cols=0), INV),
        (dict(cols=-5), INV), (dict(eps=-1e-5), INV), (dict(eps=float("nan")), INV),
        (dict(eps=float("inf")), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV),
    ]] + [
    (LG, "muon_layer_norm_grad", bad, status) for bad, status in [
        (dict(dy=None), INV), (dict(x=None), INV), (dict(dx=None), INV), (dict(mean=None), INV),
        (dict(rstd=None), INV), (dict(dy=0x10001), ALIGN), (dict(dx=0x60001), ALIGN),
        (dict(w=0x30002), ALIGN), (dict(mean=0x40002), ALIGN), (dict(dw=0x70002), ALIGN),
        (dict(db=0x80001), ALIGN), (dict(lddy=63), INV), (dict(ldx=63), INV), (dict(lddx=63), INV),
        (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(cols=0), INV), (dict(dtype=4), INV),
        (dict(ws=None), INV), (dict(ws_bytes=4 * 2 * 64 * 4 - 1), INV), (dict(ws=0x90008), ALIGN),
        (dict(dw=None, ws_bytes=0), INV),
    ]]


@pytest.mark.parametrize("base,call,bad,status", CASES)
def test_refusals(base, call, bad, status):
    args = {**base, **bad}
    assert getattr(capi.lib, call)(*args.values()) == status
    assert capi.muon_last_error()


def test_layer_norm_workspace():
    v = ctypes.c_size_t()

    def size(rows, cols):
        assert capi.lib.muon_layer_norm_grad_workspace_bytes(rows, cols, ctypes.byref(v)) == capi.MUON_OK
        return v.value

    assert size(0, 64) == 0
    assert size(4, 64) == 4 * 2 * 64 * 4
    assert size(100_000, 4096) == 608 * 2 * 4096 * 4
    assert size(100_000, 16385) == 304 * 2 * 16385 * 4
    assert size((1 << 31) - 1, (1 << 31) - 1) == 304 * 2 * ((1 << 31) - 1) * 4
    for bad in ((-1, 64), (4, 0)):
        assert capi.lib.muon_layer_norm_grad_workspace_bytes(*bad, ctypes.byref(v)) == INV
    assert capi.lib.muon_layer_norm_grad_workspace_bytes(4, 64, None) == INV
