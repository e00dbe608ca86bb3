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


GM = dict(x=0x10000, ldx=64, wg=0x20000, ldwg=32, sg=2048, wu=0x30000, ldwu=32, su=2048, off=0x40000, p=None,
          out=0x50000, ldo=32, gate=None, ldg=0, up=None, ldu=0, rows=10, experts=4, k=64, n=32, trans=0, dtype=BF16,
          ws=None, ws_bytes=0, stream=None)
GG = dict(dy=0x10000, lddy=64, w=0x20000, ldw=64, sw=2048, off=0x30000, gate=0x40000, ldg=32, up=0x50000, ldu=32,
          p=None, dgate=0x60000, lddg=32, dup=0x70000, lddu=32, out=None, ldo=0, dp=None, rows=10, experts=4, k=64,
          n=32, trans=1, dtype=BF16, ws=None, ws_bytes=0, stream=None)
MS = dict(x1=0x10000, ldx1=64, w1=0x20000, ldw1=32, s1=2048, x2=0x30000, ldx2=64, w2=0x40000, ldw2=32, s2=2048,
          off=0x50000, y=0x60000, ldy=32, rows=10, experts=4, k=64, n=32, trans=0, dtype=BF16, out=BF16, ws=None,
          ws_bytes=0, stream=None)
QR = dict(x=0x10000, ldx=200, q=0x20000, ldq=200, scale=0x30000, lds=10, rows=10, cols=200, dtype=BF16, stream=None)
QW = dict(w=0x10000, ldw=200, sw=2000, q=0x20000, ldq=200, sq=2000, scale=0x30000, n=3, rows=10, cols=200, trans=0,
          dtype=BF16, stream=None)
M8 = dict(x=0x10000, ldx=64, xs=0x20000, ldxs=10, w=0x30000, ldw=64, sw=2048, ws=0x40000, off=0x50000, y=0x60000,
          ldy=32, rows=10, experts=4, k=64, n=32, out=BF16, stream=None)
BIG = (1 << 31) - 1
CASES += [
    (GM, "muon_gated_mm", bad, status) for bad, status in [
        (dict(x=None), INV), (dict(wg=None), INV), (dict(wu=None), INV), (dict(out=None), INV),
        (dict(x=0x10001), ALIGN), (dict(wu=0x30001), ALIGN), (dict(out=0x50001), ALIGN), (dict(p=0x60002), ALIGN),
        (dict(off=None), INV), (dict(off=0x40004), ALIGN), (dict(gate=0x70001, ldg=32), ALIGN),
        (dict(gate=0x70000, ldg=31), INV), (dict(up=0x70000, ldu=31), INV), (dict(up=0x70001, ldu=32), ALIGN),
        (dict(ldx=63), INV), (dict(ldwg=31), INV), (dict(ldwu=31), INV), (dict(trans=1), INV), (dict(ldo=31), INV),
        (dict(sg=0), INV), (dict(su=-1), INV), (dict(rows=-1), INV), (dict(rows=1 << 31), INV),
        (dict(experts=0), INV), (dict(experts=1025), INV), (dict(k=0), INV), (dict(n=0), INV), (dict(dtype=F32), INV),
        (dict(dtype=3), INV), (dict(x=0x10002), INV), (dict(ldwu=33, ws=0x80000, ws_bytes=16), INV),
        (dict(ldx=65, ws=0x80010, ws_bytes=1 << 20), ALIGN),
        (dict(rows=BIG, n=BIG, ldwg=1 << 31, ldwu=1 << 31, ldo=1 << 31), capi.MUON_ERR_UNSUPPORTED),
    ]] + [
    (GG, "muon_gated_mm_grad", bad, status) for bad, status in [
        (dict(dy=None), INV), (dict(w=None), INV), (dict(gate=None), INV), (dict(up=None), INV),
        (dict(dgate=None), INV), (dict(dup=None), INV), (dict(dy=0x10001), ALIGN), (dict(gate=0x40001), ALIGN),
        (dict(dgate=0x60001), ALIGN), (dict(out=0x80001, ldo=32), ALIGN), (dict(out=0x80000, ldo=31), INV),
        (dict(p=0x90002), ALIGN), (dict(dp=0x90002), ALIGN), (dict(dp=0x90000), INV), (dict(off=None), INV),
        (dict(dp=0x90000, ws=0xa0000, ws_bytes=39), INV), (dict(lddy=63), INV), (dict(ldw=63), INV),
        (dict(trans=0, ldw=31), INV), (dict(ldg=31), INV), (dict(ldu=31), INV), (dict(lddg=31), INV),
        (dict(lddu=31), INV), (dict(sw=0), INV), (dict(rows=1 << 31), INV), (dict(experts=0), INV), (dict(k=0), INV),
        (dict(n=-1), INV), (dict(dtype=F32), INV), (dict(ldw=65), INV),
    ]] + [
    (MS, "muon_grouped_mm_sum", bad, status) for bad, status in [
        (dict(x1=None), INV), (dict(x2=None), INV), (dict(w1=None), INV), (dict(w2=0x40001), ALIGN),
        (dict(y=None), INV), (dict(off=None), INV), (dict(ldx1=63), INV), (dict(ldx2=63), INV), (dict(ldw1=31), INV),
        (dict(ldw2=31), INV), (dict(s2=0), INV), (dict(ldy=31), INV), (dict(out=F16), INV), (dict(out=F32, y=0x60002), ALIGN),
        (dict(dtype=F32, out=F32), INV), (dict(rows=-1), INV), (dict(experts=2000), INV), (dict(k=0), INV),
        (dict(ldx2=65), INV), (dict(x2=0x30002, ws=0x70000, ws_bytes=64), INV),
    ]] + [
    (QR, "muon_quantize_rows", bad, status) for bad, status in [
        (dict(x=None), INV), (dict(q=None), INV), (dict(scale=None), INV), (dict(x=0x10001), ALIGN),
        (dict(scale=0x30002), ALIGN), (dict(ldx=199), INV), (dict(ldq=199), INV), (dict(lds=9), INV),
        (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(cols=0), INV), (dict(dtype=3), INV),
        (dict(dtype=F32, x=0x10002), ALIGN),
    ]] + [
    (QW, "muon_quantize_weights", bad, status) for bad, status in [
        (dict(w=None), INV), (dict(q=None), INV), (dict(scale=None), INV), (dict(w=0x10001), ALIGN),
        (dict(scale=0x30001), ALIGN), (dict(ldw=199), INV), (dict(ldq=199), INV), (dict(sw=0), INV),
        (dict(sq=1999), INV), (dict(trans=1, ldq=9), INV), (dict(trans=1, ldq=16, sq=199 * 16 + 9), INV), (dict(sq=-5), INV),
        (dict(n=0), INV), (dict(n=1025), INV), (dict(rows=0), INV), (dict(cols=-1), INV), (dict(dtype=-1), INV),
    ]] + [
    (M8, "muon_grouped_mm_fp8", bad, status) for bad, status in [
        (dict(x=None), INV), (dict(w=None), INV), (dict(xs=None), INV), (dict(ws=None), INV), (dict(y=None), INV),
        (dict(x=0x10008), ALIGN), (dict(w=0x30008), ALIGN), (dict(xs=0x20002), ALIGN), (dict(ws=0x40002), ALIGN),
        (dict(y=0x60001), ALIGN), (dict(ldx=72), ALIGN), (dict(ldw=72), ALIGN), (dict(sw=2056), ALIGN),
        (dict(ldx=48), INV), (dict(ldw=48), INV), (dict(sw=0), INV), (dict(ldxs=9), INV), (dict(ldy=31), INV),
        (dict(off=None), INV), (dict(off=0x50004), ALIGN), (dict(rows=-1), INV), (dict(rows=1 << 31), INV),
        (dict(experts=0), INV), (dict(k=0), INV), (dict(n=0), INV), (dict(out=3), INV), (dict(out=-1), INV),
        (dict(rows=BIG, n=BIG, ldy=1 << 31, ldxs=1 << 31), capi.MUON_ERR_UNSUPPORTED),
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


def test_gated_workspaces():
    """Nothing for operands whose rows start on 16 bytes; else copies of those that do not, and the sums of
    the row weights' gradient."""
    v = ctypes.c_size_t()

    def size(call, *args):
        assert getattr(capi.lib, call)(*args, ctypes.byref(v)) == capi.MUON_OK, capi.muon_last_error()
        return v.value

    def gated(ldx=64, ldg=32, ldu=32, rows=10, trans=0):
        return size("muon_gated_mm_workspace_bytes", 0x1000, ldx, 0x2000, ldg, 4096, 0x3000, ldu, 4096, rows, 4, 64, 32,
                    trans)

    assert gated() == 0 and gated(rows=0, ldx=65) == 0
    assert 10 * 64 * 2 <= gated(ldx=65) <= 10 * 64 * 2 + 1024
    assert 4 * 64 * 32 * 2 <= gated(ldu=33) <= 4 * 64 * 32 * 2 + 1024
    assert gated(ldg=33, ldu=33, ldx=65) == gated(ldg=33) + gated(ldu=33) + gated(ldx=65)

    def grad(lddy=64, dp=0, n=32):
        return size("muon_gated_mm_grad_workspace_bytes", 0x1000, lddy, 0x2000, 64, 1 << 20, 10, 4, 64, n, 1, dp)

    assert grad() == 0 and grad(dp=1) == 10 * 4 and grad(dp=1, n=33) == 2 * 10 * 4
    assert grad(lddy=65, dp=1) == grad(lddy=65) + 10 * 4 and grad(lddy=65) % 1024 == 0

    def both(ldx1=64, ldx2=64, ldw2=32):
        return size("muon_grouped_mm_sum_workspace_bytes", 0x1000, ldx1, 0x2000, 32, 4096, 0x3000, ldx2, 0x4000, ldw2,
                    4096, 10, 4, 64, 32, 0)

    assert both() == 0 and both(ldx1=65) == both(ldx2=65) > 0 and both(ldx2=65, ldw2=33) == both(ldx2=65) + both(ldw2=33)
    assert capi.lib.muon_gated_mm_workspace_bytes(0x1000, 64, 0x2000, 32, 4096, 0x3000, 32, 4096, 10, 4, 64, 32, 0,
                                                  None) == INV
    assert capi.lib.muon_gated_mm_grad_workspace_bytes(0x1000, 64, 0x2000, 64, 4096, 10, 4, 64, 32, 1, 0, None) == INV
