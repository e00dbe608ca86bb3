"""Operands and results that are columns of wider buffers, at widths that do not fill 16 bytes: what
lies between the rows is neither read into a result nor written."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


def _padded(t, pitch):
    """t's values in rows of `pitch` elements, NaN between them."""
    buf = torch.full((*t.shape[:-1], pitch), float("nan"), dtype=t.dtype, device=t.device)
    buf[..., :t.shape[-1]] = t
    return buf[..., :t.shape[-1]]


def _integers(gen, *shape):
    return torch.randint(-8, 9, shape, generator=gen, device="cuda").bfloat16()


def _setup(sizes):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sum(sizes))
    return gen, torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], device="cuda")


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,k,n", [
    ([9, 0, 70, 33], 77, 130), ([9, 0, 70, 33], 63, 133), ([3, 1], 1, 1), ([2], 1027, 77),
    ([700, 300, 0, 900], 203, 2309), ([64, 1, 40], 781, 1411), ([9], 5, 3), ([1], 2051, 131),
])
def test_products(capi, sizes, k, n, trans):
    gen, off = _setup(sizes)
    x = _integers(gen, sum(sizes), k)
    w = _integers(gen, *((len(sizes), n, k) if trans else (len(sizes), k, n)))
    want = torch.cat([a.double() @ (b.double().T if trans else b.double())
                      for a, b in zip(x.split(sizes), w)])
    up = lambda v: (v + 7) // 8 * 8 + 8
    buf = torch.full((sum(sizes), up(n)), 7.0, device="cuda")
    capi.muon_grouped_mm(_padded(x, up(k)), _padded(w, up(w.shape[2])), off, buf[:, :n], trans_w=trans)
    capi.muon_check()
    assert torch.equal(buf[:, :n].double(), want)
    assert (buf[:, n:] == 7.0).all()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,m,n", [
    ([9, 0, 70, 33], 77, 130), ([9, 0, 70, 33], 63, 133), ([3, 1], 1, 1), ([5000], 33, 217),
    ([700, 300, 0, 900], 203, 2309), ([600, 513, 700], 781, 1411), ([2300, 0, 4097], 72, 131),
])
def test_weight_gradients(capi, sizes, m, n, accumulate):
    gen, off = _setup(sizes)
    a, b = _integers(gen, sum(sizes), m), _integers(gen, sum(sizes), n)
    want = torch.stack([x.double().T @ y.double() for x, y in zip(a.split(sizes), b.split(sizes))])
    up = lambda v: (v + 7) // 8 * 8 + 8
    buf = torch.full((len(sizes), m, up(n)), 5.0, device="cuda")
    capi.muon_grouped_wgrad(_padded(a, up(m)), _padded(b, up(n)), off, buf[:, :, :n],
                            accumulate=accumulate)
    capi.muon_check()
    assert torch.equal(buf[:, :, :n].double(), want + 5.0 * accumulate)
    assert (buf[:, :, n:] == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(3, 7), (5000, 129), (37, 1411), (2, 1)])
def test_activation(capi, rows, cols, dtype):
    gen, _ = _setup([rows, cols])
    pitch = (cols + 7) // 8 * 8 + 8
    g, u, da = (torch.randn(rows, cols, generator=gen, device="cuda").to(dtype) for _ in range(3))
    a, dg, du = (torch.empty_like(g) for _ in range(3))
    dp, dp2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    capi.muon_swiglu(g, u, a)
    capi.muon_swiglu_grad(da, g, u, dg, du, d_row_weight=dp)
    bufs = [torch.full((rows, pitch), 7.0, dtype=dtype, device="cuda") for _ in range(3)]
    outs = [b[:, :cols] for b in bufs]
    g, u, da = (_padded(t, pitch) for t in (g, u, da))
    capi.muon_swiglu(g, u, outs[0])
    capi.muon_swiglu_grad(da, g, u, outs[1], outs[2], d_row_weight=dp2)
    capi.muon_check()
    assert all(torch.equal(x, y) for x, y in zip(outs, (a, dg, du)))
    assert all((b[:, cols:] == 7.0).all() for b in bufs) and torch.equal(dp, dp2)
