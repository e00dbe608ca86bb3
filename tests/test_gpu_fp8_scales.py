"""8-bit products with scales at the ends of fp32, on every kind of tile, against the 64-bit form.

The bound is that of test_gpu_fp8.py: 128 u of a block's sum of magnitudes for its 128 terms, and for B
blocks (B + 3) u / 2 for the scaling (the product of two scales and its product with the block's sum, rounded
once each) and the additions, wherever the values themselves lie in fp32's normal range.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_fp8 import DT, E4M3, TINY, U, Operands, _blocks, _gen  # noqa: E402

# Tiles that a cluster shares, narrow ones, tiles of y itself (k of whole blocks and a part).
SHAPES = [([5], 1100, 128), ([0, 9, 40, 3], 400, 264), ([7] * 64, 400, 1408), ([900, 0, 1100, 700], 400, 1096)]


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


def _check(capi, o, out="fp32"):
    want, mag = o.exact()
    y = torch.full((o.rows, o.n), 7.0, dtype=DT[out], device="cuda")
    capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, o.offsets, y)
    capi.muon_check()
    bound = (128 + (_blocks(o.k) + 3) / 2) * U * mag
    bound = bound + torch.finfo(y.dtype).eps / 2 * (want.abs() + bound) + TINY[y.dtype]
    assert torch.isfinite(y).all()
    worst = ((y.double() - want).abs() - bound).max().item()
    assert worst <= 0.0, f"over the bound by {worst:.3g}"


def _small(gen, t):
    """e4m3 values of magnitude 2^-9 .. 2^-6, many of them zero."""
    code = torch.randint(0, 9, t.shape, generator=gen, device="cuda").to(torch.uint8)
    sign = torch.randint(0, 2, t.shape, generator=gen, device="cuda").to(torch.uint8) << 7
    room = t.view(torch.uint8)
    room.copy_(torch.where(torch.rand(t.shape, generator=gen, device="cuda") < 0.3, code | sign, torch.zeros_like(code)))


def _scaled(gen, o, ex, ew):
    """Scales of about 2^ex and 2^ew with fractions of their own."""
    o.xs, o.ws = (((1 + torch.rand(s.shape, generator=gen, device="cuda")).double() * 2.0 ** (e - 1)).float()
                  for s, e in ((o.xs, ex), (o.ws, ew)))


@pytest.mark.parametrize("ex,ew", [(120, 8), (8, 120), (64, 64), (100, 28), (127, 5), (127, -40), (60, 45), (50, 50)])
@pytest.mark.parametrize("sizes,k,n", SHAPES)
def test_scales_whose_product_is_large(capi, sizes, k, n, ex, ew):
    """Small values under large scales: |sum| below 2^-12 * 1100, the product of the scales up to 2^132."""
    gen = _gen(ex)
    o = Operands(gen, sizes, k, n)
    _small(gen, o.x)
    _small(gen, o.w)
    _scaled(gen, o, ex, ew)
    want, mag = o.exact()
    assert mag.max() < 2.0 ** 127
    _check(capi, o)
    _check(capi, o, "bf16")


@pytest.mark.parametrize("ex,ew", [(-126, -16), (-100, -42), (-71, -71), (-120, -10), (-145, 20), (-10, -130), (-50, -51)])
@pytest.mark.parametrize("sizes,k,n", SHAPES)
def test_scales_whose_product_is_small(capi, sizes, k, n, ex, ew):
    """Large values under small scales; a scale may be a subnormal number itself."""
    gen = _gen(-ex)
    o = Operands(gen, sizes, k, n)
    _scaled(gen, o, ex, ew)
    want, mag = o.exact()
    assert mag.max() > 2.0 ** -126
    _check(capi, o, "bf16")
    # (In 32 bits: where a value is a subnormal number, each of its additions rounds to 2^-149.)
    y = torch.empty(o.rows, n, device="cuda")
    capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, o.offsets, y)
    bound = (128 + (_blocks(k) + 3) / 2) * U * mag + 2.0 ** -24 * want.abs() * 1.001 + _blocks(k) * 2.0 ** -149
    assert ((y.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("sizes,k,n", SHAPES)
def test_products_of_scales_below_fp32(capi, sizes, k, n):
    """Scales of 2^-149 and 2^-126 by 2^24 sums: results of 0, and no NaN."""
    o = Operands(_gen(3), sizes, k, n)
    o.xs.fill_(2.0 ** -149)
    o.ws.fill_(2.0 ** -126)
    y = torch.full((o.rows, n), 7.0, device="cuda")
    capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, o.offsets, y)
    capi.muon_check()
    assert (y == 0).all()


@pytest.mark.parametrize("sizes,k,n", SHAPES)
def test_zeros_under_any_scales(capi, sizes, k, n):
    """Blocks of zeros add nothing, however large their scales; a scale of 0 is one too."""
    gen = _gen(4)
    o = Operands(gen, sizes, k, n, plain_scales=True)
    o.x.view(torch.uint8)[:, :128] = 0
    o.w.view(torch.uint8)[:, :, 256:384] = 0
    o.xs[0] = 3.0e38
    o.ws[:, :, 0] = 3.0e38
    o.xs[2] = 2.0 ** 127
    o.ws[:, :, 2] = 2.0 ** 90
    _check(capi, o)
    o.xs[1] = 0.0                              # by 3e38, and by what is far below 1
    o.ws[:, :, 1] = 3.0e38
    _check(capi, o)
    o.ws[:, :, 1] = 2.0 ** -149
    o.ws[:, :, 3] = 0.0
    _check(capi, o)


@pytest.mark.parametrize("sizes,k,n", SHAPES)
def test_rows_and_blocks_of_every_size_together(capi, sizes, k, n):
    """Rows whose scales are 2^100, 1 and 2^-100 by blocks that take them back, the others' sums zeros."""
    gen = _gen(5)
    o = Operands(gen, sizes, k, n, plain_scales=True)
    third = torch.arange(o.rows, device="cuda") % 3
    # Row r has values in block r % 3 of k only.
    for b in range(_blocks(k)):
        o.x.view(torch.uint8)[third != b, 128 * b:128 * (b + 1)] = 0
    power = torch.tensor([2.0 ** 100, 1.0, 2.0 ** -100], device="cuda")
    o.xs *= power[third]
    o.ws[:, :, :3] /= power
    _check(capi, o)


def test_a_product_of_the_largest_quantized_values(capi):
    """What the two quantizations make of rows near the largest bf16 value and weights above 57344: the
    product of the scales is 2^128.  The weights of these rows' columns are small or zero."""
    gen = _gen(6)
    rows, k, n = 3000, 256, 1024
    x = torch.zeros(rows, k, device="cuda")
    x[:, 0] = 3.0e38
    x[:, 128:] = torch.randn(rows, 128, generator=gen, device="cuda")
    x = x.bfloat16()
    w = torch.randn(1, n, k, generator=gen, device="cuda")
    w[:, :, 0] = 0.0
    w[:, ::128, 1] = 60000.0
    w = w.bfloat16()
    xq, xs = torch.empty(rows, k, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(2, rows, device="cuda")
    wq, ws = torch.empty(1, n, k, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(1, 8, 2, device="cuda")
    capi.muon_quantize_rows(x, xq, xs)
    capi.muon_quantize_weights(w, wq, ws)
    assert (xs[0] == 2.0 ** 120).all() and (ws[0, :, 0] == 2.0 ** 8).all()
    o = Operands(gen, [rows], k, n)
    o.x, o.xs, o.w, o.ws = xq, xs, wq, ws
    for part in (rows, 300, 5):
        o.rows, o.sizes, o.x, o.xs = part, [part], xq[:part], xs[:, :part].contiguous()
        o.offsets = torch.tensor([0, part], device="cuda")
        _check(capi, o)
