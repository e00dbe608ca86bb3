"""Quantization to e4m3 with block scales, and the products of such operands, on the GPU against plain
forms.

Quantization has one right answer: scales and values are compared bit by bit with a plain form in 64
bits.  A product's bound (element by element, u = 2^-23): a block's 128 terms are summed in fp32 with at
most u of the sum of magnitudes lost per term, so 128 u of it; scaling, and adding B blocks with
rounding to nearest, lose at most (B + 3) u / 2 of the sum of all magnitudes more; the store rounds once.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -23
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _blocks(n):
    return -(-n // 128)


def _power(e):
    """2^e in 64 bits, made of its bits: the GPU's pow may be off by an ulp."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _quantized(t, high):
    """(values, scales) of (n, rows, cols) with blocks of high x 128, in 64 bits."""
    n, rows, cols = t.shape
    rb, cb = -(-rows // high), _blocks(cols)
    d = t.double()
    finite = torch.isfinite(d)
    room = torch.zeros(n, rb * high, cb * 128, dtype=torch.float64, device=t.device)
    room[:, :rows, :cols] = torch.where(finite, d, 0.0)
    amax = room.view(n, rb, high, cb, 128).abs().amax((2, 4))
    e = torch.full_like(amax, -126.0)
    for k in range(-125, 121):                # powers are exact in 64 bits
        e = torch.where(amax > 448.0 * 2.0 ** (k - 1), torch.full_like(e, float(k)), e)
    scale = torch.where(amax > 0, _power(e), torch.ones_like(amax))
    spread = scale.repeat_interleave(high, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :cols]
    v = d / spread
    size = v.abs().clamp(min=2.0 ** -6)
    exp = torch.frexp(size).exponent.double() - 1
    step = _power(exp - 3)
    q = torch.round(v / step) * step          # ties to even
    return torch.where(finite, q, float("nan")), scale


def _same(got, want):
    g, w = got.double(), want.double()
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(w))


def _values(gen, shape, dtype):
    t = torch.randn(shape, generator=gen, device="cuda")
    t *= torch.exp2(torch.randint(-12, 12, (*shape[:-1], 1), generator=gen, device="cuda").float())
    return t.to(DT[dtype])


def _check_rows(capi, x, pad=0, start=0, qpad=0, qstart=0, spad=0):
    rows, cols = x.shape
    src = x
    if pad or start:
        buf = torch.full((start + max(1, rows) * (cols + pad) + 8,), float("nan"), dtype=x.dtype, device="cuda")
        src = buf.as_strided((rows, cols), (cols + pad, 1), start)
        src.copy_(x)
    raw = torch.full((qstart + (rows + 1) * (cols + qpad),), 0x55, dtype=torch.uint8, device="cuda")
    q = raw.as_strided((rows, cols), (cols + qpad, 1), qstart)
    sraw = torch.full((_blocks(cols) + 1, rows + spad), 7.0, device="cuda")
    scale = sraw[:-1, :rows]
    capi.muon_quantize_rows(src, q.view(E4M3), scale)
    capi.muon_check()
    want, ws = _quantized(x[None], 1)
    _same(q.contiguous().view(E4M3), want[0])
    assert torch.equal(scale.double(), ws[0].T)
    q.fill_(0x55)
    assert (raw == 0x55).all() and (sraw[-1] == 7.0).all() and (sraw[:, rows:] == 7.0).all(), "wrote outside"


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [1, 7, 8, 127, 128, 129, 136, 512, 771, 2048, 4100])
def test_rows(capi, cols, dtype):
    for rows in (1, 3, 50):
        _check_rows(capi, _values(_gen(cols + rows), (rows, cols), dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_strides_and_many(capi, dtype):
    for cols in (136, 771):
        x = _values(_gen(1), (33, cols), dtype)
        _check_rows(capi, x, pad=8, qpad=8, spad=3)
        _check_rows(capi, x, pad=3, start=1, qpad=5, qstart=3)
        _check_rows(capi, x, qpad=0, qstart=8)
    _check_rows(capi, _values(_gen(2), (70_001, 40), dtype))
    _check_rows(capi, _values(_gen(3), (9000, 2048), dtype))


def _special():
    x = torch.zeros(8, 300, device="cuda")
    x[1, 5], x[1, 6], x[1, 200] = float("inf"), 3.0, float("nan")
    x[2] = 448.0
    x[3, :128], x[3, 128:] = 449.0, 896.5
    x[4, 0], x[4, 1] = 1e-42, -1e-45
    x[5, 0], x[5, 150] = 3.4e38, -3e-39
    x[6, :17] = torch.arange(17, device="cuda") / 16 + 16          # ties of the rounding
    x[6, 100] = 448.0
    x[7] = -0.0
    return x


def test_rows_of_special_values(capi):
    """Zeros, the largest value and the next, subnormals, infinities, NaN, ties."""
    x = _special()
    _check_rows(capi, x)
    _check_rows(capi, x[:, :296].contiguous())
    _check_rows(capi, x[:6].bfloat16())


def _check_weights(capi, w, transpose, pad=0, start=0, qpad=0, qstart=0):
    n, rows, cols = w.shape
    src = w
    if pad or start:
        buf = torch.full((start + n * rows * (cols + pad) + 8,), float("nan"), dtype=w.dtype, device="cuda")
        src = buf.as_strided(w.shape, (rows * (cols + pad), cols + pad, 1), start)
        src.copy_(w)
    t = w.transpose(1, 2).contiguous() if transpose else w
    pitch = t.shape[2] + qpad
    raw = torch.full((qstart + n * t.shape[1] * pitch + 40,), 0x55, dtype=torch.uint8, device="cuda")
    q = raw.as_strided(t.shape, (t.shape[1] * pitch, pitch, 1), qstart)
    scale = torch.full((n + 1, _blocks(t.shape[1]), _blocks(t.shape[2])), 7.0, device="cuda")
    capi.muon_quantize_weights(src, q.view(E4M3), scale[:n], transpose=transpose)
    capi.muon_check()
    want, ws = _quantized(t, 128)
    _same(q.contiguous().view(E4M3), want)
    assert torch.equal(scale[:n].double(), ws)
    q.fill_(0x55)
    assert (raw == 0x55).all() and (scale[n] == 7.0).all(), "wrote outside"


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (3, 7, 130), (2, 128, 128), (2, 129, 264), (4, 300, 517),
                                         (5, 640, 72), (1, 1000, 2048), (1, 130, 8)])
def test_weights(capi, n, rows, cols, dtype, transpose):
    _check_weights(capi, _values(_gen(rows), (n, rows, cols), dtype), transpose)


@pytest.mark.parametrize("transpose", [False, True])
def test_weights_strides_and_special_values(capi, transpose):
    w = _values(_gen(4), (3, 136, 264), "bf16")
    _check_weights(capi, w, transpose, pad=8, qpad=8)
    _check_weights(capi, w, transpose, pad=3, start=1, qpad=3, qstart=1)
    _check_weights(capi, w, transpose, qpad=16, qstart=8)
    _check_weights(capi, _special()[None].repeat(2, 40, 1)[:, :300], transpose)
    _check_weights(capi, _values(_gen(5), (700, 130, 140), "bf16"), transpose)     # more blocks than CTAs


class Operands:
    def __init__(self, gen, sizes, k, n, first=0, tail=0, plain_scales=False, pitch=0):
        self.sizes, self.k, self.n, self.first = sizes, k, n, first
        self.rows = first + sum(sizes) + tail
        line = k + -k % 16 + pitch
        e = len(sizes)

        def values(*shape):
            room = torch.full((*shape[:-1], line), 0x7f, dtype=torch.uint8, device="cuda")   # NaN behind k
            v = (torch.randn(shape, generator=gen, device="cuda") * 60).clamp(-448, 448).to(E4M3)
            room[..., :k] = v.view(torch.uint8)
            return room.view(E4M3)[..., :k]

        def scales(*shape):
            if plain_scales:
                return torch.rand(shape, generator=gen, device="cuda") + 0.01
            return torch.exp2(torch.randint(-9, 0, shape, generator=gen, device="cuda").float())

        self.x, self.w = values(self.rows, k), values(e, n, k)
        self.xs, self.ws = scales(_blocks(k), self.rows), scales(e, _blocks(n), _blocks(k))
        o = [first]
        for s in sizes:
            o.append(o[-1] + s)
        self.offsets = torch.tensor(o, dtype=torch.int64, device="cuda")

    def exact(self):
        y = torch.zeros(self.rows, self.n, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(y)
        r = self.first
        for i, s in enumerate(self.sizes):
            a = self.x[r:r + s].double() * self.xs[:, r:r + s].double().T.repeat_interleave(128, 1)[:, :self.k]
            b = self.w[i].double() * self.ws[i].double().repeat_interleave(128, 0)[:self.n].repeat_interleave(
                128, 1)[:, :self.k]
            y[r:r + s], mag[r:r + s] = a @ b.T, a.abs() @ b.abs().T
            r += s
        return y, mag


def _check_mm(capi, sizes, k, n, out="bf16", first=0, tail=0, plain_scales=False, pitch=0, offsets=True,
              extra=0, seed=1):
    o = Operands(_gen(seed + k), sizes, k, n, first, tail, plain_scales, pitch)
    if first:
        o.x.view(torch.uint8)[:first] = 0x7f
        o.xs[:, :first] = float("nan")
    if tail:
        o.x.view(torch.uint8)[o.rows - tail:] = 0x7f
        o.xs[:, o.rows - tail:] = float("inf")
    buf = torch.full((o.rows + 1, n + extra), 7.0, dtype=DT[out], device="cuda")
    y = buf[:o.rows, :n]
    capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, o.offsets if offsets else None, y)
    capi.muon_check()
    assert (buf[o.rows] == 7.0).all() and (buf[:, n:] == 7.0).all(), "wrote outside y"
    assert (y[:first] == 0).all() and (y[o.rows - tail:] == 0).all(), "rows of no expert"
    keep = slice(first, o.rows - tail)
    want, mag = (t[keep] for t in o.exact())
    bound = (128 + (_blocks(k) + 3) / 2) * U * mag
    half = torch.finfo(DT[out]).eps / 2
    bound = bound + half * (want.abs() + bound) + TINY[DT[out]]
    got = y[keep]
    assert torch.isfinite(got).all()
    worst = ((got.double() - want).abs() - bound).max().item() if got.numel() else -1.0
    assert worst <= 0.0, f"over the bound by {worst:.3g}"


SIZES = [
    ([1], 64, 128), ([0, 1, 0, 2, 0], 256, 136), ([3, 16, 17, 1], 16, 8), ([15, 16, 17, 33, 1, 63, 64, 65], 144, 264),
    ([200], 8192, 192), ([7] * 64, 208, 1408), ([255, 256, 257, 0, 513], 400, 1040), ([700, 90], 1408, 640),
    ([1500, 0, 2100, 700], 512, 1096), ([4100], 128, 2048), ([0, 0, 0], 64, 64),
]


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("sizes,k,n", SIZES)
def test_mm(capi, sizes, k, n, out):
    _check_mm(capi, sizes, k, n, "bf16" if out == "fp16" and k > 1000 else out)


@pytest.mark.parametrize("k,n", [(1, 1), (5, 3), (771, 517), (63, 129), (129, 640), (640, 65)])
def test_mm_odd_sizes(capi, k, n):
    _check_mm(capi, [9, 0, 70, 33], k, n, "fp32", first=2, tail=3, extra=3)
    _check_mm(capi, [900, 0, 1100, 1], k, n, "bf16", first=1, plain_scales=True, pitch=32)


def test_mm_dense_and_any_scales(capi):
    for rows, k, n in ((1, 512, 264), (300, 208, 1000), (3000, 272, 1600)):
        _check_mm(capi, [rows], k, n, "fp32", offsets=False, plain_scales=True)


def test_mm_many_k_blocks(capi):
    """More k-blocks than slots of scales and stages, on every kind of tile."""
    for sizes, n in (([5], 128), ([40, 3, 60], 2048), ([300, 500], 2048), ([2500, 2300], 2048)):
        _check_mm(capi, sizes, 128 * 37 + 16, n, "fp32", plain_scales=True)


def test_mm_of_no_rows_and_bad_offsets(capi):
    o = Operands(_gen(9), [10, 0, 30], 64, 128)
    y = torch.ones(40, 128, device="cuda")
    for off in ([0, 30, 20, 40], [0, 10, 20, 41], [-1, 10, 20, 40]):
        capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, torch.tensor(off, device="cuda"), y.fill_(1))
        assert capi.muon_check_status() == capi.MUON_ERR_ROW_OFFSETS and (y == 0).all()
    capi.muon_grouped_mm_fp8(o.x[:0], o.xs[:, :0], o.w, o.ws, torch.zeros(4, dtype=torch.int64, device="cuda"), y[:0])
    capi.muon_check()


def test_bad_values_stay_in_their_rows(capi):
    for sizes in ([20, 13, 7], [900, 700, 800]):
        o = Operands(_gen(10), sizes, 400, 264)
        y, want = (torch.empty(o.rows, 264, device="cuda") for _ in range(2))
        capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, o.offsets, want)
        o.x.view(torch.uint8)[5, 399] = 0x7f
        o.xs[2, sizes[0]] = float("nan")
        capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, o.offsets, y)
        keep = torch.ones(o.rows, dtype=torch.bool)
        keep[5] = keep[sizes[0]] = False
        assert torch.equal(y[keep], want[keep]) and torch.isnan(y[~keep]).all()


def test_quantized_product_of_a_layer(capi):
    """Weights turned and quantized once, activations on the way: against the product in 64 bits of
    what the 8-bit values stand for, and the whole within their rounding (2^-4 per value at most)."""
    gen, sizes, k, n = _gen(11), [130, 0, 61, 400], 328, 264
    rows = sum(sizes)
    x = torch.randn(rows, k, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(4, k, n, generator=gen, device="cuda") * 0.05).bfloat16()
    off = torch.tensor([0, 130, 130, 191, 591], device="cuda")
    xq, wq = (torch.empty(*s, 336, dtype=torch.uint8, device="cuda").view(E4M3)[..., :k] for s in ((rows,), (4, n)))
    xs, ws = torch.empty(3, rows, device="cuda"), torch.empty(4, 3, 3, device="cuda")
    y = torch.empty(rows, n, device="cuda").bfloat16()
    capi.muon_quantize_weights(w, wq, ws, transpose=True)
    capi.muon_quantize_rows(x, xq, xs)
    capi.muon_grouped_mm_fp8(xq, xs, wq, ws, off, y)
    capi.muon_check()
    full = torch.cat([a.double() @ b.double() for a, b in zip(x.split(sizes), w)])
    mag = torch.cat([a.double().abs() @ b.double().abs() for a, b in zip(x.split(sizes), w)])
    assert ((y.double() - full).abs() <= (2 * 2.0 ** -4 + 2.0 ** -7) * mag + 1e-3).all()


def test_captured_streams_and_equal_bits(capi):
    gen, sizes, k, n = _gen(12), [700, 0, 900], 771, 520
    rows = sum(sizes)
    x = torch.randn(rows, k, generator=gen, device="cuda")
    o = Operands(gen, sizes, k, n)
    y = torch.empty(rows, n, device="cuda")

    def step(stream=None):
        capi.muon_quantize_rows(x, o.x, o.xs, stream=stream)
        capi.muon_grouped_mm_fp8(o.x, o.xs, o.w, o.ws, o.offsets, y, stream=stream)

    step()
    want = y.clone()
    step()
    assert torch.equal(y, want)
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        y.zero_()
        side.wait_stream(torch.cuda.current_stream())
        step(handle)
        side.synchronize()
        assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.mul_(1.7)
    o.offsets.copy_(torch.tensor([5, 600, 1000, 1600]))
    graph.replay()
    got = y.clone()
    step()
    capi.muon_check()
    assert torch.equal(got, y) and not torch.equal(got, want)
