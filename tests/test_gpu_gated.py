"""The gated block's products, forward and backward, on the GPU against plain 64-bit forms.

Bounds (derived, element by element; u = 2^-23):

* a product of K terms summed in fp32 is off by at most K u sum |a b| =: d (every partial sum is at
  most that sum of magnitudes, and an addition that truncates loses at most u of it);
* sigmoid and silu take fewer than 16 fp32 operations of at most an ulp each, and the fast exponential
  is off by 2 + 1.2 |g| ulp: (16 + 2 |g|) u =: r, relative;
* silu's slope lies in -0.1 .. 1.1 and it is at most 1.1 |g|, so p silu(g) u is off by
  |p| (1.1 dg (|u| + du) + |silu(g)| du) + r |p silu(g) u|;
* the gradient's 1 + g (1 - s) cancels near g = -1.28: its error is r relative to
  s (1 + |g| (1 - s)); dp adds n such terms;
* each store rounds once, by half a step of its type.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -23
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


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


def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _placed(t, pitch, start):
    """The same values in a larger buffer: row pitch `pitch`, `start` elements in, the rest NaN."""
    flat = t.reshape(-1, t.shape[-1])
    buf = torch.full((start + flat.shape[0] * pitch + 8,), float("nan"), dtype=t.dtype, device=t.device)
    shape, strides = t.shape, (pitch, 1) if t.dim() == 2 else (t.shape[-2] * pitch, pitch, 1)
    view = buf.as_strided(shape, strides, start)
    view.copy_(t)
    return view


def _within(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bound = bound + half * (want.abs() + bound) + TINY[got.dtype]
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = ((got.double() - want).abs() - bound).max().item() if got.numel() else -1.0
    assert worst <= 0.0, f"{what}: over the bound by {worst:.3g}"


class Results:
    """Result matrices inside buffers of 7, where nothing else may be written."""

    def __init__(self, rows, n, dtype, extra):
        self.rows, self.n, self.dtype, self.extra, self.bufs = rows, n, dtype, extra, []

    def new(self):
        buf = torch.full((self.rows + 1, self.n + self.extra), 7.0, dtype=self.dtype, device="cuda")
        self.bufs.append(buf)
        return buf[:self.rows, :self.n]

    def check(self):
        for b in self.bufs:
            assert (b[self.rows] == 7.0).all() and (b[:, self.n:] == 7.0).all(), "wrote outside a result"


class Rows:
    """Rows of experts of the given sizes, `first` rows of none before them and `tail` behind."""

    def __init__(self, sizes, first=0, tail=0):
        self.sizes, self.first, self.tail = sizes, first, tail
        self.rows = first + sum(sizes) + tail
        self.dense = sizes == "dense"

    @property
    def offsets(self):
        o = [self.first]
        for s in self.sizes:
            o.append(o[-1] + s)
        return torch.tensor(o, dtype=torch.int64, device="cuda")

    def spoil(self, *matrices):
        for t in matrices:
            t[:self.first] = float("nan")          # rows of no expert must not reach anything
            t[self.rows - self.tail:] = float("inf") if self.tail else 0

    def product(self, x, w, trans):
        """(exact product, its error bound) of the experts' rows."""
        n = w.shape[1] if trans else w.shape[2]
        y = torch.zeros(self.rows, n, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(y)
        r = self.first
        for i, s in enumerate(self.sizes):
            a, b = x[r:r + s].double(), w[i].double()
            b = b.T if trans else b
            y[r:r + s], mag[r:r + s] = a @ b, a.abs() @ b.abs()
            r += s
        return y, x.shape[1] * U * mag

    def none(self, t):
        """t's rows of no expert."""
        return torch.cat([t[:self.first], t[self.rows - self.tail:]])

    def owned(self, t):
        return t[self.first:self.rows - self.tail]


def _weights(gen, e, k, n, trans, dtype):
    return _randn(gen, *((e, n, k) if trans else (e, k, n)), dtype=dtype, std=0.5 * k ** -0.5)


def _rel(g):
    return (16 + 2 * g.abs()) * U


def _check_gated(capi, sizes, k, n, trans=False, dtype="bf16", first=0, tail=0, weighted=True, keep=True,
                 place=None, extra=0, offsets=True, seed=1):
    gen, rows, t = _gen(seed), Rows(sizes, first, tail), DT[dtype]
    x = _randn(gen, rows.rows, k, dtype=t)
    wg, wu = (_weights(gen, len(sizes), k, n, trans, t) for _ in range(2))
    p = torch.rand(rows.rows, generator=gen, device="cuda") * 2 - 0.5 if weighted else None
    rows.spoil(x)
    if place:
        xs, gs, us = (_placed(v, v.shape[-1] + a, b) for v, (a, b) in zip((x, wg, wu), place))
    else:
        xs, gs, us = x, wg, wu
    res = Results(rows.rows, n, t, extra)
    out, gate, up = res.new(), res.new() if keep else None, res.new() if keep else None
    capi.muon_gated_mm(xs, gs, us, rows.offsets if offsets else None, out, gate=gate, up=up, row_weight=p,
                       trans_w=trans)
    capi.muon_check()
    res.check()
    for v in (out, gate, up):
        assert v is None or (rows.none(v) == 0).all(), "rows of no expert"
    (g, dg), (u, du) = rows.product(x, wg, trans), rows.product(x, wu, trans)
    w = p.double()[:, None] if weighted else torch.ones(rows.rows, 1, device="cuda", dtype=torch.float64)
    silu = g * torch.sigmoid(g)
    want = w * silu * u
    bound = w.abs() * (1.1 * dg * (u.abs() + du) + silu.abs() * du) + _rel(g) * want.abs()
    _within(rows.owned(out), rows.owned(want), rows.owned(bound), "out")
    if keep:
        _within(rows.owned(gate), rows.owned(g), rows.owned(dg), "gate")
        _within(rows.owned(up), rows.owned(u), rows.owned(du), "up")


# Sizes that run on each kind of tile: a cluster per tile, narrow, single CTAs, pairs.
SIZES = [
    ([1], 64, 128), ([0, 1, 0, 2, 0], 256, 136), ([3, 16, 17, 1], 8, 8), ([15, 16, 17, 33, 1, 63, 64, 65], 72, 264),
    ([200], 4096, 192), ([7] * 64, 200, 1408), ([255, 256, 257, 0, 513], 200, 1040), ([700, 90], 1408, 640),
    ([1500, 0, 2100, 700], 256, 1096), ([4100], 128, 2048), ([0, 0, 0], 64, 64),
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,k,n", SIZES)
def test_gated(capi, sizes, k, n, trans, dtype):
    _check_gated(capi, sizes, k, n, trans, dtype)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("k,n", [(1, 1), (5, 3), (771, 517), (63, 129), (65, 640), (640, 65)])
def test_gated_odd_sizes(capi, k, n, trans):
    _check_gated(capi, [9, 0, 70, 33], k, n, trans, "fp16", weighted=False)
    _check_gated(capi, [900, 0, 1100, 1], k, n, trans, "bf16", keep=False)


@pytest.mark.parametrize("trans", [False, True])
def test_gated_rows_of_no_expert_and_strides(capi, trans):
    for sizes in ([5, 0, 40], [600, 700, 900]):
        _check_gated(capi, sizes, 136, 328, trans, first=3, tail=5, extra=5)
        _check_gated(capi, sizes, 136, 328, trans, place=((8, 8), (16, 0), (0, 8)), extra=8)
        _check_gated(capi, sizes, 136, 328, trans, place=((3, 1), (0, 0), (5, 3)), first=2)
        _check_gated(capi, sizes, 136, 328, trans, place=((0, 0), (1, 2), (0, 0)))


def test_gated_dense(capi):
    for rows, k, n in ((1, 512, 264), (300, 200, 1000), (3000, 264, 1600)):
        for trans in (False, True):
            _check_gated(capi, [rows], k, n, trans, offsets=False)


def _check_grad(capi, sizes, k, n, trans=True, dtype="bf16", first=0, tail=0, weighted=True, dp=True,
                out=True, place=None, extra=0, offsets=True, seed=2):
    gen, rows, t = _gen(seed), Rows(sizes, first, tail), DT[dtype]
    dy = _randn(gen, rows.rows, k, dtype=t)
    w = _weights(gen, len(sizes), k, n, trans, t)
    gate, up = _randn(gen, rows.rows, n, dtype=t, std=2.0), _randn(gen, rows.rows, n, dtype=t)
    p = torch.rand(rows.rows, generator=gen, device="cuda") * 2 - 0.5 if weighted else None
    rows.spoil(dy, gate, up)
    ins = [_placed(v, v.shape[-1] + a, b) for v, (a, b) in zip((dy, w, gate, up), place)] if place else \
        [dy, w, gate, up]
    res = Results(rows.rows, n, t, extra)
    dgate, dup, act = res.new(), res.new(), res.new() if out else None
    grad_p = torch.full((rows.rows + 1,), 7.0, device="cuda") if dp else None
    capi.muon_gated_mm_grad(ins[0], ins[1], rows.offsets if offsets else None, ins[2], ins[3], dgate, dup,
                            out=act, row_weight=p, d_row_weight=grad_p[:-1] if dp else None, trans_w=trans)
    capi.muon_check()
    res.check()
    assert not dp or grad_p[-1] == 7.0
    for v in (dgate, dup, act, grad_p[:-1] if dp else None):
        assert v is None or (rows.none(v) == 0).all(), "rows of no expert"
    dh, d = (rows.owned(v) for v in rows.product(dy, w, trans))
    g, u = rows.owned(gate).double(), rows.owned(up).double()
    one = torch.ones(len(g), 1, device="cuda", dtype=torch.float64)
    q = rows.owned(p).double()[:, None] if weighted else one
    s = torch.sigmoid(g)
    silu, slope, r = g * s, s * (1 + g * (1 - s)), _rel(g)
    _within(rows.owned(dup), dh * q * silu, (q * silu).abs() * d + r * (dh * q * silu).abs(), "dup")
    _within(rows.owned(dgate), dh * q * u * slope,
            (q * u * slope).abs() * d + (dh.abs() + d) * (q * u).abs() * s * (1 + g.abs() * (1 - s)) * r, "dgate")
    if out:
        _within(rows.owned(act), q * silu * u, r * (q * silu * u).abs(), "out")
    if dp:
        terms = (dh * silu * u).abs()
        _within(rows.owned(grad_p[:-1]), (dh * silu * u).sum(1),
                ((silu * u).abs() * d + terms * r).sum(1) + n * U * terms.sum(1), "dp")


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,k,n", SIZES)
def test_grad(capi, sizes, k, n, trans, dtype):
    _check_grad(capi, sizes, k, n, trans, dtype)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("k,n", [(1, 1), (5, 3), (771, 517), (63, 129), (65, 640), (640, 65)])
def test_grad_odd_sizes(capi, k, n, trans):
    _check_grad(capi, [9, 0, 70, 33], k, n, trans, "fp16", weighted=False)
    _check_grad(capi, [900, 0, 1100, 1], k, n, trans, "bf16", dp=False)
    _check_grad(capi, [9, 1100], k, n, trans, "bf16", out=False)


@pytest.mark.parametrize("trans", [False, True])
def test_grad_rows_of_no_expert_and_strides(capi, trans):
    for sizes in ([5, 0, 40], [600, 700, 900]):
        _check_grad(capi, sizes, 136, 328, trans, first=3, tail=5, extra=5)
        _check_grad(capi, sizes, 136, 328, trans, place=((8, 8), (16, 0), (0, 8), (8, 0)), extra=8)
        _check_grad(capi, sizes, 136, 328, trans, place=((3, 1), (0, 0), (5, 3), (1, 1)), first=2)
        _check_grad(capi, sizes, 136, 328, trans, place=((0, 0), (1, 2), (0, 0), (0, 7)))


def test_grad_dense(capi):
    for rows, k, n in ((1, 512, 264), (300, 200, 1000), (3000, 264, 1600)):
        _check_grad(capi, [rows], k, n, offsets=False, weighted=False, dp=rows == 300)


def _check_sum(capi, sizes, k, n, trans=True, dtype="bf16", out="bf16", first=0, tail=0, place=None,
               extra=0, offsets=True, seed=3):
    gen, rows, t = _gen(seed), Rows(sizes, first, tail), DT[dtype]
    x1, x2 = (_randn(gen, rows.rows, k, dtype=t) for _ in range(2))
    w1, w2 = (_weights(gen, len(sizes), k, n, trans, t) for _ in range(2))
    rows.spoil(x1, x2)
    ins = [_placed(v, v.shape[-1] + a, b) for v, (a, b) in zip((x1, w1, x2, w2), place)] if place else \
        [x1, w1, x2, w2]
    res = Results(rows.rows, n, DT[out], extra)
    y = res.new()
    capi.muon_grouped_mm_sum(*ins, rows.offsets if offsets else None, y, trans_w=trans)
    capi.muon_check()
    res.check()
    assert (rows.none(y) == 0).all(), "rows of no expert"
    (a, da), (b, db) = rows.product(x1, w1, trans), rows.product(x2, w2, trans)
    _within(rows.owned(y), rows.owned(a + b), 2 * rows.owned(da + db), "y")


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("sizes,k,n", SIZES)
def test_sum(capi, sizes, k, n, trans, dtype, out):
    _check_sum(capi, sizes, k, n, trans, dtype, out)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("k,n", [(1, 1), (5, 3), (771, 517), (63, 129), (65, 640), (640, 65)])
def test_sum_odd_sizes(capi, k, n, trans):
    _check_sum(capi, [9, 0, 70, 33], k, n, trans, "fp16", "fp32")
    _check_sum(capi, [900, 0, 1100, 1], k, n, trans, "bf16", "bf16", first=1, tail=2)


def test_sum_strides_and_dense(capi):
    for trans in (False, True):
        for place in (((8, 8), (16, 0), (0, 8), (8, 0)), ((3, 1), (0, 0), (5, 3), (1, 1))):
            _check_sum(capi, [5, 0, 40], 136, 328, trans, place=place, extra=3)
            _check_sum(capi, [600, 700, 900], 136, 328, trans, place=place, extra=8)
        _check_sum(capi, [900], 200, 1000, trans, offsets=False)


def test_gates_of_any_size(capi):
    """Gates far from zero: silu(g) is g or 0 there, and no exponential overflows on the way."""
    g = torch.tensor([[-3e38, -1e4, -200.0, -100.0, -90.0, -88.0, -20.0, 20.0, 90.0, 200.0, 1e4, 3e38, 0.0, -0.0,
                       1e-30, -1e-30]], device="cuda").bfloat16()
    n = g.shape[1]
    dy, w = torch.ones(1, 8, device="cuda").bfloat16(), torch.zeros(1, n, 8, device="cuda").bfloat16()
    w[:, :, 0] = 1.0
    up = torch.full_like(g, 0.5)
    dgate, dup, out = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    capi.muon_gated_mm_grad(dy, w, None, g, up, dgate, dup, out=out, trans_w=True)
    gd = g.double()
    s = torch.sigmoid(gd)
    slope = 0.5 * torch.where(gd.abs() > 1e3, (gd > 0).double(), s * (1 + gd * (1 - s)))
    for got, want in ((dup, gd * s), (out, gd * s * 0.5), (dgate, slope)):
        assert torch.isfinite(got).all()
        assert ((got.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-37).all(), (got, want)


def test_bad_offsets(capi):
    x, w = _randn(_gen(4), 40, 64).bfloat16(), _randn(_gen(5), 3, 64, 128).bfloat16()
    for off in ([0, 30, 20, 40], [0, 10, 20, 41], [-1, 10, 20, 40]):
        o = torch.tensor(off, dtype=torch.int64, device="cuda")
        out, gate, up = (torch.ones(40, 128, device="cuda").bfloat16() for _ in range(3))
        dp = torch.ones(40, device="cuda")
        capi.muon_gated_mm(x, w, w, o, out, gate=gate, up=up)
        assert capi.muon_check_status() == capi.MUON_ERR_ROW_OFFSETS
        assert (out == 0).all() and (gate == 0).all() and (up == 0).all()
        dgate, dup = torch.ones_like(out), torch.ones_like(out)
        capi.muon_gated_mm_grad(x, w, o, gate, up, dgate, dup, d_row_weight=dp)
        assert capi.muon_check_status() == capi.MUON_ERR_ROW_OFFSETS
        assert (dgate == 0).all() and (dup == 0).all() and (dp == 0).all()
        capi.muon_grouped_mm_sum(x, w, x, w, o, out.fill_(1))
        assert capi.muon_check_status() == capi.MUON_ERR_ROW_OFFSETS and (out == 0).all()


def test_bad_rows_stay_alone(capi):
    """A NaN or an infinity in one row reaches no other."""
    gen = _gen(6)
    for sizes in ([20, 13, 7], [700, 900, 800]):
        rows = Rows(sizes)
        x = _randn(gen, rows.rows, 136).bfloat16()
        w = _weights(gen, 3, 136, 264, False, torch.bfloat16)
        out, want = (torch.empty(rows.rows, 264, device="cuda").bfloat16() for _ in range(2))
        capi.muon_gated_mm(x, w, w, rows.offsets, want)
        bad = x.clone()
        bad[5, 3], bad[sizes[0], 0] = float("nan"), float("inf")
        capi.muon_gated_mm(bad, w, w, rows.offsets, out)
        keep = torch.ones(rows.rows, dtype=torch.bool)
        keep[5] = keep[sizes[0]] = False
        assert torch.equal(out[keep], want[keep]) and torch.isnan(out[5]).all()


def test_block_against_autograd_and_differences(capi):
    """Forward and backward of a whole block of experts, as a layer runs them, against automatic
    differentiation in 64 bits, and its loss against central differences.  Values pass at most four
    16-bit stores (2^-9 each in the root mean square): 4 * 2^-9 < 1e-2."""
    gen, sizes, k, n = _gen(7), [120, 0, 37, 300], 192, 328
    rows = Rows(sizes)
    off = rows.offsets
    x = _randn(gen, rows.rows, k).bfloat16()
    wg, wu, wd = (_randn(gen, 4, a, b, std=a ** -0.5).bfloat16() for a, b in ((k, n), (k, n), (n, k)))
    p = torch.rand(rows.rows, generator=gen, device="cuda")
    c = _randn(gen, rows.rows, k).bfloat16()

    def new(cols):
        return torch.empty(rows.rows, cols, device="cuda", dtype=torch.bfloat16)

    act, gate, up, y, dgate, dup, act2, dx = new(n), new(n), new(n), new(k), new(n), new(n), new(n), new(k)
    dp = torch.empty_like(p)
    dwg, dwu = torch.empty(2, 4, k, n, device="cuda")
    dwd = torch.empty(4, n, k, device="cuda")
    capi.muon_gated_mm(x, wg, wu, off, act, gate=gate, up=up, row_weight=p)
    capi.muon_grouped_mm(act, wd, off, y)
    capi.muon_gated_mm_grad(c, wd, off, gate, up, dgate, dup, out=act2, row_weight=p, d_row_weight=dp,
                            trans_w=True)
    capi.muon_grouped_mm_sum(dgate, wg, dup, wu, off, dx, trans_w=True)
    capi.muon_grouped_wgrad(act2, c, off, dwd)
    capi.muon_grouped_wgrad(x, dgate, off, dwg)
    capi.muon_grouped_wgrad(x, dup, off, dwu)
    capi.muon_check()

    def loss(x, wg, wu, wd, p):
        parts, r = [], 0
        for i, s in enumerate(sizes):
            a = x[r:r + s]
            h = torch.nn.functional.silu(a @ wg[i]) * (a @ wu[i]) * p[r:r + s, None]
            parts.append(h @ wd[i])
            r += s
        return (torch.cat(parts) * c.double()).sum()

    leaves = [t.double().requires_grad_(True) for t in (x, wg, wu, wd, p)]
    want = torch.autograd.grad(loss(*leaves), leaves)
    for got, ref, name in zip((dx, dwg, dwu, dwd, dp), want, ("dx", "dwg", "dwu", "dwd", "dp")):
        assert (got.double() - ref).norm() <= 1e-2 * ref.norm(), name
    with torch.no_grad():
        for i, got in enumerate((dx, dwg, dwu, dwd, dp)):
            v = got.double() / got.double().norm()
            hi, lo = [t.detach().clone() for t in leaves], [t.detach().clone() for t in leaves]
            hi[i] += 1e-5 * v
            lo[i] -= 1e-5 * v
            slope = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(slope - (got.double() * v).sum()) <= 1e-2 * got.double().norm(), i


def test_captured_streams_and_equal_bits(capi):
    """Odd sizes (operands are copied, dp has partial sums): the same bits captured and replayed with
    new inputs, on another stream, and twice."""
    gen, rows, k, n = _gen(8), Rows([100, 3, 60]), 77, 130
    off = rows.offsets
    x = _randn(gen, rows.rows, k).bfloat16()
    w1, w2 = _randn(gen, 2, 3, k, n).bfloat16()
    p = torch.rand(rows.rows, generator=gen, device="cuda")
    wd = _randn(gen, 3, n, k).bfloat16()
    new = lambda c: torch.zeros(rows.rows, c, device="cuda").bfloat16()  # noqa: E731
    outs = [new(n), new(n), new(n), new(n), new(n), new(n), new(k), torch.zeros_like(p)]
    out, gate, up, dgate, dup, act, dx, dp = outs

    def step(stream=None, **ws):
        capi.muon_gated_mm(x, w1, w2, off, out, gate=gate, up=up, row_weight=p, stream=stream)
        capi.muon_gated_mm_grad(x, wd, off, gate, up, dgate, dup, out=act, row_weight=p, d_row_weight=dp,
                                trans_w=True, stream=stream)
        capi.muon_grouped_mm_sum(dgate, w1, dup, w2, off, dx, trans_w=True, stream=stream)

    step()
    want = [t.clone() for t in outs]
    step()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        for t in outs:
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        step(handle)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.mul_(0.5)
    off.copy_(torch.tensor([2, 2, 60, 160]))
    graph.replay()
    got = [t.clone() for t in outs]
    step()
    capi.muon_check()
    assert all(torch.equal(a, b) for a, b in zip(got, outs)) and not torch.equal(got[0], want[0])
