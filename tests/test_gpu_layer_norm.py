"""Layer norm and its gradient on the GPU against plain 64-bit forms.

Bounds (derived, element by element; u = 2^-24, D additions on the longest way of a value through a
sum: 64 in a thread or cols / 1024 of a long row, 5 in a warp, 32 over the warps, so D <= 160 +
cols / 1024):

* the mean is off by d <= (D + 2) u mean|x|; the deviations by d and a rounding; the variance by
  (D + 4) u of itself and d^2 (the deviations sum to zero); rstd by half of that and 4 ulp (8 u) of
  rsqrtf and the sum with eps; so y is off by |w| rstd (d + 2 u |x - mean|) + |w (x - mean) rstd| (D + 16) u +
  d^2 rstd^2 |w (x - mean) rstd| + 3 u (|w (x - mean) rstd| + |b|), and half a step of the store;
* dx, from given mean and rstd: (D + 16) u rstd (|t| + mean|t| + |xh| mean|t xh|) and the store;
* dw, db: a sum of `rows` terms of three roundings each, in any order: (rows + 8) u times the sum of
  their magnitudes (and the old value's, accumulating).
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


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


def _within(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bound = bound + half * (want.abs() + bound) + TINY[got.dtype]
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() - bound).max().item() if got.numel() else -1.0
    assert worst <= 0.0, f"{what}: over the bound by {worst:.3g}"


def _depth(cols):
    return 160 + cols / 1024


def _placed(t, pitch, start):
    """t's values in a larger buffer of NaN: rows `pitch` apart, `start` elements in."""
    buf = torch.full((start + max(1, t.shape[0]) * pitch + 8,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf.as_strided(t.shape, (pitch, 1), start)
    v.copy_(t)
    return buf, v


def _forward(x, w, b, eps):
    xd = x.double()
    var, mean = torch.var_mean(xd, 1, correction=0) if x.shape[0] else (xd.sum(1), xd.sum(1))
    rstd = (var + eps).rsqrt()
    wd = torch.ones(x.shape[1], device="cuda", dtype=torch.float64) if w is None else w.double()
    bd = torch.zeros_like(wd) if b is None else b.double()
    return xd, mean, rstd, wd, bd


def _check_forward(capi, x, w, b, eps=1e-5, place=None, keep=True):
    rows, cols = x.shape
    mean = torch.full((rows,), 9.0, device="cuda") if keep else None
    rstd = torch.full((rows,), 9.0, device="cuda") if keep else None
    xin, ybuf = x, torch.full((rows + 1, cols), 7.0, dtype=x.dtype, device="cuda")
    y = ybuf[:rows]
    if place:
        _, xin = _placed(x, cols + place[0], place[1])
        ybuf, y = _placed(torch.full_like(x, 7.0), cols + place[2], place[3])
    capi.muon_layer_norm(xin, w, b, y, mean=mean, rstd=rstd, eps=eps)
    capi.muon_check()
    if not place:
        assert (ybuf[rows] == 7.0).all(), "wrote behind the last row"
    else:
        flat = ybuf.clone()
        flat.as_strided(y.shape, y.stride(), place[3]).fill_(float("nan"))
        assert torch.isnan(flat).all(), "wrote outside y"
    xd, m, r, wd, bd = _forward(x, w, b, eps)
    d = (_depth(cols) + 2) * U * xd.abs().mean(1) if rows else m
    dev = (xd - m[:, None]).abs()
    main = wd.abs() * dev * r[:, None]
    bound = wd.abs() * r[:, None] * (d[:, None] + 2 * U * dev) + main * ((_depth(cols) + 16) * U
                                                                         + (d * r)[:, None] ** 2) \
        + 3 * U * (main + bd.abs())
    _within(y, (xd - m[:, None]) * r[:, None] * wd + bd, bound, "y")
    if keep:
        _within(mean, m, d, "mean")
        _within(rstd, r, r * ((_depth(cols) + 16) * U + (d * r) ** 2), "rstd")


def _inputs(gen, rows, cols, dtype, shift=0.5):
    x = torch.randn(rows, cols, generator=gen, device="cuda") * 1.5 + shift
    return (x.to(DT[dtype]), 1 + 0.3 * torch.randn(cols, generator=gen, device="cuda"),
            torch.randn(cols, generator=gen, device="cuda"))


COLS = [1, 2, 7, 8, 64, 72, 256, 264, 771, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8193, 8200, 16384,
        16385, 16392, 20001]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", COLS)
def test_forward(capi, cols, dtype):
    gen = _gen(cols)
    for rows in (1, 5, 37):
        _check_forward(capi, *_inputs(gen, rows, cols, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("place", [(8, 0, 16, 8), (3, 1, 0, 0), (0, 0, 1, 5), (8, 1, 8, 1)])
def test_forward_strides(capi, place, dtype):
    for cols in (40, 768, 4096):
        _check_forward(capi, *_inputs(_gen(cols), 19, cols, dtype), place=place, keep=False)


def test_forward_many_rows(capi):
    for rows, cols, dtype in ((20_011, 64, "bf16"), (3001, 771, "fp16"), (2500, 4096, "bf16"), (700, 16392, "fp32")):
        _check_forward(capi, *_inputs(_gen(rows), rows, cols, dtype))


def test_forward_weights_at_any_offset(capi):
    """Weights inside a flat buffer start wherever the parameters before them end."""
    x, w, b = _inputs(_gen(3), 9, 1024, "bf16")
    flat = torch.cat([w.new_zeros(3), w, b])
    _check_forward(capi, x, flat[3:1027], flat[1027:])
    _check_forward(capi, x, None, b)
    _check_forward(capi, x, w, None)
    _check_forward(capi, x, None, None, keep=False)


def test_forward_large_means_and_constant_rows(capi):
    """Rows whose mean is 1000 times their spread keep their variance; constant ones give the bias."""
    _check_forward(capi, *_inputs(_gen(4), 11, 1536, "fp32", shift=1000.0))
    x = torch.full((3, 512), 3.0, device="cuda")
    w, b = torch.ones(512, device="cuda"), torch.arange(512.0, device="cuda")
    y = torch.empty_like(x)
    capi.muon_layer_norm(x, w, b, y)
    assert torch.equal(y, b.expand(3, 512))
    _check_forward(capi, *_inputs(_gen(5), 4, 320, "fp32"), eps=0.0)


def test_forward_bad_rows_stay_alone(capi):
    for cols in (64, 771, 4096, 16385):
        x, w, b = _inputs(_gen(6), 9, cols, "bf16")
        y, want = torch.empty_like(x), torch.empty_like(x)
        capi.muon_layer_norm(x, w, b, want)
        bad = x.clone()
        bad[3, 0], bad[5, cols - 1] = float("nan"), float("inf")
        capi.muon_layer_norm(bad, w, b, y)
        keep = [0, 1, 2, 4, 6, 7, 8]
        assert torch.equal(y[keep], want[keep]) and torch.isnan(y[[3, 5]]).all()


def _check_grad(capi, rows, cols, dtype, accumulate=False, place=None, want_dw=True, want_db=True,
                weight=True, seed=1):
    gen = _gen(seed + rows * 31 + cols)
    x, w, _ = _inputs(gen, rows, cols, dtype)
    if not weight:
        w = None
    dy = torch.randn(rows, cols, generator=gen, device="cuda").to(DT[dtype])
    xd, m, r, wd, _ = _forward(x, w, None, 1e-5)
    mean, rstd = m.float(), r.float()
    old = torch.randn(2, cols, generator=gen, device="cuda")
    dw, db = old.clone()
    xin, din, dx = x, dy, torch.full((rows + 1, cols), 7.0, dtype=x.dtype, device="cuda")
    if place:
        _, xin = _placed(x, cols + place[0], place[1])
        _, din = _placed(dy, cols + place[1], place[0])
        dxbuf, dxv = _placed(torch.full_like(x, 7.0), cols + place[2], place[3])
    else:
        dxv = dx[:rows]
    capi.muon_layer_norm_grad(din, xin, w, mean, rstd, dxv, dw if want_dw else None, db if want_db else None,
                              accumulate=accumulate)
    capi.muon_check()
    if place:
        dxbuf = dxbuf.clone()
        dxbuf.as_strided(dxv.shape, dxv.stride(), place[3]).fill_(float("nan"))
        assert torch.isnan(dxbuf).all()
    else:
        assert (dx[rows] == 7.0).all()
    dd, md, rd = dy.double(), mean.double()[:, None], rstd.double()[:, None]
    xh, t = (xd - md) * rd, dd * wd
    if rows:
        m1, m2 = t.mean(1)[:, None], (t * xh).mean(1)[:, None]
        mag = rd * (t.abs() + t.abs().mean(1)[:, None] + xh.abs() * (t * xh).abs().mean(1)[:, None])
        _within(dxv, rd * (t - m1 - xh * m2), (_depth(cols) + 16) * U * mag, "dx")
    base = old.double() if accumulate else torch.zeros_like(old.double())
    for got, terms, k, on in ((dw, dd * xh, 0, want_dw), (db, dd, 1, want_db)):
        if on:
            _within(got, base[k] + terms.sum(0), (rows + 8) * U * (terms.abs().sum(0) + base[k].abs()),
                    ("dw", "db")[k])
        else:
            assert torch.equal(got, old[k])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", COLS)
def test_grad(capi, cols, dtype):
    for rows in (1, 5, 40):
        _check_grad(capi, rows, cols, dtype, accumulate=rows == 5)


@pytest.mark.parametrize("rows,cols,dtype", [(20_011, 64, "bf16"), (5003, 40, "fp32"), (3001, 771, "fp32"),
                                             (2500, 4096, "bf16"), (700, 16392, "fp16"), (1500, 200, "fp16")])
def test_grad_many_rows(capi, rows, cols, dtype):
    _check_grad(capi, rows, cols, dtype)
    _check_grad(capi, rows, cols, dtype, accumulate=True)


@pytest.mark.parametrize("cols", [1024, 1032, 1536, 2040, 2048, 2056, 4096, 4104, 8192, 8200])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_where_slabs_change(capi, cols, dtype):
    """The lengths of a row on both sides of each change in the rows and threads of a block."""
    for rows in (305, 1003):
        _check_forward(capi, *_inputs(_gen(cols), rows, cols, dtype))
        _check_grad(capi, rows, cols, dtype, accumulate=rows == 305)


@pytest.mark.parametrize("place", [(8, 0, 16, 8), (3, 1, 0, 0), (0, 0, 1, 5), (8, 8, 8, 1)])
def test_grad_strides(capi, place):
    for cols in (40, 768, 4096):
        _check_grad(capi, 19, cols, "bf16", place=place)


def test_grad_of_parts(capi):
    """Without the weight gradients, with one of them, without weights."""
    for cols in (48, 1024, 4096, 16400):
        _check_grad(capi, 33, cols, "bf16", want_dw=False, want_db=False)
        _check_grad(capi, 33, cols, "bf16", want_db=False, accumulate=True)
        _check_grad(capi, 33, cols, "bf16", want_dw=False)
        _check_grad(capi, 33, cols, "fp32", weight=False)


def test_no_rows(capi):
    for cols in (64, 20001):
        x = torch.empty(0, cols, device="cuda")
        none = torch.empty(0, device="cuda")
        capi.muon_layer_norm(x, None, None, x.clone(), mean=none, rstd=none)
        dw, db = torch.ones(2, cols, device="cuda")
        capi.muon_layer_norm_grad(x, x, None, none, none, x, dw, db, accumulate=True)
        assert (dw == 1).all() and (db == 1).all()
        capi.muon_layer_norm_grad(x, x, None, none, none, x, dw, db)
        assert (dw == 0).all() and (db == 0).all()


def test_grad_against_differences(capi):
    """Central differences of the 64-bit forward pass in random directions: h = 1e-4 leaves h^2 / 6 of
    a third derivative (of the order of the first: below 1e-6 of the sum of magnitudes)."""
    gen = _gen(8)
    x, w, b = _inputs(gen, 6, 200, "fp32")
    c = torch.randn(6, 200, generator=gen, device="cuda", dtype=torch.float64)
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(200, device="cuda"), torch.empty(200, device="cuda")
    capi.muon_layer_norm(x, w, b, y, mean=mean, rstd=rstd)
    capi.muon_layer_norm_grad(c.float(), x, w, mean, rstd, dx, dw, db)

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return (c.float().double() * (d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b)).sum()

    base = [x.double(), w.double(), b.double()]
    for k, grad in enumerate((dx, dw, db)):
        for _ in range(4):
            v = torch.randn(base[k].shape, generator=gen, device="cuda", dtype=torch.float64)
            hi, lo = list(base), list(base)
            hi[k], lo[k] = base[k] + 1e-4 * v, base[k] - 1e-4 * v
            want = (loss(*hi) - loss(*lo)) / 2e-4
            assert abs((grad.double() * v).sum() - want) <= 3e-6 * (grad.double() * v).abs().sum()


def test_equal_inputs_give_equal_bits(capi):
    x, w, b = _inputs(_gen(9), 4001, 777, "bf16")
    dy = torch.randn(4001, 777, generator=_gen(10), device="cuda").bfloat16()
    mean, rstd = torch.empty(2, 4001, device="cuda")
    runs = []
    for _ in range(2):
        y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        capi.muon_layer_norm(x, w, b, y, mean=mean, rstd=rstd)
        capi.muon_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db)
        runs.append((y, dx, dw, db))
    assert all(torch.equal(p, q) for p, q in zip(*runs))


def test_rows_beyond_32_bit_offsets(capi):
    """Three rows 2^30 + 8 elements apart: the last starts behind 2^31."""
    pitch, cols = (1 << 30) + 8, 520
    x, w, b = _inputs(_gen(11), 3, cols, "bf16")
    buf = torch.empty(2 * pitch + cols, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((3, cols), (pitch, 1))
    far.copy_(x)
    mean, rstd = torch.empty(2, 3, device="cuda")
    y, want = torch.empty_like(x), torch.empty_like(x)
    capi.muon_layer_norm(far, w, b, y, mean=mean, rstd=rstd)
    capi.muon_layer_norm(x, w, b, want)
    assert torch.equal(y, want)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    dx2, dw2, db2 = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    capi.muon_layer_norm_grad(far, far, w, mean, rstd, dx, dw, db)
    capi.muon_layer_norm_grad(x, x, w, mean, rstd, dx2, dw2, db2)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    capi.muon_layer_norm(x, w, b, far)           # far results as well
    assert torch.equal(far, want)


def test_captured_and_on_another_stream(capi):
    x, w, b = _inputs(_gen(12), 300, 771, "fp32")
    dy = torch.randn_like(x)
    mean, rstd = torch.empty(2, 300, device="cuda")
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(608 * 2 * 771, device="cuda")

    def step(stream=None):
        capi.muon_layer_norm(x, w, b, y, mean=mean, rstd=rstd, stream=stream)
        capi.muon_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db, workspace=ws, stream=stream)

    step()
    want = [t.clone() for t in (y, dx, dw, db)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (y, dx, dw, db):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, (y, dx, dw, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.mul_(2)                       # the replay sees the values of its time
    graph.replay()
    got = [t.clone() for t in (y, dx, dw, db)]
    step()
    assert all(torch.equal(p, q) for p, q in zip(got, (y, dx, dw, db))) and not torch.equal(got[1], want[1])
