"""Products grouped by expert, the gated activation and its gradient, on the GPU against plain
64-bit forms.

Bounds (derived, element by element):

* a product of K terms summed in fp32 is off by at most K * 2^-23 * sum |a b| (every partial
  sum is at most that sum of magnitudes, and an addition that truncates loses at most 2^-23
  of it), and the store rounds once: 2^-8 of the value in bfloat16, 2^-11 (and half of the
  smallest subnormal, 2^-25) in float16;
* the activation takes fewer than ten fp32 operations of at most 2 ulp each (expf included):
  2^-19 of the value, before the same store rounding.  Its gradient's factor 1 + g (1 - s)
  cancels near g = -1.28, so there the bound is relative to |da p u| s (1 + |g| (1 - s)).
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STORE = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25),
         torch.float32: (2.0 ** -24, 2.0 ** -149)}


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


def _offsets(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int64, device="cuda")


def _strided(t, pitch, start):
    """The same values in a larger buffer: row pitch `pitch`, `start` elements in, the rest NaN."""
    flat = t.reshape(-1, t.shape[-1])
    buf = torch.full((start + flat.shape[0] * pitch + 8,), float("nan"), dtype=t.dtype, device=t.device)
    view = buf[start:start + flat.shape[0] * pitch].view(flat.shape[0], pitch)[:, :t.shape[-1]]
    view.copy_(flat)
    if t.dim() == 3:
        view = buf.as_strided(t.shape, (t.shape[1] * pitch, pitch, 1), start)
    return view


def _close(got, want, mag, terms, what):
    """|got - want| <= terms * 2^-23 * mag + the store's rounding, everywhere."""
    rel, tiny = STORE[got.dtype]
    bound = terms * 2.0 ** -23 * mag
    bound = bound + rel * (want.abs() + bound) + tiny
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (err - bound).max().item() if err.numel() else -1.0
    assert worst <= 0.0, f"{what}: over the bound by {worst:.3g}"


def _check_mm(capi, sizes, k, n, trans, dtype, out, first=0, tail=0, pitch=None, start=0, seed=1,
              wstart=0):
    gen = _gen(seed)
    rows, e = first + sum(sizes) + tail, len(sizes)
    x = _randn(gen, rows, k, dtype=DT[dtype])
    w = _randn(gen, *((e, n, k) if trans else (e, k, n)), dtype=DT[dtype], std=0.1)
    if first:
        x[:first] = float("nan")        # rows of no expert must not reach anything
    if tail:
        x[rows - tail:] = float("inf")
    off = _offsets(sizes, first)
    xs = x if pitch is None else _strided(x, pitch[0], start)
    ws = w if pitch is None else _strided(w, pitch[1], wstart)
    ldy = n + 5 if pitch is not None else n
    ybuf = torch.full((rows + 1, ldy), 7.0, dtype=DT[out], device="cuda")
    y = ybuf[:rows, :n]
    capi.muon_grouped_mm(xs, ws, off, y, trans_w=trans)
    capi.muon_check()
    assert (ybuf[rows] == 7.0).all() and (ybuf[:, n:] == 7.0).all(), "wrote outside y"
    assert (y[:first] == 0).all() and (y[rows - tail:] == 0).all(), "rows of no expert"
    r = first
    for i, s in enumerate(sizes):
        xd, wd = x[r:r + s].double(), w[i].double()
        wd = wd.T if trans else wd
        _close(y[r:r + s], xd @ wd, xd.abs() @ wd.abs(), k, f"expert {i} of {sizes}")
        r += s


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32")])
@pytest.mark.parametrize("sizes,k,n", [
    ([1], 64, 128),                         # a single row
    ([0, 1, 0, 2, 0], 256, 136),            # a few tokens, experts without rows
    ([3, 16, 17, 1], 8, 8),                 # one k-block, partly filled; narrow outputs
    ([15, 16, 17, 127, 128, 129], 72, 264),  # around the tile edges
    ([255, 256, 257, 0, 513], 200, 130 * 8),
    ([700], 1408, 256),
])
def test_mm(capi, sizes, k, n, trans, dtype, out):
    _check_mm(capi, sizes, k, n, trans, dtype, out)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("k,n", [(1, 1), (5, 3), (771, 517), (63, 129), (65, 640), (640, 65)])
def test_mm_odd_sizes(capi, k, n, trans):
    _check_mm(capi, [9, 0, 70, 33], k, n, trans, "fp16", "fp16")
    _check_mm(capi, [9, 0, 70, 33], k, n, trans, "bf16", "fp32")


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("start,wstart,extra", [(0, 0, 8), (8, 16, 24), (3, 8, 8), (8, 5, 8), (8, 8, 3)])
def test_mm_strides_and_starts(capi, start, wstart, extra, trans):
    k, n = 200, 136
    _check_mm(capi, [5, 131, 0, 40], k, n, trans, "bf16", "bf16", first=3, tail=11,
              pitch=(k + extra, (k if trans else n) + extra), start=start, wstart=wstart)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp32")])
@pytest.mark.parametrize("sizes,k,n", [
    ([300, 0, 33, 31, 512, 129], 200, 2312),
    ([1, 2, 95, 96, 97, 256, 257, 600], 1608, 1416),   # several segments of an fp32 sum
    ([5000], 72, 1160),
])
def test_mm_enough_tiles_for_pairs(capi, sizes, k, n, trans, dtype, out):
    _check_mm(capi, sizes, k, n, trans, dtype, out, first=2, tail=5)


@pytest.mark.parametrize("k", [1, 7, 65, 771])
def test_mm_single_row_of_any_length(capi, k):
    """The pitch of one row means nothing: no copy, and nothing read behind the row."""
    for n in (1, 24):
        _check_mm(capi, [0, 1], k, n, True, "bf16", "fp32")
        _check_mm(capi, [1], k, n, False, "fp16", "fp16")


def test_mm_many_experts(capi):
    sizes = [(i * 7) % 5 for i in range(1024)]
    _check_mm(capi, sizes, 64, 64, False, "bf16", "bf16")
    _check_mm(capi, sizes, 64, 64, True, "bf16", "fp32", first=1, tail=3)


def test_mm_no_rows(capi):
    w = torch.randn(3, 16, 24, device="cuda").bfloat16()
    y = torch.empty(0, 24, device="cuda", dtype=torch.bfloat16)
    capi.muon_grouped_mm(torch.empty(0, 16, device="cuda", dtype=torch.bfloat16), w,
                         _offsets([0, 0, 0]), y)
    y = torch.full((5, 24), 3.0, device="cuda", dtype=torch.bfloat16)   # rows, but none in a group
    x = torch.full((5, 16), float("nan"), device="cuda", dtype=torch.bfloat16)
    capi.muon_grouped_mm(x, w, _offsets([0, 0, 0], first=2), y)
    capi.muon_check()
    assert (y == 0).all()


def test_mm_special_values_stay_in_their_rows(capi):
    """A NaN or infinite row changes its own outputs only, whatever shares its tile."""
    gen = _gen(5)
    sizes = [20, 30, 90, 1]
    x = _randn(gen, sum(sizes), 96, dtype=torch.bfloat16)
    w = _randn(gen, 4, 96, 160, dtype=torch.bfloat16)
    w[2, 5] = float("inf")
    off = _offsets(sizes)
    y0 = torch.empty(sum(sizes), 160, device="cuda", dtype=torch.bfloat16)
    capi.muon_grouped_mm(x, w, off, y0)
    x[25] = float("nan")
    x[50:140, 5] = 0.0   # inf * 0: NaN in all of expert 2's rows
    y = torch.empty_like(y0)
    capi.muon_grouped_mm(x, w, off, y)
    capi.muon_check()
    assert torch.isnan(y[25]).all() and torch.isnan(y[50:140]).all()
    keep = torch.ones(sum(sizes), dtype=torch.bool, device="cuda")
    keep[25] = False
    keep[50:140] = False
    assert torch.equal(y[keep], y0[keep]) and torch.isfinite(y[keep]).all()


def _check_wgrad(capi, sizes, m, n, dtype, accumulate, first=0, tail=0, pitch=None, start=0, gap=0,
                 dstart=0, seed=3):
    gen = _gen(seed)
    rows, e = first + sum(sizes) + tail, len(sizes)
    a = _randn(gen, rows, m, dtype=DT[dtype])
    b = _randn(gen, rows, n, dtype=DT[dtype])
    for t in (a, b):
        t[:first] = float("nan")
        t[rows - tail:] = float("inf")
    off = _offsets(sizes, first)
    as_, bs = (a, b) if pitch is None else (_strided(a, pitch[0], start), _strided(b, pitch[1], start))
    step = m * n + gap
    buf = _randn(gen, dstart + e * step + 3)
    before = buf.clone()
    dw = buf.as_strided((e, m, n), (step, n, 1), dstart)
    old = before.as_strided((e, m, n), (step, n, 1), dstart)
    capi.muon_grouped_wgrad(as_, bs, off, dw, accumulate=accumulate)
    capi.muon_check()
    outside = torch.ones_like(buf, dtype=torch.bool)
    outside.as_strided((e, m, n), (step, n, 1), dstart).zero_()
    assert torch.equal(buf[outside], before[outside]), "wrote outside dw"
    r = first
    for i, s in enumerate(sizes):
        ad, bd = a[r:r + s].double(), b[r:r + s].double()
        want, mag = ad.T @ bd, ad.abs().T @ bd.abs()
        if accumulate:
            want, mag = want + old[i].double(), mag + old[i].double().abs()
        if s == 0:
            assert torch.equal(dw[i], old[i] if accumulate else torch.zeros_like(dw[i]))
        _close(dw[i], want, mag, s + 1, f"expert {i} of {sizes}")
        r += s


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,m,n", [
    ([1], 8, 8),
    ([0, 1, 0, 2], 128, 256),
    ([15, 16, 17, 63, 64, 65], 136, 72),      # around the k-block and MMA edges
    ([127, 0, 129, 200], 264, 520),
    ([5, 700], 256, 1408),
])
def test_wgrad(capi, sizes, m, n, dtype, accumulate):
    _check_wgrad(capi, sizes, m, n, dtype, accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,m,n", [
    ([1, 15, 16, 17, 63, 64, 65], 776, 520),
    ([0, 3, 5, 0, 33, 47, 1, 2000], 264, 1416),
    ([511, 512, 513, 1030, 1], 512, 2000),     # segments of the sum
])
def test_wgrad_enough_tiles_for_pairs(capi, sizes, m, n, accumulate):
    _check_wgrad(capi, sizes, m, n, "bf16", accumulate, first=3, tail=7)
    _check_wgrad(capi, sizes, m, n, "fp16", accumulate, first=3, tail=7, dstart=3)


@pytest.mark.parametrize("m,n", [(1, 1), (3, 5), (130, 520), (129, 257), (517, 63)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_odd_sizes(capi, m, n, accumulate):
    _check_wgrad(capi, [9, 0, 70, 33], m, n, "fp16", accumulate)


@pytest.mark.parametrize("dstart,gap", [(0, 0), (4, 12), (1, 0), (3, 5)])
@pytest.mark.parametrize("start,extra", [(0, 8), (5, 8), (8, 3)])
def test_wgrad_strides_and_starts(capi, dstart, gap, start, extra):
    m, n = 72, 136
    _check_wgrad(capi, [5, 131, 0, 40], m, n, "bf16", True, first=3, tail=11,
                 pitch=(m + extra, n + extra), start=start, gap=gap, dstart=dstart)


def test_wgrad_long_reduction_and_no_rows(capi):
    _check_wgrad(capi, [20000, 3], 72, 136, "bf16", False)
    _check_wgrad(capi, [0, 0, 0], 72, 136, "bf16", False)
    a = torch.empty(0, 8, device="cuda", dtype=torch.bfloat16)
    dw = torch.ones(2, 8, 8, device="cuda")
    capi.muon_grouped_wgrad(a, a, _offsets([0, 0]), dw, accumulate=True)
    assert (dw == 1).all()
    capi.muon_grouped_wgrad(a, a, _offsets([0, 0]), dw)
    capi.muon_check()
    assert (dw == 0).all()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,m,n,dstart", [
    ([5000], 32, 216, 0),              # one tile, its rows split over a cluster
    ([2300, 0, 4097, 1], 72, 136, 0),  # shares of very different lengths, one without rows
    ([3001, 2], 130, 40, 3),           # two row tiles, dw off the 16-byte grid
    ([9, 1500], 256, 65, 0),
])
def test_wgrad_rows_split_over_a_cluster(capi, sizes, m, n, dstart, accumulate):
    _check_wgrad(capi, sizes, m, n, "bf16", accumulate, first=3, tail=5, dstart=dstart)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,k,n", [([1], 2048, 256), ([0, 3, 1, 0], 1600, 264),
                                       ([33], 1090, 130), ([2], 4099, 77)])
def test_mm_k_split_over_a_cluster(capi, sizes, k, n, trans):
    for dtype, out in (("bf16", "bf16"), ("fp16", "fp32")):
        _check_mm(capi, sizes, k, n, trans, dtype, out, first=1, tail=2)


def test_wgrad_special_values_stay_with_their_expert(capi):
    gen = _gen(9)
    sizes = [20, 30, 91, 7]
    a = _randn(gen, sum(sizes), 96, dtype=torch.bfloat16)
    b = _randn(gen, sum(sizes), 160, dtype=torch.bfloat16)
    off = _offsets(sizes)
    d0 = torch.empty(4, 96, 160, device="cuda")
    capi.muon_grouped_wgrad(a, b, off, d0)
    a[20:50] = float("nan")
    b[50:141] = float("inf")
    d1 = torch.empty_like(d0)
    capi.muon_grouped_wgrad(a, b, off, d1)
    capi.muon_check()
    assert torch.equal(d1[0], d0[0]) and torch.equal(d1[3], d0[3])
    assert torch.isnan(d1[1]).all() and not torch.isfinite(d1[2]).any()


def test_products_repeat_bit_for_bit(capi):
    gen = _gen(11)
    sizes = [300, 5, 0, 1000]
    x = _randn(gen, sum(sizes), 512, dtype=torch.bfloat16)
    w = _randn(gen, 4, 512, 264, dtype=torch.bfloat16)
    off = _offsets(sizes)
    ys, ds = [], []
    for _ in range(3):
        y = torch.empty(sum(sizes), 264, device="cuda", dtype=torch.bfloat16)
        capi.muon_grouped_mm(x, w, off, y)
        d = torch.empty(4, 512, 264, device="cuda")
        capi.muon_grouped_wgrad(x, y, off, d)
        ys.append(y)
        ds.append(d)
    capi.muon_check()
    assert all(torch.equal(y, ys[0]) for y in ys) and all(torch.equal(d, ds[0]) for d in ds)


def test_layer_gradients_against_differences(capi):
    """d/dt of sum(dy * mm(x + t v, w + t z)) from the kernels' gradients, against central
    differences of the product in 64 bits (exact for a bilinear form but for rounding)."""
    gen = _gen(13)
    sizes = [40, 0, 7, 129]
    r, k, n = sum(sizes), 72, 136
    x = _randn(gen, r, k, dtype=torch.float16)
    w = _randn(gen, 4, k, n, dtype=torch.float16)
    dy = _randn(gen, r, n, dtype=torch.float16)
    off = _offsets(sizes)
    dx = torch.empty(r, k, device="cuda")
    dw = torch.empty(4, k, n, device="cuda")
    capi.muon_grouped_mm(dy, w, off, dx, trans_w=True)
    capi.muon_grouped_wgrad(x, dy, off, dw)
    capi.muon_check()
    v, z = torch.randn_like(dx).double(), torch.randn_like(dw).double()

    def loss(t):
        xs, total, row = x.double() + t * v, 0.0, 0
        for i, s in enumerate(sizes):
            total = total + (dy[row:row + s].double() * (xs[row:row + s] @ (w[i].double() + t * z[i]))).sum()
            row += s
        return total

    h = 2.0 ** -10
    want = (loss(h) - loss(-h)) / (2 * h)
    got = (dx.double() * v).sum() + (dw.double() * z).sum()
    mag = (dx.double() * v).abs().sum() + (dw.double() * z).abs().sum()
    assert abs(got - want) <= 1e-5 * mag


@pytest.mark.parametrize("k", [16, 1024])   # 1024: split over a cluster
def test_bad_offsets_are_reported_and_move_nothing(capi, k):
    x = torch.randn(10, k, device="cuda").bfloat16()
    w = torch.randn(3, k, 24, device="cuda").bfloat16()
    for bad in ([0, 4, 3, 10], [0, 4, 8, 11], [-1, 4, 8, 10], [0, 2 ** 40, 8, 10]):
        off = torch.tensor(bad, dtype=torch.int64, device="cuda")
        y = torch.full((10, 24), 3.0, device="cuda").bfloat16()
        capi.muon_grouped_mm(x, w, off, y)
        assert capi.muon_check_status() == capi.MUON_ERR_ROW_OFFSETS
        assert (y == 0).all()
        dw = torch.ones(3, k, 24, device="cuda")
        capi.muon_grouped_wgrad(x, y, off, dw)
        assert capi.muon_check_status() == capi.MUON_ERR_ROW_OFFSETS
        assert (dw == 0).all()
        capi.muon_check()


def test_products_on_another_stream_and_in_a_graph(capi):
    gen = _gen(17)
    sizes = [100, 3, 60]
    x = _randn(gen, sum(sizes), 77, dtype=torch.bfloat16)     # rows off the 16-byte grid
    w = _randn(gen, 3, 77, 130, dtype=torch.bfloat16)
    off = _offsets(sizes)
    want = torch.empty(sum(sizes), 130, device="cuda")
    capi.muon_grouped_mm(x, w, off, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)
    capi.muon_grouped_mm(x, w, off, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.muon_grouped_mm(x, w, off, y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    # the graph reads the offsets of the moment
    off.copy_(_offsets([3, 100, 60]))
    graph.replay()
    capi.muon_grouped_mm(x, w, off, want)
    capi.muon_check()
    assert torch.equal(y, want)


def test_products_on_several_streams_at_once(capi):
    """Launches that share the GPU's SMs: pairs, narrow tiles, clusters and weight gradients."""
    gen = _gen(31)
    jobs = []
    for sizes, k, n in (([700, 300, 0, 900], 512, 2312), ([3, 0, 9, 1], 1024, 264),
                        ([40, 64, 1, 200], 200, 136), ([2000, 3, 700, 90], 264, 776)):
        x = _randn(gen, sum(sizes), k, dtype=torch.bfloat16)
        w = _randn(gen, 4, k, n, dtype=torch.bfloat16)
        off = _offsets(sizes)
        y, d = torch.empty(sum(sizes), n, device="cuda").bfloat16(), torch.empty(4, k, n, device="cuda")
        capi.muon_grouped_mm(x, w, off, y)
        capi.muon_grouped_wgrad(x, y, off, d)
        jobs.append((x, w, off, y, d, torch.empty_like(y), torch.empty_like(d), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, off, y, d, y2, d2, side in jobs:
            capi.muon_grouped_mm(x, w, off, y2, stream=side)
            capi.muon_grouped_wgrad(x, y2, off, d2, stream=side)
    torch.cuda.synchronize()
    capi.muon_check()
    for x, w, off, y, d, y2, d2, side in jobs:
        assert torch.equal(y, y2) and torch.equal(d, d2)


def test_products_past_2_to_the_31_elements(capi):
    """Rows whose first element lies past 2^31 elements (4 GB) of x, y and a."""
    rows, k, n = 1_050_000, 2048, 2056
    x = torch.zeros(rows, k, device="cuda", dtype=torch.bfloat16)
    gen = _gen(19)
    x[-200:] = _randn(gen, 200, k, dtype=torch.bfloat16)
    w = _randn(gen, 2, k, n, dtype=torch.bfloat16, std=0.1)
    off = torch.tensor([0, rows - 100, rows], dtype=torch.int64, device="cuda")
    y = torch.full((rows, n), 3.0, device="cuda", dtype=torch.bfloat16)
    capi.muon_grouped_mm(x, w, off, y)
    capi.muon_check()
    for i, part in ((0, slice(rows - 200, rows - 100)), (1, slice(rows - 100, rows))):
        xd, wd = x[part].double(), w[i].double()
        _close(y[part], xd @ wd, xd.abs() @ wd.abs(), k, f"expert {i}")
    assert (y[:rows - 200] == 0).all()
    dw = torch.empty(2, 64, n, device="cuda")
    capi.muon_grouped_wgrad(x[:, :64], y, off, dw)
    capi.muon_check()
    ad, bd = x[-100:, :64].double(), y[-100:].double()
    _close(dw[1], ad.T @ bd, ad.abs().T @ bd.abs(), 100, "dw of the last rows")


def test_binding_refuses(capi):
    x = torch.zeros(4, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(2, 16, 8, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)
    off = _offsets([2, 2])
    ok = (x, w, off, y)
    capi.muon_grouped_mm(*ok)
    bad = [(x.float(), w, off, y), (x.half(), w, off, y), (x.cpu(), w, off, y), (x, w, off.int(), y),
           (x, w, off[:2], y), (x, w, off.cpu(), y), (x, w, off, y[:3]), (x, w, off, y.half()),
           (x[:, :8], w, off, y), (x.T.contiguous().T, w, off, y), (x, w.float(), off, y)]
    for args in bad:
        with pytest.raises(ValueError):
            capi.muon_grouped_mm(*args)
    with pytest.raises(capi.MuonError):      # expanded rows overlap
        capi.muon_grouped_mm(x[:1].expand(4, 16), w, off, y)
    dw = torch.zeros(2, 16, 8, device="cuda")
    capi.muon_grouped_wgrad(x, y, off, dw)
    for args in ((x, y, off, dw.bfloat16()), (x[:2], y, off, dw), (x, y.half(), off, dw),
                 (x, y, off[:2], dw)):
        with pytest.raises(ValueError):
            capi.muon_grouped_wgrad(*args)
    with pytest.raises(capi.MuonError):      # a workspace that is too small
        xo = torch.zeros(4, 17, device="cuda", dtype=torch.bfloat16)
        wo = torch.zeros(2, 17, 8, device="cuda", dtype=torch.bfloat16)
        capi.muon_grouped_mm(xo, wo, off, y,
                             workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    capi.muon_check()


# ----------------------------------------------------------------------------- activation
def _swiglu_exact(g, u, p):
    g, u = g.double(), u.double()
    s = torch.sigmoid(g)
    return p.double()[:, None] * g * s * u


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,cols,extra", [(1, 1, 0), (1, 1408, 0), (3, 7, 0), (192, 1408, 8),
                                             (37, 129, 3), (11000, 24, 0), (11000, 25, 7),
                                             (2, 16384, 0), (300, 4096, 16)])
@pytest.mark.parametrize("weighted", [True, False])
def test_swiglu_and_gradient(capi, dtype, rows, cols, extra, weighted):
    gen = _gen(rows * 31 + cols)
    t = DT[dtype]

    def make(std=1.0):
        return _strided(_randn(gen, rows, cols, dtype=t, std=std), cols + extra, 0)

    g, u, da = make(3.0), make(), make()
    p = torch.rand(rows, generator=gen, device="cuda") if weighted else None
    p1 = p if weighted else torch.ones(rows, device="cuda")
    bufs = [torch.full((rows, cols + extra), 9.0, dtype=t, device="cuda") for _ in range(3)]
    a, dg, du = (b[:, :cols] for b in bufs)
    dp = torch.empty(rows, device="cuda") if weighted else None
    capi.muon_swiglu(g, u, a, row_weight=p)
    capi.muon_swiglu_grad(da, g, u, dg, du, row_weight=p, d_row_weight=dp)
    capi.muon_check()
    assert all((b[:, cols:] == 9.0).all() for b in bufs), "wrote outside"
    G, U, D = g.double(), u.double(), da.double()
    s = torch.sigmoid(G)
    P = p1.double()[:, None]
    want = P * G * s * U
    _close(a, want, want.abs(), 16, "a")
    want = D * P * G * s
    _close(du, want, want.abs(), 16, "du")
    want = D * P * U * s * (1 + G * (1 - s))
    _close(dg, want, (D * P * U * s).abs() * (1 + G.abs() * (1 - s)), 16, "dg")
    if weighted:
        terms = D * G * s * U
        _close(dp, terms.sum(1), terms.abs().sum(1), 16 + cols, "dp")


def test_swiglu_extreme_gates(capi):
    g = torch.tensor([[0.0, -0.0, 30.0, -30.0, 100.0, -100.0, 3e38, -3e38]], device="cuda")
    u = torch.ones_like(g)
    a, dg, du = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    capi.muon_swiglu(g, u, a)
    capi.muon_swiglu_grad(u, g, u, dg, du)
    capi.muon_check()
    assert torch.isfinite(a).all() and torch.isfinite(du).all()
    assert torch.allclose(a[0, :5].double(), (g[0, :5].double() * torch.sigmoid(g[0, :5].double())), rtol=1e-6, atol=0)
    assert (a[0, 5] == 0 or abs(a[0, 5]) < 1e-40) and a[0, 6] == g[0, 6] and abs(a[0, 7]) == 0
    assert torch.allclose(dg[0, :5].cpu(), torch.tensor([0.5, 0.5, 1.0, -29 * math.exp(-30.0), 1.0]),
                          rtol=1e-5)
    assert dg[0, 6] == 1.0 and dg[0, 5].abs() < 1e-40 and dg[0, 7].abs() == 0


def test_swiglu_gradient_against_differences(capi):
    gen = _gen(23)
    rows, cols = 5, 40
    g, u, da = (_randn(gen, rows, cols) for _ in range(3))
    p = torch.rand(rows, generator=gen, device="cuda")
    dg, du, dp = torch.empty_like(g), torch.empty_like(u), torch.empty_like(p)
    capi.muon_swiglu_grad(da, g, u, dg, du, row_weight=p, d_row_weight=dp)
    capi.muon_check()
    h = 1e-5
    for t, grad, move in ((g, dg, lambda e: (g.double() + e, u, p)),
                          (u, du, lambda e: (g, u.double() + e, p))):
        diff = (_swiglu_exact(*move(h)) - _swiglu_exact(*move(-h))) / (2 * h) * da.double()
        assert torch.allclose(grad.double(), diff, rtol=1e-5, atol=1e-6)
    diff = ((_swiglu_exact(g, u, p.double() + h) - _swiglu_exact(g, u, p.double() - h)) / (2 * h)
            * da.double()).sum(1)
    assert torch.allclose(dp.double(), diff, rtol=1e-5, atol=1e-5)


def test_swiglu_halves_of_one_tensor_and_refusals(capi):
    gen = _gen(29)
    h = _randn(gen, 10, 64, dtype=torch.bfloat16)
    a = torch.empty(10, 32, device="cuda", dtype=torch.bfloat16)
    capi.muon_swiglu(h[:, :32], h[:, 32:], a)
    b = torch.empty_like(a)
    capi.muon_swiglu(h[:, :32].contiguous(), h[:, 32:].contiguous(), b)
    empty = torch.empty(0, 32, device="cuda", dtype=torch.bfloat16)
    capi.muon_swiglu(empty, empty, empty)
    capi.muon_check()
    assert torch.equal(a, b)
    for args, kw in (((a, b.half(), a), {}), ((a, b[:5], a), {}), ((a.cpu(), b, a), {}),
                     ((a, b, a), {"row_weight": torch.ones(9, device="cuda")}),
                     ((a, b, a), {"row_weight": torch.ones(10, device="cuda").double()}),
                     ((a.double(), b, a), {}), ((a.T, a.T, a.T), {})):
        with pytest.raises(ValueError):
            capi.muon_swiglu(*args, **kw)
