"""The feed-forward calls at the ends of their ranges: rows further apart than 32-bit offsets reach, the
most experts, several streams at once, long rows in a graph."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FAR = (1 << 30) + 16      # the third row starts behind 2^31 elements
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


def _randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


@pytest.fixture()
def far():
    """A matrix of 3 rows, FAR elements apart, of a buffer that is not written elsewhere by the test."""
    buf = torch.empty(2 * FAR + 1024, dtype=torch.bfloat16, device="cuda")

    def view(cols, at=0):
        return buf.as_strided((3, cols), (FAR, 1), at)

    yield view
    del buf
    torch.cuda.empty_cache()


def test_far_rows_of_the_gated_block(capi, far):
    x, w1, w2 = _randn(1, 3, 136), _randn(2, 1, 136, 264), _randn(3, 1, 136, 264)
    out, gate, up = (torch.empty(3, 264, device="cuda").bfloat16() for _ in range(3))
    capi.muon_gated_mm(x, w1, w2, None, out, gate=gate, up=up)
    fx = far(136)
    fx.copy_(x)
    got = far(264, 512)
    capi.muon_gated_mm(fx, w1, w2, None, got)          # far operands and results
    capi.muon_check()
    assert torch.equal(got, out)
    dy, wd = _randn(4, 3, 72), _randn(5, 1, 264, 72)
    want = [torch.empty_like(out) for _ in range(3)]
    capi.muon_gated_mm_grad(dy, wd, None, gate, up, *want[:2], out=want[2], trans_w=True)
    for k in range(3):      # each result far in turn, and the gate far
        mine = [torch.empty_like(out) for _ in range(3)]
        mine[k] = far(264)
        fg = far(264, 512)
        fg.copy_(gate)
        capi.muon_gated_mm_grad(dy, wd, None, fg, up, *mine[:2], out=mine[2], trans_w=True)
        capi.muon_check()
        assert all(torch.equal(a, b) for a, b in zip(mine, want))
    y = torch.empty(3, 136, device="cuda").bfloat16()
    capi.muon_grouped_mm_sum(want[0], w1, want[1], w2, None, y, trans_w=True)
    fy = far(136, 512)
    capi.muon_grouped_mm_sum(want[0], w1, want[1], w2, None, fy, trans_w=True)
    capi.muon_check()
    assert torch.equal(fy, y)


def test_far_rows_in_8_bits(capi, far):
    x = _randn(6, 3, 272)
    q, scale = torch.empty(3, 272, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(3, 3, device="cuda")
    q2, scale2 = torch.empty_like(q), torch.empty_like(scale)
    capi.muon_quantize_rows(x, q, scale)
    fx = far(272)
    fx.copy_(x)
    capi.muon_quantize_rows(fx, q2, scale2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale, scale2)
    wq, ws = torch.empty(1, 200, 272, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(1, 2, 3, device="cuda")
    capi.muon_quantize_weights(_randn(7, 1, 272, 200), wq, ws, transpose=True)
    y, fy = torch.empty(3, 200, device="cuda").bfloat16(), far(200, 512)
    capi.muon_grouped_mm_fp8(q, scale, wq, ws, None, y)
    capi.muon_grouped_mm_fp8(q, scale, wq, ws, None, fy)
    capi.muon_check()
    assert torch.equal(y, fy)


@pytest.mark.parametrize("rows", [1024, 20_000])
def test_the_most_experts(capi, rows):
    """1024 experts, some without rows: against the products of each by itself in the plain call."""
    e, k, n = 1024, 64, 136
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    cut = torch.randint(0, rows + 1, (e - 1,), generator=g, device="cuda").sort().values
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), rows)])
    x, w1, w2 = _randn(1, rows, k), _randn(2, e, k, n) * 0.125, _randn(3, e, k, n) * 0.125
    gate, up, out, a, b = (torch.empty(rows, n, device="cuda").bfloat16() for _ in range(5))
    capi.muon_gated_mm(x, w1, w2, off, out, gate=gate, up=up)
    capi.muon_grouped_mm(x, w1, off, a)
    capi.muon_grouped_mm(x, w2, off, b)
    capi.muon_check()
    # (Sums may be cut at other places: a rounding of the store apart at most, 2^-7 of the value and of
    # the fp32 sums' errors, 64 * 2^-23 * sum |x w| < 2^-14.)
    for got, want in ((gate, a), (up, b)):
        assert ((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -13).all()
    xq, xs = torch.empty(rows, k, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(1, rows, device="cuda")
    wq, ws = torch.empty(e, n, k, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(e, 2, 1, device="cuda")
    capi.muon_quantize_rows(x, xq, xs)
    capi.muon_quantize_weights(w1, wq, ws, transpose=True)
    y = torch.empty(rows, n, device="cuda")
    capi.muon_grouped_mm_fp8(xq, xs, wq, ws, off, y)
    capi.muon_check()
    xd = xq.float() * xs[0][:, None]
    wd = wq.float() * ws[:, :, 0].repeat_interleave(128, 1)[:, :n, None]
    owner = torch.searchsorted(off[1:].contiguous(), torch.arange(rows, device="cuda"), right=True)
    for r in range(0, rows, max(1, rows // 200)):
        want = wd[owner[r]].double() @ xd[r].double()
        mag = wd[owner[r]].double().abs() @ xd[r].double().abs()
        assert ((y[r].double() - want).abs() <= 132 * 2.0 ** -23 * mag + 2.0 ** -24 * want.abs()).all()


def test_many_streams(capi):
    """Odd sizes, whose operands are copied to workspaces, on four streams at once while the current stream
    takes and frees blocks."""
    jobs = []
    for i, (rows, k, n) in enumerate(((700, 513, 231), (13, 1023, 265), (305, 201, 135), (2793, 263, 777))):
        x, w1, w2 = _randn(i, rows, k), _randn(i + 9, 1, k, n), _randn(i + 19, 1, k, n)
        wd = _randn(i + 29, 1, n, k)
        p = torch.rand(rows, device="cuda")

        def new(c):
            return torch.zeros(rows, c, device="cuda").bfloat16()

        def step(stream, x=x, w1=w1, w2=w2, wd=wd, p=p, outs=None):
            out, gate, up, dgate, dup, dx, n_, dn, mean, rstd, dw, dp = outs
            capi.muon_layer_norm(x, None, None, n_, mean=mean, rstd=rstd, stream=stream)
            capi.muon_gated_mm(n_, w1, w2, None, out, gate=gate, up=up, row_weight=p, stream=stream)
            capi.muon_gated_mm_grad(x, wd, None, gate, up, dgate, dup, row_weight=p, d_row_weight=dp,
                                    trans_w=True, stream=stream)
            capi.muon_grouped_mm_sum(dgate, w1, dup, w2, None, dx, trans_w=True, stream=stream)
            capi.muon_layer_norm_grad(dx, x, None, mean, rstd, dn, dw, None, stream=stream)

        def outs():
            return [new(n), new(n), new(n), new(n), new(n), new(k), new(k), new(k), torch.zeros(rows, device="cuda"),
                    torch.zeros(rows, device="cuda"), torch.zeros(k, device="cuda"), torch.zeros(rows, device="cuda")]

        want, mine = outs(), outs()
        step(None, outs=want)
        jobs.append((step, want, mine, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(10):
        for step, want, mine, side in jobs:
            step(side if i % 2 else side.cuda_stream, outs=mine)
            torch.full((50_000 * (i + 1),), 3.0e38, device="cuda").mul_(2)
    torch.cuda.synchronize()
    capi.muon_check()
    for step, want, mine, side in jobs:
        assert all(torch.equal(a, b) for a, b in zip(want, mine))


def test_long_rows_captured_first(capi):
    """The gradient of rows whose weights take more shared memory than a launch has by default, in a graph
    before any eager call of that size."""
    x, dy = _randn(1, 900, 14336), _randn(2, 900, 14336)
    w = torch.rand(14336, device="cuda")
    mean, rstd = torch.zeros(900, device="cuda"), torch.ones(900, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    capi.muon_layer_norm(x[:, :64].contiguous(), None, None, torch.empty(900, 64, device="cuda").bfloat16())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.muon_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db)
    graph.replay()
    got = [t.clone() for t in (dx, dw, db)]
    capi.muon_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db)
    assert all(torch.equal(a, b) for a, b in zip(got, (dx, dw, db)))


def test_no_rows(capi):
    x, w = torch.empty(0, 64, device="cuda").bfloat16(), _randn(1, 2, 64, 136)
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    y, p = torch.empty(0, 136, device="cuda").bfloat16(), torch.empty(0, device="cuda")
    capi.muon_gated_mm(x, w, w, off, y, gate=y, up=y, row_weight=p)
    capi.muon_gated_mm_grad(x, w, off, y, y, y, y, out=y, row_weight=p, d_row_weight=p)
    capi.muon_grouped_mm_sum(x, w, x, w, off, y)
    capi.muon_quantize_rows(x, torch.empty(0, 64, dtype=torch.uint8, device="cuda").view(E4M3),
                            torch.empty(1, 0, device="cuda"))
    capi.muon_check()
