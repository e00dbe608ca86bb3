"""How the grouped products add up.

The tensor core cuts what does not fit its accumulator, always towards zero, so a sum's error grows
with its number of steps.  Results are therefore summed in segments, added with rounding to nearest,
and their error does not grow with the length."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


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


def _offsets(sizes):
    o = [0]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("k", [4096, 16384])
@pytest.mark.parametrize("dtype,bits", [("bf16", 7), ("fp16", 10)])
@pytest.mark.parametrize("sizes,n", [
    ([1500, 700, 1], 2312),      # pairs
    ([900, 3], 1416),            # single CTAs
    ([60, 50, 64, 7], 2056),     # narrow tiles
    ([40, 20], 264),             # k split over a cluster
])
def test_long_16_bit_results_are_rounded_right(capi, sizes, n, dtype, bits, k):
    """The share of results that are not the exact sum's rounding.  A value v in 2^e .. 2^(e+1) is stored
    in steps of 2^(e - bits), so an error of d |v| moves it to another step with a chance of at
    most 2 d 2^bits, and one of c times the results' root mean square with about 6 c 2^bits (0.4 c
    2^bits from each octave of small values, some 15 of them).  With d = 6.5e-7 for what a segment cuts
    and c = 2.5e-7 for the rest that is 2.8e-6 2^bits; 4e-6 2^bits are allowed (whole sums of 4096
    terms: 7e-6 and more, of 16384: 2e-5)."""
    gen = _gen(len(sizes) * n + k)
    x = torch.randn(sum(sizes), k, generator=gen, device="cuda").to(DT[dtype])
    w = (torch.randn(len(sizes), k, n, generator=gen, device="cuda") * 0.1).to(DT[dtype])
    y = torch.empty(sum(sizes), n, dtype=DT[dtype], device="cuda")
    capi.muon_grouped_mm(x, w, _offsets(sizes), y)
    capi.muon_check()
    want = torch.cat([a.double() @ b.double() for a, b in zip(x.split(sizes), w)])
    wrong = (y != want.to(DT[dtype])).double().mean().item()
    assert wrong <= 4e-6 * 2.0 ** bits + 2 / y.numel()


def _frobenius(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.fixture()
def plain_products():
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = old


@pytest.mark.parametrize("experts,rows,m,n", [(1, 1536, 520, 1416), (1, 1536, 72, 136), (1, 20000, 72, 136),
                                              (1, 20000, 776, 1416), (8, 1536, 2048, 1408), (13, 320, 130, 520),
                                              (64, 384, 256, 1408)])
def test_weight_gradients_are_as_exact_as_plain_fp32(capi, plain_products, experts, rows, m, n):
    """At most one rounding (2^-24) more than torch's fp32 product of the same values."""
    gen = _gen(rows + m)
    a = torch.randn(experts * rows, m, generator=gen, device="cuda").bfloat16()
    b = torch.randn(experts * rows, n, generator=gen, device="cuda").bfloat16()
    dw = torch.empty(experts, m, n, device="cuda")
    capi.muon_grouped_wgrad(a, b, _offsets([rows] * experts), dw)
    capi.muon_check()
    a, b = a.view(experts, rows, m).mT, b.view(experts, rows, n)
    want = a.double() @ b.double()
    plain = torch.stack([x @ y for x, y in zip(a.float(), b.float())])
    assert _frobenius(dw, want) <= _frobenius(plain, want) + 2.0 ** -24


@pytest.mark.parametrize("rows,k,n", [(3000, 2048, 1416), (600, 771, 517), (40, 2048, 2056),
                                      (33, 4104, 264)])
def test_fp32_products_are_as_exact_as_plain_fp32(capi, plain_products, rows, k, n):
    gen = _gen(rows + k)
    x = torch.randn(rows, k, generator=gen, device="cuda").half()
    w = torch.randn(1, k, n, generator=gen, device="cuda").half()
    y = torch.empty(rows, n, device="cuda")
    capi.muon_grouped_mm(x, w, _offsets([rows]), y)
    capi.muon_check()
    want = x.double() @ w[0].double()
    assert _frobenius(y, want) <= _frobenius(x.float() @ w[0].float(), want) + 2.0 ** -24


def _integers(gen, *shape, dtype="bf16"):
    return torch.randint(-8, 9, shape, generator=gen, device="cuda").to(DT[dtype])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("sizes,m,n", [
    ([20000, 3], 72, 136),                                # one tile: shares of a cluster
    ([19969, 0, 19983, 19984, 19985], 32, 216),           # off and on the 16-row steps
    ([8191, 8192, 8193, 4095, 4097, 1], 130, 40),         # off and on the shares' edges
    ([511, 512, 513, 1023, 1025, 15, 16, 17, 1], 776, 520),
    ([2000, 1999, 65, 63, 64, 1], 264, 1416),
])
def test_weight_gradients_of_integers_are_exact(capi, sizes, m, n, accumulate):
    """Sums of products of integers up to 8 stay below 2^24: every row has to be in, exactly once."""
    gen = _gen(sum(sizes))
    a, b = _integers(gen, sum(sizes), m), _integers(gen, sum(sizes), n)
    dw = _integers(gen, len(sizes), m, n, dtype="fp32")
    want = torch.stack([x.double().T @ y.double() for x, y in zip(a.split(sizes), b.split(sizes))])
    if accumulate:
        want += dw
    capi.muon_grouped_wgrad(a, b, _offsets(sizes), dw, accumulate=accumulate)
    capi.muon_check()
    assert torch.equal(dw.double(), want)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,k,n", [
    ([33], 2047, 130), ([1], 2049, 264), ([3, 0, 2], 4097, 77), ([64], 1023, 520), ([7, 9], 8255, 136),
    ([700, 300, 0, 900], 1609, 2312), ([64, 1, 40], 777, 1416),
])
def test_products_of_integers_are_exact(capi, sizes, k, n, trans):
    gen = _gen(k + n)
    x = _integers(gen, sum(sizes), k, dtype="fp16")
    w = _integers(gen, *((len(sizes), n, k) if trans else (len(sizes), k, n)), dtype="fp16")
    y = torch.empty(sum(sizes), n, device="cuda")
    capi.muon_grouped_mm(x, w, _offsets(sizes), y, trans_w=trans)
    capi.muon_check()
    want = torch.cat([a.double() @ (b.double().T if trans else b.double())
                      for a, b in zip(x.split(sizes), w)])
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("sizes,k,n", [([1], 2048, 256), ([0, 3, 2, 0], 1600, 264), ([33], 1090, 130),
                                       ([2, 7], 4099, 77)])
def test_special_values_in_split_products(capi, sizes, k, n, trans):
    """k split over a cluster: a NaN or infinity of any part reaches its row (or, in the weight, its
    column of its expert's rows), and nothing else."""
    gen = _gen(k)
    rows = sum(sizes)
    x = (0.5 + torch.rand(rows, k, generator=gen, device="cuda")).bfloat16()
    w = (0.5 + torch.rand(len(sizes), k, n, generator=gen, device="cuda")).bfloat16()
    off = _offsets(sizes)
    edge = off.tolist()

    def product():
        y = torch.empty(rows, n, device="cuda")
        capi.muon_grouped_mm(x, w.mT.contiguous() if trans else w, off, y, trans_w=trans)
        capi.muon_check()
        return y

    y0 = product()
    assert torch.isfinite(y0).all()
    for at in (0, k // 8 - 1, k // 2, k - 1):        # some part's k, the last one's among them
        for value in (float("nan"), float("inf"), float("-inf")):
            old = x[rows - 1, at].clone()
            x[rows - 1, at] = value
            y = product()
            x[rows - 1, at] = old
            assert torch.equal(y[:-1], y0[:-1])
            assert torch.isnan(y[-1]).all() if value != value else (y[-1] == value).all()
            e = max(i for i, s in enumerate(sizes) if s)
            old = w[e, at, n - 1].clone()
            w[e, at, n - 1] = value
            y = product()
            w[e, at, n - 1] = old
            hit = y[edge[e]:edge[e + 1], n - 1]
            assert torch.isnan(hit).all() if value != value else (hit == value).all()
            y[edge[e]:edge[e + 1], n - 1] = y0[edge[e]:edge[e + 1], n - 1]
            assert torch.equal(y, y0)


@pytest.mark.parametrize("sizes,m,n", [([5000], 32, 216), ([2300, 0, 4097, 1], 72, 136), ([9, 1500], 256, 65)])
def test_special_values_in_split_weight_gradients(capi, sizes, m, n):
    """Rows split over a cluster: the same for a NaN or infinity in any share's rows."""
    gen = _gen(m)
    a = (0.5 + torch.rand(sum(sizes), m, generator=gen, device="cuda")).bfloat16()
    b = (0.5 + torch.rand(sum(sizes), n, generator=gen, device="cuda")).bfloat16()
    off = _offsets(sizes)
    edge = off.tolist()

    def gradient():
        dw = torch.empty(len(sizes), m, n, device="cuda")
        capi.muon_grouped_wgrad(a, b, off, dw)
        capi.muon_check()
        return dw

    d0 = gradient()
    assert torch.isfinite(d0).all()
    for e, size in enumerate(sizes):
        for row in {0, size // 3, size // 2, size - 1} if size else ():
            for value in (float("nan"), float("inf")):
                at = edge[e] + row
                old = a[at, m - 1].clone()
                a[at, m - 1] = value
                dw = gradient()
                a[at, m - 1] = old
                hit = dw[e, m - 1]
                assert torch.isnan(hit).all() if value != value else (hit == value).all()
                dw[e, m - 1] = d0[e, m - 1]
                assert torch.equal(dw, d0)
