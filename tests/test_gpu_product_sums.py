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
                                              (1, 20000, 776, 1416), (8, 1536, 2048, 1408)])
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
