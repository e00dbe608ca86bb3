"""The gated activation where its exponential leaves the ordinary range, and the exactness of the
gradient of the row weights, against plain 64-bit forms.

Bounds (derived): the sigmoid is e / (1 + e) or 1 / (1 + e) with e = exp(-|g|) of at most 2 ulp, a
division of at most 2 ulp and two roundings more; with the products around it 2^-19 of the value
covers the activation.  Below g = -87.3 the sigmoid is a subnormal number: each operation on it
may be off by 2^-149 on top, which the other factors then carry."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STORE = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (2.0 ** -24, 2.0 ** -149)}


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


@pytest.mark.parametrize("cols", [96, 97])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_gates_from_minus_110_to_110(capi, dtype, cols):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(cols)
    rows, t = 64, DT[dtype]
    g = torch.linspace(-110, 110, rows * cols, device="cuda").view(cols, rows).T.to(t)
    size = 6e4 if dtype == "fp16" else 1e36
    u = ((torch.rand(rows, cols, generator=gen, device="cuda") - 0.5) * size).to(t)
    u = torch.where(g > -60, torch.randn(rows, cols, generator=gen, device="cuda").to(t), u).contiguous()
    da = torch.randn(rows, cols, generator=gen, device="cuda").to(t)
    g = g.contiguous()
    p = torch.rand(rows, generator=gen, device="cuda") + 0.5
    a, dg, du = (torch.empty_like(g) for _ in range(3))
    dp = torch.empty_like(p)
    capi.muon_swiglu(g, u, a, row_weight=p)
    capi.muon_swiglu_grad(da, g, u, dg, du, row_weight=p, d_row_weight=dp)
    capi.muon_check()
    G, U, D, P = g.double(), u.double(), da.double(), p.double()[:, None]
    s, c = torch.sigmoid(G), torch.sigmoid(-G)
    off = s * 2.0 ** -19 + 4 * 2.0 ** -149       # of the sigmoid

    def close(got, want, bound, what):
        rel, tiny = STORE[dtype]
        bound = bound + rel * (want.abs() + bound) + tiny
        assert torch.isfinite(got).all(), what
        assert ((got.double() - want).abs() <= bound).all(), what

    close(a, P * G * s * U, (P * G * U).abs() * off, "a")
    close(du, D * P * G * s, (D * P * G).abs() * off, "du")
    close(dg, D * P * U * s * (1 + G * c), (D * P * U).abs() * (1 + G.abs() * c) * off, "dg")
    terms = (D * G * U).abs()
    err = (dp.double() - (D * G * U * s).sum(1)).abs()
    assert (err <= (terms * off).sum(1) + cols * 2.0 ** -24 * (terms * s).sum(1) + 2.0 ** -149).all(), "dp"


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_row_weight_gradients_are_fp32_results(capi, dtype):
    """A row of equal gates and terms of one sign: 2 ulp for the exponential and for the division
    (2^-22 each), four more roundings in a term and one for each addition (2^-24)."""
    rows, cols, t = 4096, 8, DT[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    g = torch.linspace(-80, 20, rows, device="cuda")[:, None].expand(rows, cols).to(t).contiguous()
    u, da = ((torch.rand(rows, cols, generator=gen, device="cuda") + 0.5).to(t) for _ in range(2))
    dg, du, dp = torch.empty_like(g), torch.empty_like(g), torch.empty(rows, device="cuda")
    capi.muon_swiglu_grad(da, g, u, dg, du, d_row_weight=dp)
    capi.muon_check()
    want = (da.double() * g.double() * torch.sigmoid(g.double()) * u.double()).sum(1)
    err = ((dp.double() - want) / want).abs()
    ok = want != 0
    assert err[ok].max() <= 2 * 2.0 ** -22 + (4 + cols) * 2.0 ** -24
