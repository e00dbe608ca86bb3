"""The gated gradient's row-weight gradients are fp32 results, as muon_swiglu_grad's are: with dh exact (one term
in a product), what is left is the activation.

Bound (derived, u = 2^-24): the power of two is within 2 ulp (4 u) and its argument within 2 u of its value's effect,
squared: 12 u with that rounding; the reciprocal 2 u of 1 + e, itself rounded; six more roundings in a term and one
for each addition: (24 + columns) u of a row whose terms have one sign.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


@pytest.mark.parametrize("n", [8, 40, 136])
@pytest.mark.parametrize("rows", [40, 4096, 30000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_row_weight_gradients_are_fp32_results(capi, dtype, rows, n):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    g = torch.linspace(-80, 20, rows, device="cuda")[:, None].expand(rows, n).to(dtype).contiguous()
    g[g == 0] = 1.0
    u = (torch.rand(rows, n, generator=gen, device="cuda") + 0.5).to(dtype)
    dy, w = torch.zeros(rows, 8, device="cuda", dtype=dtype), torch.zeros(1, n, 8, device="cuda", dtype=dtype)
    dy[:, 0] = torch.rand(rows, generator=gen, device="cuda") + 0.5
    w[:, :, 0] = 1.0
    dgate, dup, dp = torch.empty_like(g), torch.empty_like(g), torch.empty(rows, device="cuda")
    capi.muon_gated_mm_grad(dy, w, None, g, u, dgate, dup, d_row_weight=dp, trans_w=True)
    capi.muon_check()
    gd = g.double()
    want = (dy[:, :1].double() * gd * torch.sigmoid(gd) * u.double()).sum(1)
    err = ((dp.double() - want) / want).abs()
    print("worst, in u:", err.max().item() / U)
    assert err.max() <= (24 + n) * U


def test_infinite_gates_and_nan(capi):
    """silu(inf) is inf, as the products make of it; a NaN stays in its row."""
    g = torch.full((40, 16), 1.0, device="cuda").bfloat16()
    g[3, 5], g[7, 2] = float("inf"), float("nan")
    u, dy = torch.ones_like(g), torch.ones(40, 8, device="cuda").bfloat16()
    w = torch.zeros(1, 16, 8, device="cuda").bfloat16()
    w[:, :, 0] = 1.0
    dgate, dup, out, dp = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g), torch.empty(40, device="cuda")
    capi.muon_gated_mm_grad(dy, w, None, g, u, dgate, dup, out=out, d_row_weight=dp, trans_w=True)
    capi.muon_check()
    assert (dup[3, 5] == torch.inf) and (out[3, 5] == torch.inf) and dp[3] == torch.inf
    assert dup[7, 2].isnan() and out[7, 2].isnan() and dgate[7, 2].isnan() and dp[7].isnan()
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[3] = keep[7] = False
    for t in (dgate, dup, out):
        assert torch.equal(t[keep], t[:1].expand(38, 16)) and torch.isfinite(t[keep]).all()
    assert (dp[keep] == dp[0]).all() and torch.isfinite(dp[0])
