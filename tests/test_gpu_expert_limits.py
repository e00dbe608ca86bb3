"""Products at the top of their row range: 2^31 - 1 rows (34 GB an operand)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROWS = 2 ** 31 - 1


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


@pytest.fixture(scope="module")
def operands(capi):
    """Two operands of ROWS x 8, zero but for small integers in the rows `at`: the first and last
    ones and some between."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    at = torch.cat([torch.arange(200, device="cuda"), ROWS - 1 - torch.arange(200, device="cuda"),
                    torch.randint(200, ROWS - 200, (4000,), generator=gen, device="cuda")]).unique()
    out = []
    for _ in range(2):
        t = torch.zeros(ROWS, 8, device="cuda", dtype=torch.bfloat16)
        t[at] = torch.randint(-8, 9, (len(at), 8), generator=gen, device="cuda").bfloat16()
        out.append(t)
    yield at, *out
    del out, t
    torch.cuda.empty_cache()


def test_product(capi, operands):
    at, x, _ = operands
    w = torch.randint(-8, 9, (2, 8, 8), device="cuda").bfloat16()
    for first in (0, ROWS):                      # one expert has every row
        y = torch.full((ROWS, 8), 3.0, device="cuda", dtype=torch.bfloat16)
        capi.muon_grouped_mm(x, w, torch.tensor([0, first, ROWS], device="cuda"), y)
        capi.muon_check()
        want = (x[at].double() @ w[0 if first else 1].double()).bfloat16()
        assert torch.equal(y[at], want)
        y[at] = 0
        assert not y.any()
        del y


@pytest.mark.parametrize("experts,owner", [(1, 0),      # the rows split over a cluster
                                           (77, 40)])   # one CTA takes them all
def test_weight_gradient(capi, operands, experts, owner):
    at, a, b = operands
    want = a[at].double().T @ b[at].double()
    off = torch.tensor([0] * (owner + 1) + [ROWS] * (experts - owner), device="cuda")
    dw = torch.ones(experts, 8, 8, device="cuda")
    capi.muon_grouped_wgrad(a, b, off, dw, accumulate=True)
    capi.muon_check()
    assert torch.equal(dw[owner].double(), want + 1)
    dw[owner] = 1
    assert (dw == 1).all()
