"""Weight gradients into matrices that do not lie one behind the other."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("m,n,gap", [(72, 136, 0), (130, 37, 3), (300, 264, 8)])
def test_rows_of_all_experts_side_by_side(capi, m, n, gap, accumulate):
    """dw[e, i, :] in an (m, experts, n + gap) buffer: exact sums of small integers, the rest untouched."""
    sizes = [33, 0, 100, 700]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m)
    a, b = (torch.randint(-8, 9, (sum(sizes), c), generator=gen, device="cuda").bfloat16() for c in (m, n))
    buf = torch.full((m, 4, n + gap), 5.0, device="cuda")
    off = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], device="cuda")
    capi.muon_grouped_wgrad(a, b, off, buf[:, :, :n].transpose(0, 1), accumulate=accumulate)
    capi.muon_check()
    want = torch.stack([x.double().T @ y.double() for x, y in zip(a.split(sizes), b.split(sizes))], 1)
    assert torch.equal(buf[:, :, :n].double(), want + 5.0 * accumulate)
    assert (buf[:, :, n:] == 5.0).all()


def test_overlapping_rows_are_refused(capi):
    a = torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)
    buf = torch.zeros(1000, device="cuda")
    off = torch.tensor([0, 2, 4], device="cuda")
    for strides in ((63, 8, 1), (60, 16, 1), (8, 15, 1)):
        with pytest.raises(capi.MuonError) as e:
            capi.muon_grouped_wgrad(a, a, off, buf.as_strided((2, 8, 8), strides))
        assert e.value.status == capi.MUON_ERR_INVALID_ARG
    for strides in ((64, 8, 1), (8, 16, 1), (9, 17, 1)):
        capi.muon_grouped_wgrad(a, a, off, buf.as_strided((2, 8, 8), strides))
    capi.muon_check()
