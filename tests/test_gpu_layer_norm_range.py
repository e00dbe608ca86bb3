"""The layer norm's gradient for rows of a tiny spread, whose rstd squared is beyond fp32 (eps = 0 allows
them), with every share of a row: the same bound as for ordinary rows (see test_gpu_layer_norm.py), which is
relative to the values."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gpu_layer_norm import DT, U, _depth, _gen, _within  # noqa: E402


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


@pytest.mark.parametrize("spread", [2.0 ** -60, 2.0 ** -64, 2.0 ** -70])
@pytest.mark.parametrize("rows,cols,dtype", [
    (7, 1, "fp32"), (9, 8, "fp32"), (40, 32, "fp32"), (40, 96, "fp32"), (900, 128, "fp32"), (20, 2048, "fp32"),
    (400, 2048, "fp32"), (400, 4096, "fp32"), (400, 771, "fp32"), (400, 8192, "fp32"), (9, 8200, "fp32"),
    (400, 48, "bf16"), (40, 96, "bf16"), (40, 200, "bf16"), (5, 4096, "bf16"), (5, 500, "bf16"), (400, 1024, "bf16"),
    (400, 4096, "bf16"), (20, 4097, "bf16"), (20, 8192, "bf16"), (20, 16400, "bf16"),
])
def test_rows_of_a_tiny_spread(capi, rows, cols, dtype, spread):
    gen = _gen(rows + cols)
    x = (torch.randn(rows, cols, generator=gen, device="cuda") * spread).to(DT[dtype])
    dy = (torch.randn(rows, cols, generator=gen, device="cuda") * 2.0 ** -10).to(DT[dtype])
    w = 1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")
    # (One value by itself has no spread: any mean and rstd will do.)
    xd = x.double()
    mean = (xd.mean(1) if cols > 1 else torch.zeros(rows, device="cuda")).float()
    rstd = (1.0 / xd.std(1, correction=0) if cols > 1 else torch.full((rows,), 1.0 / spread, device="cuda")).float()
    dx, dw, db = torch.full_like(x, 7.0), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    capi.muon_layer_norm_grad(dy, x, w, mean, rstd, dx, dw, db)
    capi.muon_check()
    md, rd, dd = mean.double()[:, None], rstd.double()[:, None], dy.double()
    xh, t = (xd - md) * rd, dd * w.double()
    m1, m2 = t.mean(1)[:, None], (t * xh).mean(1)[:, None]
    mag = rd * (t.abs() + t.abs().mean(1)[:, None] + xh.abs() * (t * xh).abs().mean(1)[:, None])
    _within(dx, rd * (t - m1 - xh * m2), (_depth(cols) + 16) * U * mag, "dx")
    for got, terms in ((dw, dd * xh), (db, dd)):
        _within(got, terms.sum(0), (rows + 8) * U * terms.abs().sum(0), "sums over the rows")
