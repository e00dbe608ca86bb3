"""Calls on a stream of their own while the current stream goes on: their workspace must be
nobody else's."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


def _pending_use(nbytes, value):
    """A block of nbytes that the current stream still reads after it was freed, and the copy."""
    block = torch.full((nbytes,), value, dtype=torch.uint8, device="cuda")
    copy = torch.zeros_like(block)
    torch.cuda._sleep(50_000_000)
    copy.copy_(block)
    return copy


def _handles(side):
    return [side, side.cuda_stream]


def test_norm_leaves_pending_blocks_alone(capi):
    grads = [torch.randn(n, device="cuda") for n in (3_000_001, 77, 500_000)]
    want, got = torch.empty(2, device="cuda"), torch.zeros(2, device="cuda")
    capi.muon_grad_norm(grads, 1.0, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in _handles(side):
        for nbytes in (600, 2000, 4000, 4872, 5120):
            copy = _pending_use(nbytes, 1)
            capi.muon_grad_norm(grads, 1.0, got, stream=stream)
            torch.cuda.synchronize()
            assert (copy == 1).all() and torch.equal(got, want)
    outs = [torch.empty_like(g) for g in grads]
    side.wait_stream(torch.cuda.current_stream())
    capi.muon_clip_grads(grads, outs, 0.5, got, stream=side)
    side.synchronize()
    capi.muon_check()
    assert all(torch.equal(o, g * got[1]) for g, o in zip(grads, outs))


def test_products_leave_pending_blocks_alone(capi):
    sizes, k, n = [100, 3, 60], 77, 130          # rows off the 16-byte grid: both operands are copied
    x = torch.randn(sum(sizes), k, device="cuda").bfloat16()
    w = torch.randn(3, k, n, device="cuda").bfloat16()
    off = torch.tensor([0, 100, 103, 163], device="cuda")
    y, y2 = torch.zeros(sum(sizes), n, device="cuda"), torch.zeros(sum(sizes), n, device="cuda")
    d, d2 = torch.zeros(3, k, n, device="cuda"), torch.zeros(3, k, n, device="cuda")
    b = torch.randn(sum(sizes), n, device="cuda").bfloat16()
    capi.muon_grouped_mm(x, w, off, y)
    capi.muon_grouped_wgrad(x, b, off, d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in _handles(side):
        for nbytes in (20_000, 60_000, 80_000, 90_000, 120_000, 130_000):
            copy = _pending_use(nbytes, 2)
            capi.muon_grouped_mm(x, w, off, y2, stream=stream)
            capi.muon_grouped_wgrad(x, b, off, d2, stream=stream)
            torch.cuda.synchronize()
            assert (copy == 2).all() and torch.equal(y, y2) and torch.equal(d, d2)
    capi.muon_check()


def test_many_streams_with_workspaces(capi):
    """Odd sizes on four streams at once, while the current stream takes and frees blocks."""
    jobs = []
    for i, (sizes, k, n) in enumerate((([700, 300, 0, 900], 513, 231), ([3, 0, 9, 1], 1023, 265),
                                       ([40, 64, 1, 200], 201, 135), ([2000, 3, 700, 90], 263, 777))):
        x = torch.randn(sum(sizes), k, device="cuda").bfloat16()
        w = torch.randn(4, k, n, device="cuda").bfloat16()
        off = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], device="cuda")
        y, d = torch.empty(sum(sizes), n, device="cuda"), torch.empty(4, k, n, device="cuda")
        b = torch.randn(sum(sizes), n, device="cuda").bfloat16()
        capi.muon_grouped_mm(x, w, off, y)
        capi.muon_grouped_wgrad(x, b, off, d)
        jobs.append((x, w, b, off, y, d, torch.zeros_like(y), torch.zeros_like(d), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(20):
        for x, w, b, off, y, d, y2, d2, side in jobs:
            capi.muon_grouped_mm(x, w, off, y2, stream=side)
            capi.muon_grouped_wgrad(x, b, off, d2, stream=side if i % 2 else side.cuda_stream)
            torch.full((50_000 * (i + 1),), 3.0e38, device="cuda").mul_(2)
    torch.cuda.synchronize()
    capi.muon_check()
    for x, w, b, off, y, d, y2, d2, side in jobs:
        assert torch.equal(y, y2) and torch.equal(d, d2)


def test_default_stream_by_its_handle(capi):
    """0 is the default stream, where torch's own work also goes."""
    g = torch.ones(100_000, device="cuda")
    norm = torch.empty(2, device="cuda")
    torch.cuda._sleep(20_000_000)
    g.mul_(3)
    capi.muon_grad_norm([g], 1.0, norm, stream=0)
    assert float(norm[0]) == pytest.approx(3 * 100_000 ** 0.5, rel=1e-6)
