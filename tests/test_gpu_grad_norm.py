"""The global gradient norm, clipping, and the step that takes the coefficient, on the GPU.

Bounds (derived): a square passes at most 32 additions in fp32 (each square and each addition
rounds by 2^-24) and the sums go on in fp64, so the sum of squares is within 34 * 2^-24 of itself,
the norm within 17 * 2^-24 plus its own rounding (18 * 2^-24 in all), the coefficient within
19 * 2^-24, and a clipped fp32 element within 20 * 2^-24 of coefficient * element."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from muon_optimizer_step_gb300 import inputs  # noqa: E402

EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


def _exact(grads, max_norm):
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def _check(capi, grads, max_norm, out_fp32=False):
    norm, coef = _exact(grads, max_norm)
    outs = [torch.full_like(g, 7.0, dtype=torch.float32 if out_fp32 else g.dtype) for g in grads]
    nc, nc2 = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    before = [g.clone() for g in grads]
    capi.muon_grad_norm(grads, max_norm, nc2)
    capi.muon_clip_grads(grads, outs, max_norm, nc)
    capi.muon_check()
    assert torch.equal(nc, nc2)
    assert abs(float(nc[0]) - norm) <= 18 * EPS * norm
    assert abs(float(nc[1]) - coef) <= 19 * EPS * coef
    for g, b, o in zip(grads, before, outs):
        assert torch.equal(g, b)
        # the product of the stored coefficient: one fp32 rounding, then the store's
        assert torch.equal(o, (g.float() * nc[1]).to(o.dtype))
    return nc


@pytest.mark.parametrize("numels", [[1], [0], [], [0, 5, 0], [8192], [8191, 8193], [3, 1, 4, 1, 5],
                                    [40000, 37, 1, 66000], [1_000_003] * 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("max_norm", [0.0, 0.3, 1e6])
def test_norm_and_clip(capi, numels, dtype, max_norm):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sum(numels) + 1)
    # views of one buffer back to back, so that most start off the 16-byte grid
    flat = torch.randn(sum(numels) + 3, generator=gen, device="cuda").to(dtype)
    grads = list(flat[3:].split(numels)) if numels else []
    for out_fp32 in (False, True):
        _check(capi, grads, max_norm, out_fp32)


def test_more_tensors_than_one_launch_holds_and_mixed_types(capi):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    types = (torch.float32, torch.bfloat16, torch.float16)
    grads = [torch.randn(1 + (i * 37) % 900, generator=gen, device="cuda").to(types[i % 3])
             for i in range(2500)]
    grads[7] = torch.randn(100_000, generator=gen, device="cuda")
    _check(capi, grads, 1.0)
    _check(capi, grads, 1.0, out_fp32=True)


@pytest.mark.parametrize("scale", [1e30, 1e19, 1e-19, 1e-22, 1e-30, 1e-40, 3e38])
def test_whole_fp32_range(capi, scale):
    """Squares that overflow or vanish in fp32 still count."""
    g = torch.full((20000,), 1.0, device="cuda") * scale
    g[::3] = 0.0
    ref = g.double()
    nc = torch.empty(2, device="cuda")
    capi.muon_grad_norm([g, torch.zeros(9000, device="cuda")], 1e-3, nc)
    capi.muon_check()
    norm = float(ref.square().sum().sqrt())
    if norm > 3.4028235e38:
        assert math.isinf(float(nc[0]))
    else:
        assert abs(float(nc[0]) - norm) <= 18 * EPS * norm + 2.0 ** -149
    coef = min(1.0, 1e-3 / (norm + 1e-6))
    assert abs(float(nc[1]) - coef) <= 19 * EPS * coef + 2.0 ** -149


def test_large_next_to_small(capi):
    g = torch.full((100_000,), 1e-25, device="cuda")
    g[50_000] = 1e25
    nc = torch.empty(2, device="cuda")
    capi.muon_grad_norm([g], 1.0, nc)
    capi.muon_check()
    assert abs(float(nc[0]) - 1e25) <= 18 * EPS * 1e25 + 1e18


@pytest.mark.parametrize("value,norm,coef", [(float("nan"), "nan", "nan"), (float("inf"), "inf", 0.0),
                                             (float("-inf"), "inf", 0.0)])
def test_values_that_are_not_finite_show(capi, value, norm, coef):
    g = torch.ones(70_000, device="cuda")
    g[69_999] = value
    nc = torch.empty(2, device="cuda")
    capi.muon_grad_norm([g[:5], g], 1.0, nc)
    capi.muon_check()
    assert str(float(nc[0])) == norm
    assert str(float(nc[1])) == str(coef)


def test_in_place(capi):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    grads = [torch.randn(n, generator=gen, device="cuda") for n in (9, 100_000, 1)]
    orig = [g.clone() for g in grads]
    nc = torch.empty(2, device="cuda")
    capi.muon_clip_grads(grads, grads, 1e9, nc)
    assert float(nc[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(grads, orig))
    capi.muon_clip_grads(grads, grads, 0.5, nc)
    capi.muon_check()
    assert all(torch.equal(a, b * nc[1]) for a, b in zip(grads, orig))
    assert abs(_exact(grads, 1.0)[0] - 0.5) < 1e-5


def test_same_bits_every_run_and_on_another_stream(capi):
    g = [torch.randn(n, device="cuda") for n in (3_000_001, 77, 500_000)]
    ncs = [torch.empty(2, device="cuda") for _ in range(4)]
    side = torch.cuda.Stream()
    for nc in ncs[:3]:
        capi.muon_grad_norm(g, 1.0, nc)
    side.wait_stream(torch.cuda.current_stream())
    capi.muon_grad_norm(g, 1.0, ncs[3], stream=side)
    side.synchronize()
    capi.muon_check()
    assert all(torch.equal(nc, ncs[0]) for nc in ncs)


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "split"])
@pytest.mark.parametrize("n_shards", [1, 3])
def test_scaled_step_is_the_step_of_the_scaled_gradients(capi, dtype, n_shards):
    """Bit for bit: the coefficient is multiplied in before anything else."""
    wl = inputs.WORKLOADS["ragged_small"]
    W0, Gs, _ = inputs.host_inputs(wl)
    lay = capi.muon_layout_create(wl.shapes, n_shards, dtype, wl.is_matrix)
    ws = capi.workspace_tensor(lay)

    def shards(v):
        v = np.concatenate([v, np.zeros(lay.shard_len * n_shards - v.size, np.float32)])
        return [torch.from_numpy(s.copy()).cuda() for s in np.split(v, n_shards)]

    groups = [(wl.lr, wl.wd, wl.mu, wl.nesterov)]
    g = shards(Gs[0])
    nc = torch.empty(2, device="cuda")
    capi.muon_grad_norm(capi.layout_grads(lay, g), 0.1, nc)
    norm = math.sqrt(float((Gs[0].astype(np.float64) ** 2).sum()))
    assert abs(float(nc[0]) - norm) <= 18 * EPS * norm and float(nc[1]) < 1
    res = []
    for scaled in (True, False):
        w, m = shards(W0), shards(np.zeros_like(W0))
        for step in range(2):
            if scaled:
                capi.muon_step_scaled(w, g, m, lay, ws, groups, nc[1:], wl.ns_steps)
            else:
                capi.muon_step_grouped(w, [x * nc[1] for x in g], m, lay, ws, groups, wl.ns_steps)
        capi.muon_check()
        res.append((torch.cat(w), torch.cat(m)))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert torch.equal(torch.cat(g), torch.cat(shards(Gs[0])))


def test_binding_refuses(capi):
    g = torch.ones(16, device="cuda")
    nc = torch.empty(2, device="cuda")
    for grads, outs, norm in (([g], [], nc), ([g.cpu()], [g], nc), ([g.double()], [g], nc),
                              ([g[::2]], [g[:8]], nc), ([g], [g], nc[:1]), ([g], [g], nc.double())):
        with pytest.raises(ValueError):
            capi.muon_clip_grads(grads, outs, 1.0, norm)
    for outs, max_norm in (([g[:8]], 1.0), ([g.half()], 1.0), ([g], -1.0), ([g], float("nan")),
                           ([g], float("inf"))):
        with pytest.raises(capi.MuonError) as e:
            capi.muon_clip_grads([g], outs, max_norm, nc)
        assert e.value.status == capi.MUON_ERR_INVALID_ARG
    with pytest.raises(capi.MuonError):
        capi.muon_grad_norm([torch.ones(10 ** 6, device="cuda")], 1.0, nc,
                            workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    lay = capi.muon_layout_create([(8, 8)], 1, capi.MUON_NS_BF16)
    ws = capi.workspace_tensor(lay)
    w = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        capi.muon_step_scaled([w], [w], [w], lay, ws, [(0.1, 0.0, 0.9, True)], nc.cpu())
    with pytest.raises(ValueError):
        capi.muon_step_scaled([w], [w], [w], lay, ws, [], nc)
    capi.muon_check()
