"""The layer norm's gradient where its launch needs more shared memory than a kernel has by default: aligned
16-bit rows of 12232 values and more keep 4 bytes of weight for each, beside the block's statistics."""
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Both sides of 48 KB without and with the statistics, each length in a process whose kernels have not been
# allowed more by an earlier, longer one (lengths ascend, and every type and form is a kernel of its own).
FRESH = """
from muon_optimizer_step_gb300 import capi
from tests.test_gpu_layer_norm import _check_grad
for dtype in ("bf16", "fp16"):
    for sums in (True, False):
        for cols in (12224, 12232, 12256, 12288, 12296, 16384):
            _check_grad(capi, 20, cols, dtype, want_dw=sums, want_db=sums)
print("OK")
"""


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from muon_optimizer_step_gb300 import capi as c
    return c


def test_lengths_around_the_default_limit(capi):
    r = subprocess.run([sys.executable, "-c", FRESH], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout + r.stderr


def test_lengths_from_several_threads(capi):
    """Threads whose rows need different amounts call at the same time, as they may: none is refused."""
    jobs, refused = [], []
    for i, cols in enumerate((16384, 12800, 14336, 16384)):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        x, dy = (torch.randn(1, cols, generator=gen, device="cuda").bfloat16() for _ in range(2))
        mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
        dx, want = torch.empty_like(x), torch.empty_like(x)
        capi.muon_layer_norm_grad(dy, x, None, mean, rstd, want, None, None)
        stream = torch.cuda.Stream()
        args = (dy.data_ptr(), cols, x.data_ptr(), cols, None, mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), cols,
                None, None, 1, cols, 0, capi.MUON_DTYPE_BF16, None, 0, stream.cuda_stream)
        jobs.append((args, stream, dx, want, (x, dy, mean, rstd)))

    def run(args, stream):
        # (Straight into the library: what the binding does in between leaves too little to meet in.)
        for i in range(10_000):
            st = capi.lib.muon_layer_norm_grad(*args)
            if st != capi.MUON_OK:
                refused.append((args[2], st))
            if i % 500 == 499:
                stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=j[:2]) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, f"{len(refused)} calls refused"
    for _, _, dx, want, _ in jobs:
        assert torch.equal(dx, want)
