"""The layer norm's gradient where its launch needs more shared memory than a kernel has by default: aligned
16-bit rows of 12232 values and more keep 4 bytes of weight for each, beside the block's statistics."""
import os
import subprocess
import sys

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
