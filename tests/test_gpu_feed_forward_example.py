"""The feed-forward example, as a user runs it: the gradients of a whole layer against automatic
differentiation in 64 bits, and its 8-bit forward pass.

The bound on the gradients: activations and their gradients are stored in bfloat16 (2^-9 of each value
in the root mean square at most), and no gradient passes more than five such stores on its way (the norm,
the activation, dy, its gradient, dn): 5 * 2^-9 < 1e-2.

The bound on the 8-bit pass: a value is off by at most half a step of e4m3, 2^-4 of it; uniformly
distributed over a step of 2^-3 at most, by 2^-3 / sqrt(12) = 0.036 in the root mean square.  A product
of two such factors is off by sqrt(2) of that, 0.051, in the root mean square of a sum of independent terms;
silu(g) u takes two such products (slopes of 1.1 at most: 0.079), and the second product adds its own two
roundings: sqrt(0.079^2 + 0.051^2) = 0.094, with the bf16 stores below 0.1."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("sizes", [[], ["--tokens", "257", "--hidden", "136", "--inner", "200"],
                                   ["--tokens", "1", "--hidden", "64", "--inner", "72"],
                                   ["--tokens", "300", "--hidden", "77", "--inner", "131"]])
def test_gradients_and_fp8(sizes):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import feed_forward_step
    finally:
        sys.path.pop(0)
    worst, off = feed_forward_step.main([*sizes, "--steps", "3", "--check", "--fp8"])
    assert worst <= 1e-2 and off <= 0.1


def test_command_line():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "feed_forward_step.py"),
                        "--steps", "2", "--tokens", "64", "--fp8"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "step 1: loss" in r.stdout, r.stdout + r.stderr
