"""The expert-layer example, as a user runs it: the gradients of a whole layer against automatic
differentiation in 64 bits, and losses that fall.

The bound on the gradients: activations and their gradients are stored in bfloat16 (2^-9 of
each value in the root mean square at most), and no gradient passes more than five such
stores on its way (rows' products, activation, its gradient, dy, dx): 5 * 2^-9 < 1e-2."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("sizes", [[], ["--tokens", "257", "--hidden", "136", "--inner", "88",
                                        "--experts", "7", "--top", "3"],
                                   ["--tokens", "1", "--hidden", "64", "--inner", "72", "--experts",
                                    "5", "--top", "2"]])
def test_gradients_and_falling_losses(sizes):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import expert_layer_step
    finally:
        sys.path.pop(0)
    losses, worst = expert_layer_step.main([*sizes, "--steps", "6", "--check"])
    assert worst <= 1e-2
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_command_line():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_layer_step.py"),
                        "--steps", "2", "--tokens", "64"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "step 1: loss" in r.stdout, r.stdout + r.stderr
