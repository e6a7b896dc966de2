"""The feed-forward example runs the operators together: training lowers its
loss, and the block served from 8-bit integers stays near the bf16 one."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_example_trains_and_serves():
    print("examples/feed_forward.py", flush=True)
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, errors = mod.main(["--tokens", "256", "--model", "512", "--hidden", "1408", "--steps", "10"])
    assert losses[-1] < 0.9 * losses[0]
    # codes of normal rows: a step is about 4 sigma / 127, its rounding error
    # 4 / 127 / sqrt(12) = 0.9% of the row, on both operands of both products:
    # 0.9% * sqrt(4) = 1.8%, plus bf16; the product of gate and up doubles it at most
    assert all(e < 0.04 for e in errors.values()), errors
