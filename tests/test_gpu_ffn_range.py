"""The ends of the types' range in the feed-forward operators, as
include/bsg.h states them."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import ffn_ref as R

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
DEV = "cuda"


def backward(m, n, k, dt, dh, u, w=2.0 ** -7, x=1.0):
    """Gradients of a ReLU block with G = 1 (act = act' = 1) and constant
    tensors: dG = dh u, dU = dh everywhere."""
    full = lambda rows, cols, v: torch.full((rows, cols), v, dtype=dt, device=DEV)      # noqa: E731
    t = full(m, n, dh), full(m, k, x), full(n, k, w), full(n, k, w), full(m, n, 1.0), full(m, n, u)
    out = [full(m, k, 77.0), full(n, k, 77.0), full(n, k, 77.0)]
    ws = torch.full((bsg.workspace_bytes("gemm_glu_bwd", m, n, k),), 255, dtype=torch.uint8, device=DEV)
    bsg.gemm_glu_bwd(*t, *out, m, n, k, act="relu", workspace=ws)
    for what, y, (ref, err) in zip(("dx", "dwg", "dwu"), out, R.glu_bwd64(*t, "relu", dt)):
        yield what, y, ref, err


@pytest.mark.parametrize("m,n,k", [(3, 8, 16), (70, 264, 136), (300, 520, 264)])
def test_fp16_backward_at_the_top(m, n, k):
    print("fp16 backward at the top", m, n, k, flush=True)
    # dG = 250 * 256 = 64000 is a value of fp16 (4 m of them make a weight gradient of less than 65504: x = 2^-9)
    for what, y, ref, err in backward(m, n, k, HF, 250.0, 256.0, w=2.0 ** -10, x=2.0 ** -9):
        assert bool(torch.isfinite(y).all()), what
        R.check(what, y, ref, err, HF)
    # dG = 300 * 300 is not: dX and dWg are infinite, dWu, which dG does not enter, is right
    for what, y, ref, err in backward(m, n, k, HF, 300.0, 300.0, w=2.0 ** -10, x=2.0 ** -9):
        if what == "dwu":
            R.check(what, y, ref, err, HF)
        else:
            assert bool((ref.abs() < 65504).all()) and bool(torch.isinf(y).all()), what
    # a power of two off dH, and back on the outputs, has it
    for what, y, ref, err in backward(m, n, k, HF, 300.0 / 4, 300.0, w=2.0 ** -10, x=2.0 ** -9):
        R.check(what, y, ref, err, HF)
    for what, y, ref, err in backward(m, n, k, BF, 300.0, 300.0):
        R.check(what, y, ref, err, BF)


@pytest.mark.parametrize("m,n,k", [(3, 8, 16), (70, 264, 136), (300, 520, 264)])
def test_fp16_backward_at_the_bottom(m, n, k):
    print("fp16 backward at the bottom", m, n, k, flush=True)
    # dG = 2^-24, the smallest value of fp16, is kept, and its sums are exact
    for what, y, ref, err in backward(m, n, k, HF, 2.0 ** -12, 2.0 ** -12, w=1.0, x=1.0):
        assert torch.equal(y, ref.to(HF)), what
    # dG = 2^-26 is 0: dWg is lost, dX has dU's part alone
    for what, y, ref, err in backward(m, n, k, HF, 2.0 ** -13, 2.0 ** -13, w=1.0, x=1.0):
        want = {"dx": n * 2.0 ** -13, "dwg": 0.0, "dwu": m * 2.0 ** -13}[what]
        assert torch.equal(y, torch.full_like(y, want)), what
    # scaled by 2^10 it is there
    for what, y, ref, err in backward(m, n, k, HF, 2.0 ** -3, 2.0 ** -13, w=1.0, x=1.0):
        assert torch.equal(y, ref.to(HF)), what
    for what, y, ref, err in backward(m, n, k, BF, 2.0 ** -13, 2.0 ** -13):
        R.check(what, y, ref, err, BF)
