"""CPU tests of the feed-forward operators: the host-side checks of
arguments, the workspace sizes, and the 64-bit gradients against differences
(the formula the GPU tests compare the kernels with)."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import ffn_ref as R

OK, NULLPTR, SHAPE, DTYPE, ALIGN, UNSUP = 0, 1, 2, 3, 4, 5
P = 0x10000   # a 16-byte aligned fake device address (validation never dereferences)
BIG = 1 << 40


def q(**kw):
    return bsg.quant_i8(**{**dict(x=P, q=P, scale=P, m=5, k=64, x_dtype=torch.bfloat16), **kw}, validate_only=True)


def i8(**kw):
    base = dict(a=P, b=P, a_scale=P, b_scale=P, bias=P, c=P, m=5, n=64, k=64, bias_dtype=torch.float32,
                c_dtype=torch.bfloat16, workspace=P)
    return bsg.gemm_i8(**{**base, **kw}, validate_only=True)


def glu(**kw):
    base = dict(x=P, w_gate=P, w_up=P, h=P, g=P, u=P, m=5, n=64, k=64, dtype=torch.bfloat16, workspace=P)
    return bsg.gemm_glu(**{**base, **kw}, validate_only=True)


def glu_i8(**kw):
    base = dict(a=P, w_gate=P, w_up=P, a_scale=P, gate_scale=P, up_scale=P, h=P, m=5, n=64, k=64,
                h_dtype=torch.float16, workspace=P)
    return bsg.gemm_glu_i8(**{**base, **kw}, validate_only=True)


def bwd(**kw):
    base = dict(dh=P, x=P, w_gate=P, w_up=P, g=P, u=P, dx=P, dw_gate=P, dw_up=P, m=5, n=64, k=64,
                dtype=torch.float16, workspace=P)
    return bsg.gemm_glu_bwd(**{**base, **kw}, validate_only=True)


def test_quant_i8_validation():
    assert q() == OK and q(x_dtype=torch.float32) == OK and q(m=0, x=0, q=0, scale=0) == OK
    assert q(k=0, x=0, q=0) == OK                         # scales of empty rows are written
    assert q(k=40) == ALIGN and q(x=P + 8) == ALIGN and q(q=P + 4) == ALIGN and q(scale=P + 2) == ALIGN
    assert q(x=0) == NULLPTR and q(scale=0) == NULLPTR
    assert q(m=-1) == SHAPE and q(m=1 << 23) == UNSUP and q(k=1 << 21) == UNSUP
    assert q(x_dtype=bsg.E4M3) == DTYPE


def test_gemm_i8_validation():
    assert i8() == OK and i8(bias=None) == OK and i8(m=0) == OK and i8(k=0, a=0, b=0) == OK
    assert i8(k=24) == ALIGN and i8(n=12) == ALIGN and i8(n=12, c_dtype=torch.float32) == OK
    assert i8(n=10, c_dtype=torch.float32) == ALIGN
    assert i8(a=P + 8) == ALIGN and i8(a_scale=P + 2) == ALIGN and i8(bias=P + 2) == ALIGN
    assert i8(bias=P + 2, bias_dtype=torch.float16) == OK
    assert i8(a=0) == NULLPTR and i8(b_scale=0) == NULLPTR and i8(c=0) == NULLPTR
    assert i8(c_dtype=bsg.E4M3) == DTYPE and i8(bias_dtype=bsg.E4M3) == DTYPE
    assert i8(k=131056) == OK and i8(k=131072) == UNSUP   # int32 sums
    assert i8(n=-8) == SHAPE and i8(n=1 << 21) == UNSUP and i8(m=1 << 22, n=1 << 20) == UNSUP


def test_gemm_glu_validation():
    assert glu() == OK and glu(g=None, u=None) == OK and glu(m=0, x=0, h=0) == OK
    assert glu(g=None) == NULLPTR and glu(u=None) == NULLPTR and glu(w_up=0) == NULLPTR
    assert glu(n=12) == ALIGN and glu(k=12) == ALIGN and glu(h=P + 8) == ALIGN and glu(u=P + 2) == ALIGN
    assert glu(dtype=torch.float32) == DTYPE
    assert glu(m=-1) == SHAPE
    with pytest.raises(ValueError):
        glu(act="tanh")
    assert bsg.lib().bsg_validate_gemm_glu(P, P, P, P, P, P, P, BIG, 5, 64, 64, bsg.BF16, 3) == SHAPE


def test_gemm_glu_i8_validation():
    assert glu_i8() == OK and glu_i8(m=0) == OK
    assert glu_i8(k=24) == ALIGN and glu_i8(n=12) == ALIGN and glu_i8(up_scale=P + 1) == ALIGN
    assert glu_i8(gate_scale=0) == NULLPTR and glu_i8(a=0) == NULLPTR
    assert glu_i8(h_dtype=torch.float32) == DTYPE and glu_i8(k=131072) == UNSUP


def test_gemm_glu_bwd_validation():
    assert bwd() == OK
    assert bwd(dx=None, w_gate=None, w_up=None) == OK                 # frozen input
    assert bwd(dw_gate=None, dw_up=None, x=None) == OK                # frozen weights
    assert bwd(dw_gate=None) == NULLPTR and bwd(g=None) == NULLPTR and bwd(x=None) == NULLPTR
    assert bwd(w_up=None) == NULLPTR
    assert bwd(m=0, dh=0, g=0, u=0, x=0) == OK                        # dw of no tokens is zero
    assert bwd(k=12) == ALIGN and bwd(dh=P + 8) == ALIGN and bwd(dw_up=P + 8) == ALIGN
    assert bwd(dtype=bsg.F32) == DTYPE and bwd(n=-8) == SHAPE
    assert bwd(workspace=None) == NULLPTR
    L = bsg.lib()
    need = bsg.workspace_bytes("gemm_glu_bwd", 5, 64, 64)
    assert need >= 4 * 5 * 64                                         # dG and dU
    args = [P] * 10
    assert L.bsg_validate_gemm_glu_bwd(*args, need, 5, 64, 64, bsg.BF16, 0) == OK
    assert L.bsg_validate_gemm_glu_bwd(*args, need - 1, 5, 64, 64, bsg.BF16, 0) == SHAPE
    assert L.bsg_validate_gemm_glu_bwd(*args[:-1], P + 8, need, 5, 64, 64, bsg.BF16, 0) == ALIGN


def test_grids_past_the_launch_limit_are_refused():
    """2^32 threads or 2^23 tiles: every product of sizes, and the backward's
    element-wise pass over (m, n) where both of its products are small."""
    m, n = 1 << 22, 1 << 20
    assert i8(m=m, n=n) == UNSUP and glu(m=m, n=n) == UNSUP and glu_i8(m=m, n=n) == UNSUP
    assert bwd(m=m, n=n, k=8) == UNSUP and bwd(m=m, n=8, k=1 << 20) == UNSUP and bwd(m=8, n=n, k=1 << 20) == UNSUP
    assert bwd(m=m, n=8 * 64, k=8) == OK


def test_workspace_bytes():
    for name in ("gemm_i8", "gemm_glu", "gemm_glu_i8", "gemm_glu_bwd"):
        assert bsg.workspace_bytes(name, 0, 0, 0) >= 0
        assert bsg.workspace_bytes(name, 1 << 22, 1 << 20, 1 << 20) < 1 << 45
        with pytest.raises(bsg.BsgError):
            bsg.workspace_bytes(name, -1, 8, 8)
    assert bsg.workspace_bytes("quant_i8", 4, 4, 4) == 0
    with pytest.raises(ValueError):
        bsg.workspace_bytes("gemm", 1, 1, 1)
    assert bsg.lib().bsg_workspace_bytes(9, 1, 1, 1) == -1


@pytest.mark.parametrize("kind", R.ACTS)
def test_reference_gradients_match_differences(kind):
    """Central differences of sum(dh * h) in float64: the step 1e-5 leaves
    about 1e-10 of curvature and 1e-11 of rounding."""
    gen = torch.Generator().manual_seed(3)
    m, n, k = 5, 8, 16
    x, wg, wu, dh = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((m, k), (n, k), (n, k), (m, n)))

    def loss(x, wg, wu):
        return float((dh * R.act64(x @ wg.t(), kind)[0] * (x @ wu.t())).sum())

    got = R.glu_bwd64(dh, x, wg, wu, x @ wg.t(), x @ wu.t(), kind, torch.float32)
    for t, (ref, _) in zip((x, wg, wu), got):
        for i, j in ((0, 0), (t.shape[0] - 1, 3), (2, t.shape[1] - 1)):
            v = float(t[i, j])
            t[i, j] = v + 1e-5
            hi = loss(x, wg, wu)
            t[i, j] = v - 1e-5
            lo = loss(x, wg, wu)
            t[i, j] = v
            assert abs((hi - lo) / 2e-5 - float(ref[i, j])) < 1e-7 * (1 + abs(float(ref[i, j])))


@pytest.mark.parametrize("kind", R.ACTS)
def test_reference_activation_is_torch(kind):
    g = torch.linspace(-12, 12, 2001, dtype=torch.float64)
    f = {"silu": torch.nn.functional.silu, "relu": torch.relu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[kind]
    torch.testing.assert_close(R.act64(g, kind)[0], f(g), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_rounding_constants_are_the_types(dt):
    """ROUND and STEP are what torch's own casts do at worst: reached just
    past a power of two, and at half the smallest step."""
    u, s = R.ROUND[dt], R.STEP[dt]
    worst = torch.tensor(1 + u, dtype=torch.float64)            # a tie: goes to the even 1
    assert worst.to(dt).double() == 1 and torch.tensor(1 + 1.001 * u, dtype=torch.float64).to(dt).double() == 1 + 2 * u
    v = torch.rand(1 << 16, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) + 1
    assert bool(((v.to(dt).double() - v).abs() <= u * v).all())
    assert torch.tensor(3 * s, dtype=torch.float64).to(dt).double() == 4 * s
