"""Infinities in the feed-forward operators, as include/bsg.h states them:
what the formulas give in floating point, and nothing beside the rows and
columns that hold them.  Sizes: few tokens, and tiles."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import ffn_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DEV, INF, NAN = "cuda", float("inf"), float("nan")
# act at +inf and -inf
LIMITS = {"silu": (INF, NAN), "gelu_tanh": (INF, NAN), "relu": (INF, 0.0)}


def ws(op, m, n, k):
    return torch.full((bsg.workspace_bytes(op, m, n, k),), 255, dtype=torch.uint8, device=DEV)


def same(y, want):
    """Equal, with NaN where NaN is wanted."""
    return torch.equal(torch.nan_to_num(y.float(), nan=12345.0), torch.nan_to_num(want.float(), nan=12345.0))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("m", [1, 20, 40, 300])
@pytest.mark.parametrize("kind", R.ACTS)
def test_infinite_gates(kind, m, dt):
    print("infinite gates", kind, m, dt, flush=True)
    n, k = 136, 264
    g = torch.Generator(device=DEV).manual_seed(m)
    x = torch.randint(1, 4, (m, k), generator=g, device=DEV).to(dt)
    wg, wu = (torch.randint(-2, 3, (n, k), generator=g, device=DEV).to(dt) for _ in range(2))
    base = [torch.empty(m, n, dtype=dt, device=DEV) for _ in range(3)]
    bsg.gemm_glu(x, wg, wu, *base, m, n, k, act=kind, workspace=ws("gemm_glu", m, n, k))
    wg[5, 3], wg[77, 200] = INF, -INF                # x > 0: columns 5 and 77 of G are infinite
    out = [torch.empty(m, n, dtype=dt, device=DEV) for _ in range(3)]
    bsg.gemm_glu(x, wg, wu, *out, m, n, k, act=kind, workspace=ws("gemm_glu", m, n, k))
    h, gate, u = out
    for col, limit, value in ((5, LIMITS[kind][0], INF), (77, LIMITS[kind][1], -INF)):
        assert bool((gate[:, col] == value).all())
        assert same(h[:, col], u[:, col].float() * limit)
    keep = [j for j in range(n) if j not in (5, 77)]
    for y, b in zip(out, base):
        assert torch.equal(y[:, keep], b[:, keep])
    assert torch.equal(u, base[2])
    # the same from integers, whose scales are infinite
    a, qg, qu = x.to(torch.int8)[:, :256].contiguous(), torch.ones(n, 256, dtype=torch.int8, device=DEV), \
        torch.randint(-2, 3, (n, 256), generator=g, device=DEV).to(torch.int8)
    qg[77] = -1
    one, sg = torch.ones(max(m, n), device=DEV), torch.ones(n, device=DEV)
    sg[5] = sg[77] = INF
    h = torch.empty(m, n, dtype=dt, device=DEV)
    bsg.gemm_glu_i8(a, qg, qu, one[:m], sg, one[:n], h, m, n, 256, act=kind, workspace=ws("gemm_glu_i8", m, n, 256))
    u = a.double() @ qu.double().t()
    assert same(h[:, 5], u[:, 5] * LIMITS[kind][0]) and same(h[:, 77], u[:, 77] * LIMITS[kind][1])
    # (gates of 256 to 768, whose act is the gate itself: products past fp16's 65504 round to infinity)
    gate = a.double().sum(1, keepdim=True)
    assert torch.equal(h[:, keep], (gate * u[:, keep]).float().to(dt))


@pytest.mark.parametrize("m", [1, 40, 300])
def test_infinite_scale_of_a_token(m):
    """gemm_i8: the token's row is infinite or, where its sum is 0, NaN."""
    print("infinite token scale", m, flush=True)
    n, k = 136, 272
    g = torch.Generator(device=DEV).manual_seed(m)
    a, b = (torch.randint(-3, 4, (r, k), generator=g, device=DEV).to(torch.int8) for r in (m, n))
    b[7] = 0
    sa, sb = torch.ones(m, device=DEV), torch.ones(n, device=DEV)
    sa[m - 1] = INF
    c = torch.empty(m, n, device=DEV)
    bsg.gemm_i8(a, b, sa, sb, None, c, m, n, k, workspace=ws("gemm_i8", m, n, k))
    s = (a.double() @ b.double().t()).float()
    assert same(c, s * sa[:, None])


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("m,n,k", [(3, 8, 16), (130, 264, 136), (300, 520, 264)])
@pytest.mark.parametrize("kind", R.ACTS)
def test_infinities_in_the_backward_pass(kind, m, n, k, dt):
    """An infinite gate: ReLU's derivative is 1 or 0 there, the others' NaN.
    An infinite dH or U: an infinite or NaN dG.  Each spoils its own row of dX
    and its own row of the weight gradients."""
    print("infinities backward", kind, (m, n, k), dt, flush=True)
    g = torch.Generator(device=DEV).manual_seed(m)
    rnd = lambda r, c: torch.randint(1, 4, (r, c), generator=g, device=DEV).to(dt) / 8       # noqa: E731
    dh, gate, u, x, wg, wu = rnd(m, n), rnd(m, n), rnd(m, n), rnd(m, k), rnd(n, k), rnd(n, k)

    def run(dh, gate, u):
        out = [torch.empty(r, k, dtype=dt, device=DEV) for r in (m, n, n)]
        bsg.gemm_glu_bwd(dh, x, wg, wu, gate, u, *out, m, n, k, act=kind, workspace=ws("gemm_glu_bwd", m, n, k))
        return out

    base = run(dh, gate, u)
    row, col = m // 2, n // 2
    # (input, value) -> the values of dG and dU there, from act and act' at +-inf
    a, b, both = LIMITS[kind][0], LIMITS[kind][1], (1.0, 0.0) if kind == "relu" else (NAN, NAN)
    h0, u0, act0 = float(dh[row, col]), float(u[row, col]), R.act64(gate[row, col].double(), kind)
    cases = [("gate", INF, h0 * u0 * both[0], h0 * a), ("gate", -INF, h0 * u0 * both[1], h0 * b),
             ("u", INF, INF * float(act0[1]), None), ("dh", -INF, -INF * u0 * float(act0[1]), -INF * float(act0[0]))]
    for name, value, dg, du in cases:
        t = dict(dh=dh.clone(), gate=gate.clone(), u=u.clone())
        t[name][row, col] = value
        dx, dwg, dwu = run(**t)
        for y, d, base_y in ((dwg, dg, base[1]), (dwu, du, base[2])):
            if d is None:
                assert torch.equal(y, base_y)
            elif d in (INF, -INF) or d != d:
                assert same(y[col], torch.full_like(y[col], d)), (name, value)     # x > 0
            keep = [j for j in range(n) if j != col]
            assert torch.equal(y[keep], base_y[keep]), (name, value)
        bad = [d for d in (dg, du) if d is not None and (d != d or abs(d) == INF)]
        if bad:
            total = sum(bad)
            assert same(dx[row], torch.full_like(dx[row], total)), (name, value)     # weights > 0
        keep = [i for i in range(m) if i != row]
        assert torch.equal(dx[keep], base[0][keep]), (name, value)
