"""The feed-forward operators against their 64-bit definitions (ffn_ref.py
derives the bounds), on the sizes and values where they can go wrong."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import ffn_ref as R

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda"


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rnd(g, *shape, dt=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dt)


def ints(g, *shape, lo=-127, hi=127, dt=torch.int8):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32).to(dt)


def guarded(m, n, dt):
    """An (m, n) output inside a larger buffer of sentinels, and its check."""
    pad = 1024
    buf = torch.full((m * n + 2 * pad,), 77, dtype=dt, device=DEV)

    def intact():
        assert bool((buf[:pad] == 77).all()) and bool((buf[pad + m * n:] == 77).all()), "wrote past the output"

    return buf[pad:pad + m * n].view(m, n), intact


def scratch(name, m, n, k):
    """A workspace of the exact size, full of NaN bytes."""
    return torch.full((bsg.workspace_bytes(name, m, n, k),), 255, dtype=torch.uint8, device=DEV)


# (m, n, k): one token, odd token counts around every tile edge, ragged n and
# k, long k with few rows, k of one piece
SIZES = [(1, 8, 16), (1, 256, 4112), (3, 264, 528), (16, 136, 80), (17, 520, 1040), (33, 64, 4096), (63, 248, 272),
         (64, 256, 64), (65, 1032, 336), (127, 72, 144), (129, 392, 1056), (200, 2048, 32), (257, 640, 400),
         (300, 264, 2064), (513, 1288, 192), (700, 24, 6016), (1030, 520, 112),
         # K in parts (few tiles, long K), and the largest tiles
         (100, 264, 9008), (72, 1032, 4528), (2305, 4104, 80), (4100, 2056, 1040)]


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("m,k", [(1, 16), (3, 48), (5, 4096), (2, 7168), (64, 1040), (1, 20000), (4, 65536 + 16), (1000, 272)])
def test_quant_i8(m, k, dt):
    say("quant_i8", m, k, dt)
    g = gen(m + k)
    x = rnd(g, m, k) * torch.exp(4 * torch.rand(m, 1, generator=g, device=DEV))
    x = x.to(dt)
    if m > 2:
        x[0] = 0                                    # an empty row
        x[1] = 0
        x[1, k - 1] = -3.0                          # the maximum last, and negative
    q, okq = guarded(m, k, torch.int8)
    s, oks = guarded(m, 1, F32)
    bsg.quant_i8(x, q, s.view(-1), m, k)
    okq(), oks()
    # the definition's own fp32 steps: equal bit for bit
    top = x.float().abs().amax(1).clamp_min(2.0 ** -100)
    # (both divisions by tensors: torch multiplies by the reciprocal of a number)
    full = torch.full_like(top, 127.0)
    assert torch.equal(q, torch.round(x.float() * (full / top)[:, None]).to(torch.int8))
    assert torch.equal(s.view(-1), top / full)
    # and half a step (and fp32 rounding of the quotient) of x in 64 bits
    off = (q.double() * s.double() - x.double()).abs()
    assert bool((off <= s.double() * (0.5 + 127 * 2.0 ** -22)).all())


def test_quant_i8_special_rows():
    say("quant_i8 special rows")
    x = torch.ones(6, 64, device=DEV)
    x[0] = 0.0
    x[1] = 1e-35                                    # below 2^-100: codes 0
    x[2, 5] = float("inf")
    x[3, 60] = float("nan")
    x[4] = 3.0e38
    x[5] = -(2.0 ** -99)
    q = torch.full((6, 64), 9, dtype=torch.int8, device=DEV)
    s = torch.empty(6, device=DEV)
    bsg.quant_i8(x, q, s, 6, 64)
    assert bool((q[:4] == 0).all())
    assert s[0] == torch.tensor(2.0 ** -100 / 127, device=DEV) and s[1] == s[0] and torch.isinf(s[2]) and torch.isnan(s[3])
    assert bool((q[4] == 127).all()) and bool((q[5] == -127).all())
    assert bool(torch.isfinite(s[4]))


def test_quant_i8_no_columns_and_no_rows():
    say("quant_i8 empty")
    s = torch.zeros(3, device=DEV)
    bsg.quant_i8(torch.empty(3, 0, device=DEV), torch.empty(3, 0, dtype=torch.int8, device=DEV), s, 3, 0)
    assert bool((s == torch.tensor(2.0 ** -100 / 127, device=DEV)).all())
    bsg.quant_i8(torch.empty(0, 64, device=DEV), torch.empty(0, 64, dtype=torch.int8, device=DEV), s[:0], 0, 64)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
def run_i8(a, b, sa, sb, bias, dt, ws=None):
    (m, k), n = a.shape, b.shape[0]
    c, intact = guarded(m, n, dt)
    bsg.gemm_i8(a, b, sa, sb, bias, c, m, n, k, workspace=scratch("gemm_i8", m, n, k) if ws is None else ws)
    intact()
    return c


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_gemm_i8(i, size):
    m, n, k = size
    dt, bdt = [BF, HF, F32][i % 3], [F32, BF, HF, None][i % 4]
    say("gemm_i8", size, dt, bdt)
    g = gen(i)
    a, b = ints(g, m, k), ints(g, n, k)
    sa, sb = torch.rand(m, generator=g, device=DEV) * 0.01, torch.rand(n, generator=g, device=DEV) * 0.01
    bias = None if bdt is None else rnd(g, n, dt=bdt)
    ref, err = R.i8_64(a, b, sa, sb)
    if bias is not None:
        ref = ref + bias.double()
        err = err + R.E * (ref.abs() + err)
    R.check("c", run_i8(a, b, sa, sb, bias, dt), ref, err, dt)


@pytest.mark.parametrize("m,n,k", [(1, 64, 131056), (40, 264, 16384), (300, 520, 8192)])
def test_gemm_i8_sums_are_exact(m, n, k):
    """Codes of -128 everywhere: the largest sum an int32 holds at this K, and
    nowhere a rounding but the conversion's."""
    say("gemm_i8 exact", m, n, k)
    a = torch.full((m, k), -128, dtype=torch.int8, device=DEV)
    b = torch.full((n, k), -128, dtype=torch.int8, device=DEV)
    b[::2, 0] = 127                                # even columns: 255 * 128 less
    one = torch.ones(max(m, n), device=DEV)
    c = run_i8(a, b, one[:m], one[:n], None, F32)
    want = torch.full((n,), 16384.0 * k, dtype=torch.float64)
    want[::2] -= 255 * 128
    assert torch.equal(c.cpu(), want.float().expand(m, n))


@pytest.mark.parametrize("m", [1, 20, 300])
def test_gemm_i8_empty_sum_and_nonfinite_scale(m):
    say("gemm_i8 k = 0, scales", m)
    bias = torch.arange(16, device=DEV, dtype=F32)
    e = torch.empty(m, 0, dtype=torch.int8, device=DEV)
    one = torch.ones(max(m, 16), device=DEV)
    c = run_i8(e, e.new_empty(16, 0), one[:m], one[:16], bias, F32)
    assert torch.equal(c, bias.expand(m, 16))
    # a token whose scale is NaN spoils its own row only
    g = gen(1)
    a, b = ints(g, m, 64), ints(g, 16, 64)
    sa = one[:m].clone()
    sa[m - 1] = float("nan")
    c = run_i8(a, b, sa, one[:16], None, BF)
    assert bool(torch.isnan(c[m - 1]).all()) and bool(torch.isfinite(c[:m - 1]).all())


# ---------------------------------------------------------------------------
def run_glu(x, wg, wu, kind, save):
    (m, k), n, dt = x.shape, wg.shape[0], x.dtype
    outs = [guarded(m, n, dt) for _ in range(3 if save else 1)]
    t = [o for o, _ in outs] + [None] * (0 if save else 2)
    bsg.gemm_glu(x, wg, wu, *t, m, n, k, act=kind, workspace=scratch("gemm_glu", m, n, k))
    for _, intact in outs:
        intact()
    return t


@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_gemm_glu(i, size):
    m, n, k = size
    dt, kind = [BF, HF][i % 2], R.ACTS[i % 3]
    say("gemm_glu", size, dt, kind)
    g = gen(100 + i)
    x, wg, wu = rnd(g, m, k, dt=dt), rnd(g, n, k, dt=dt, std=2 * k ** -0.5), rnd(g, n, k, dt=dt, std=k ** -0.5)
    h, eh, gr, ur, eg, eu = R.glu64(x, wg, wu, kind)
    for save in (True, False):
        t = run_glu(x, wg, wu, kind, save)
        R.check("h", t[0], h, eh, dt)
        if save:
            R.check("g", t[1], gr, eg, dt)
            R.check("u", t[2], ur, eu, dt)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("m,n,k", [(1, 520, 1032), (15, 264, 520), (40, 72, 264), (70, 136, 4104), (131, 1032, 200),
                                   (600, 392, 1000), (2500, 4104, 264)])
def test_gemm_glu_small_integers_are_exact(m, n, k, dt):
    """Small integers: every fp32 sum is exact in any order, so G, U and
    ReLU(G) * U are the 64-bit values rounded once.  A column or a piece of K
    read twice, or not at all, shows."""
    say("gemm_glu exact", m, n, k, dt)
    g = gen(k)
    x, wg, wu = (ints(g, r, k, lo=-2, hi=2, dt=dt) for r in (m, n, n))
    h, gg, uu = run_glu(x, wg, wu, "relu", True)
    gr, ur = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    assert torch.equal(gg, gr.to(dt)) and torch.equal(uu, ur.to(dt))
    assert torch.equal(h.double(), (gr.clamp(min=0) * ur).float().to(dt).double())


@pytest.mark.parametrize("m", [2, 80, 400])
@pytest.mark.parametrize("kind", R.ACTS)
def test_gemm_glu_large_preactivations(kind, m):
    """Gates far out on both sides: the activation is 0 or the identity there,
    never NaN."""
    say("gemm_glu large gates", kind, m)
    n, k = 64, 64
    x = torch.zeros(m, k, dtype=BF, device=DEV)
    x[:, 0] = 1.0
    wg = torch.zeros(n, k, dtype=BF, device=DEV)
    vals = torch.tensor([0.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4, 1e30], device=DEV)
    wg[:, 0] = vals.repeat(n // 8)
    wu = torch.zeros_like(wg)
    wu[:, 0] = 1.0
    h, g, u = run_glu(x, wg, wu, kind, True)
    ref = R.act64(wg[:, 0].double(), kind)[0]
    ref[wg[:, 0] <= -100] = 0.0
    assert torch.equal(g[0], wg[:, 0]) and bool((u == 1).all())
    assert bool(((h.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-10).all())


def test_gemm_glu_nan_and_empty():
    say("gemm_glu NaN row, k = 0, m = 0")
    for m in (5, 300):
        g = gen(m)
        x, wg, wu = rnd(g, m, 64, dt=BF), rnd(g, 64, 64, dt=BF), rnd(g, 64, 64, dt=BF)
        x[3, 7] = float("nan")
        for kind in R.ACTS:
            h, _, _ = run_glu(x, wg, wu, kind, False)
            assert bool(torch.isnan(h[3]).all())
            keep = torch.arange(m, device=DEV) != 3
            assert bool(torch.isfinite(h[keep]).all())
    z = torch.empty(4, 0, dtype=BF, device=DEV)
    h, g, u = run_glu(z, z.new_empty(16, 0), z.new_empty(16, 0), "gelu_tanh", True)
    assert bool((h == 0).all()) and bool((g == 0).all()) and bool((u == 0).all())
    run_glu(torch.empty(0, 64, dtype=BF, device=DEV), wg, wu, "silu", False)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("i,size", list(enumerate(SIZES)))
def test_gemm_glu_i8(i, size):
    m, n, k = size
    dt, kind = [HF, BF][i % 2], R.ACTS[(i + 1) % 3]
    say("gemm_glu_i8", size, dt, kind)
    g = gen(200 + i)
    a, wg, wu = ints(g, m, k), ints(g, n, k), ints(g, n, k)
    # g and u of a few units: 127^2/3 is the mean square of a code
    sa = (0.5 + torch.rand(m, generator=g, device=DEV)) / 73
    sg, su = ((0.5 + torch.rand(n, generator=g, device=DEV)) * k ** -0.5 / 73 for _ in range(2))
    h, intact = guarded(m, n, dt)
    bsg.gemm_glu_i8(a, wg, wu, sa, sg, su, h, m, n, k, act=kind, workspace=scratch("gemm_glu_i8", m, n, k))
    intact()
    gr, eg = R.i8_64(a, wg, sa, sg)
    ur, eu = R.i8_64(a, wu, sa, su)
    ref, err = R._gate(gr, ur, eg, eu, kind)
    R.check("h", h, ref, err, dt)


# ---------------------------------------------------------------------------
BWD = [(1, 8, 8), (7, 64, 24), (64, 72, 136), (129, 264, 200), (200, 520, 64), (257, 136, 1032), (515, 1288, 264),
       (1000, 256, 520), (2050, 40, 72),
       # dX with K in parts, the weight gradients with K in parts, the largest tiles for either
       (100, 4504, 264), (9000, 136, 264), (4100, 520, 4104), (200, 4104, 2056)]


def run_bwd(dh, x, wg, wu, g, u, kind, want=(True, True)):
    (m, n), k, dt = g.shape, wg.shape[1], dh.dtype
    dx, okx = guarded(m, k, dt)
    dg, okg = guarded(n, k, dt)
    du, oku = guarded(n, k, dt)
    bsg.gemm_glu_bwd(dh, x if want[1] else None, wg, wu, g, u, dx if want[0] else None, dg if want[1] else None,
                     du if want[1] else None, m, n, k, act=kind, workspace=scratch("gemm_glu_bwd", m, n, k))
    okx(), okg(), oku()
    return dx, dg, du


def bwd_inputs(seed, m, n, k, dt):
    g = gen(seed)
    return (rnd(g, m, n, dt=dt), rnd(g, m, k, dt=dt), rnd(g, n, k, dt=dt, std=k ** -0.5),
            rnd(g, n, k, dt=dt, std=k ** -0.5), rnd(g, m, n, dt=dt, std=2.0), rnd(g, m, n, dt=dt))


@pytest.mark.parametrize("i,size", list(enumerate(BWD)))
def test_gemm_glu_bwd(i, size):
    m, n, k = size
    for dt in (BF, HF):
        kind = R.ACTS[(i + (dt == HF)) % 3]
        say("gemm_glu_bwd", size, dt, kind)
        t = bwd_inputs(300 + i, m, n, k, dt)
        ref = R.glu_bwd64(*t, kind, dt)
        got = run_bwd(*t, kind)
        for name, y, (r, e) in zip(("dx", "dwg", "dwu"), got, ref):
            R.check(name, y, r, e, dt)
        # the gradients that are asked for alone are the same ones
        only_x = run_bwd(*t, kind, (True, False))
        only_w = run_bwd(*t, kind, (False, True))
        assert torch.equal(only_x[0], got[0]) and bool((only_x[1] == 77).all()) and bool((only_x[2] == 77).all())
        assert torch.equal(only_w[1], got[1]) and torch.equal(only_w[2], got[2]) and bool((only_w[0] == 77).all())


@pytest.mark.parametrize("m,n,k", [(40, 136, 264), (300, 264, 520), (1001, 72, 136), (4099, 264, 4104)])
def test_gemm_glu_bwd_small_integers_are_exact(m, n, k):
    """ReLU, small integers: dG, dU and every sum are exact."""
    say("gemm_glu_bwd exact", m, n, k)
    g = gen(n)
    dh, x, wg, wu, gg, uu = (ints(g, *s, lo=-2, hi=2, dt=BF) for s in ((m, n), (m, k), (n, k), (n, k), (m, n), (m, n)))
    dx, dwg, dwu = run_bwd(dh, x, wg, wu, gg, uu, "relu")
    on = (gg > 0).double()
    dg, du = dh.double() * uu.double() * on, dh.double() * gg.double() * on
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).to(BF))
    assert torch.equal(dwg, (dg.t() @ x.double()).to(BF)) and torch.equal(dwu, (du.t() @ x.double()).to(BF))


@pytest.mark.parametrize("m,n,k", [(1001, 2120, 520), (2900, 712, 208)])
def test_products_of_many_middle_tiles(m, n, k):
    """More than 256 tiles of 128 x 128 with ragged edges, where two workgroups
    share a compute unit: exact sums of small integers in every operator."""
    say("many middle tiles", m, n, k)
    g = gen(n)
    a, b = ints(g, m, 2 * k, lo=-2, hi=2), ints(g, 2 * n, 2 * k, lo=-2, hi=2)
    one = torch.ones(max(m, 2 * n), device=DEV)
    assert torch.equal(run_i8(a, b, one[:m], one[:2 * n], None, F32), (a.double() @ b.double().t()).float())
    h, intact = guarded(m, n, BF)
    bsg.gemm_glu_i8(a, b[:n], b[n:], one[:m], one[:n], one[:n], h, m, n, 2 * k, act="relu",
                    workspace=scratch("gemm_glu_i8", m, n, 2 * k))
    intact()
    gr, ur = a.double() @ b[:n].double().t(), a.double() @ b[n:].double().t()
    assert torch.equal(h, (gr.clamp(min=0) * ur).float().to(BF))
    for dt in (BF, HF):
        x, wg, wu = a[:, :k].to(dt).contiguous(), b[:n, :k].to(dt).contiguous(), b[n:, :k].to(dt).contiguous()
        gr, ur = x.double() @ wg.double().t(), x.double() @ wu.double().t()
        t = run_glu(x, wg, wu, "relu", True)
        assert torch.equal(t[1], gr.to(dt)) and torch.equal(t[2], ur.to(dt))
        assert torch.equal(t[0].double(), (gr.clamp(min=0) * ur).float().to(dt).double())


@pytest.mark.parametrize("m,n,k", [(1001, 1416, 2056)])
def test_gemm_glu_bwd_of_many_middle_tiles(m, n, k):
    """The gradients on the same tiles, in one launch: ReLU and small integers,
    so that every sum is exact."""
    say("bwd many middle tiles", m, n, k)
    g = gen(n)
    for dt in (BF, HF):
        dh, x, wg, wu, gg, uu = (ints(g, *s, lo=-2, hi=2, dt=dt) for s in ((m, n), (m, k), (n, k), (n, k), (m, n), (m, n)))
        dx, dwg, dwu = run_bwd(dh, x, wg, wu, gg, uu, "relu")
        on = (gg > 0).double()
        dg, du = dh.double() * uu.double() * on, dh.double() * gg.double() * on
        assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).to(dt))
        assert torch.equal(dwg, (dg.t() @ x.double()).to(dt)) and torch.equal(dwu, (du.t() @ x.double()).to(dt))


@pytest.mark.parametrize("kind", R.ACTS)
def test_gemm_glu_bwd_matches_differences(kind):
    """dX and dWg, dWu against central differences of sum(dH * H) in 64 bits.
    The saved G and U are the forward kernel's, rounded: act and act' move by
    at most 1.6 r |G|, which the bound adds (r = 2^-11, fp16)."""
    say("gemm_glu_bwd differences", kind)
    m, n, k, dt = 9, 64, 64, HF
    g = gen(5)
    x, wg, wu, dh = rnd(g, m, k, dt=dt), rnd(g, n, k, dt=dt, std=k ** -0.5), rnd(g, n, k, dt=dt, std=k ** -0.5), rnd(g, m, n, dt=dt)
    _, gg, uu = run_glu(x, wg, wu, kind, True)
    got = run_bwd(dh, x, wg, wu, gg, uu, kind)
    X, G, U, D = (t.double().cpu() for t in (x, wg, wu, dh))

    def loss():
        return float((D * R.act64(X @ G.t(), kind)[0] * (X @ U.t())).sum())

    r = R.ROUND[dt]
    gp, up = X @ G.t(), X @ U.t()
    edg = D.abs() * (1.6 * r * gp.abs() * up.abs() + 1.13 * r * up.abs())
    edu = D.abs() * 1.13 * r * gp.abs()
    extra = (edg @ G.abs() + edu @ U.abs(), edg.t() @ X.abs(), edu.t() @ X.abs())
    ref = R.glu_bwd64(D, X, G, U, gp, up, kind, dt)
    for t, y, (_, e), ex in zip((X, G, U), got, ref, extra):
        for i, j in ((0, 0), (t.shape[0] - 1, 5), (3, t.shape[1] - 1), (4, 33)):
            v = float(t[i, j])
            t[i, j] = v + 1e-6
            hi = loss()
            t[i, j] = v - 1e-6
            lo = loss()
            t[i, j] = v
            d = (hi - lo) / 2e-6
            tol = float(e[i, j]) + float(ex[i, j]) + r * abs(d) + 1e-6
            if kind == "relu":      # a gate within the step of 0 may switch: none does at these values
                assert float(gp.abs().min()) > 1e-5
            assert abs(float(y[i, j]) - d) <= tol, (kind, i, j, float(y[i, j]), d, tol)


def test_gemm_glu_bwd_no_tokens_and_no_channels():
    say("gemm_glu_bwd empty")
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    w = torch.ones(64, 64, dtype=BF, device=DEV)
    _, dwg, dwu = run_bwd(e, e, w, w, e, e, "silu")
    assert bool((dwg == 0).all()) and bool((dwu == 0).all())
    n0 = torch.empty(5, 0, dtype=BF, device=DEV)
    x = torch.ones(5, 64, dtype=BF, device=DEV)
    w0 = torch.empty(0, 64, dtype=BF, device=DEV)
    dx, _, _ = run_bwd(n0, x, w0, w0, n0, n0, "silu")
    assert bool((dx == 0).all())


# ---------------------------------------------------------------------------
def block(m, n, k, ws, out):
    """The training pass and the serving pass of one block, into `out`."""
    g = gen(9)
    x, wg, wu = rnd(g, m, k, dt=BF), rnd(g, n, k, dt=BF, std=k ** -0.5), rnd(g, n, k, dt=BF, std=k ** -0.5)
    dh, b = rnd(g, m, n, dt=BF), ints(g, k, n)
    qw = torch.empty(2 * n, k, dtype=torch.int8, device=DEV)
    sw = torch.empty(2 * n, device=DEV)
    bsg.quant_i8(torch.cat([wg, wu]), qw, sw, 2 * n, k)
    sb = torch.full((k,), 1e-3, device=DEV)

    def call():
        bsg.gemm_glu(x, wg, wu, out["h"], out["g"], out["u"], m, n, k, workspace=ws["gemm_glu"])
        bsg.gemm_glu_bwd(dh, x, wg, wu, out["g"], out["u"], out["dx"], out["dwg"], out["dwu"], m, n, k,
                         workspace=ws["gemm_glu_bwd"])
        bsg.quant_i8(x, out["q"], out["s"], m, k)
        bsg.gemm_glu_i8(out["q"], qw[:n], qw[n:], out["s"], sw[:n], sw[n:], out["h8"], m, n, k, workspace=ws["gemm_glu_i8"])
        bsg.quant_i8(out["h8"], out["qh"], out["sh"], m, n)
        bsg.gemm_i8(out["qh"], b, out["sh"], sb, None, out["y"], m, k, n, workspace=ws["gemm_i8"])

    return call


def block_state(m, n, k):
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device=DEV)     # noqa: E731
    out = dict(h=e(m, n), g=e(m, n), u=e(m, n), dx=e(m, k), dwg=e(n, k), dwu=e(n, k), q=e(m, k, dt=torch.int8),
               s=e(m, dt=F32), h8=e(m, n), qh=e(m, n, dt=torch.int8), sh=e(m, dt=F32), y=e(m, k))
    ws = {op: scratch(op, m, *((k, n) if op == "gemm_i8" else (n, k)))
          for op in ("gemm_glu", "gemm_glu_bwd", "gemm_glu_i8", "gemm_i8")}
    return out, ws


@pytest.mark.parametrize("m,n,k", [(1, 256, 512), (40, 512, 2048), (300, 528, 1040)])
def test_streams_graph_and_repeats(m, n, k):
    """The same bits on the default stream, on two other streams at once (a
    workspace each), again, and from a graph replayed between eager work."""
    say("ffn streams and graph", m, n, k)
    ref, ws = block_state(m, n, k)
    block(m, n, k, ws, ref)()
    torch.cuda.synchronize()

    def same(out, what):
        for name in ref:
            assert torch.equal(out[name].view(torch.uint8), ref[name].view(torch.uint8)), (what, name)

    runs = []
    for _ in range(2):
        out, w = block_state(m, n, k)
        call = block(m, n, k, w, out)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        runs.append((out, w, call, st))
    torch.cuda.synchronize()
    for _, _, call, st in runs:
        with torch.cuda.stream(st):
            call()
            call()
    torch.cuda.synchronize()
    for out, *_ in runs:
        same(out, "stream")
    out, w = block_state(m, n, k)
    call = block(m, n, k, w, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    torch.cuda.synchronize()
    for r in range(3):
        for t in out.values():
            t.fill_(3)
        graph.replay()
        runs[0][2]()
        torch.cuda.synchronize()
        same(out, f"replay {r}")


def test_binding_refuses_mismatched_tensors():
    say("ffn binding checks")
    e = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=DEV)     # noqa: E731
    kw = dict(x=e(4, 64), w_gate=e(32, 64), w_up=e(32, 64), h=e(4, 32), g=None, u=None, m=4, n=32, k=64,
              workspace=scratch("gemm_glu", 4, 32, 64))
    bsg.gemm_glu(**kw)

    def status(**over):
        with pytest.raises(bsg.BsgError) as err:
            bsg.gemm_glu(**{**kw, **over})
        return err.value.status

    assert status(w_up=e(32, 64, dt=HF)) == 3
    assert status(h=e(4, 16)) == 2
    assert status(x=e(64, 4).t()) == 4
    assert status(x=torch.zeros(4, 64, dtype=BF)) == 6            # host memory
    b = dict(dh=e(4, 32), x=e(4, 64), w_gate=e(32, 64), w_up=e(32, 64), g=e(4, 32), u=e(4, 32), dx=e(4, 64),
             dw_gate=e(32, 64), dw_up=e(32, 64), m=4, n=32, k=64, workspace=e(16, dt=torch.uint8))
    with pytest.raises(bsg.BsgError) as err:
        bsg.gemm_glu_bwd(**b)                                     # workspace too small
    assert err.value.status == 2
    with pytest.raises(bsg.BsgError) as err:
        bsg.gemm_i8(e(4, 64), e(32, 64, dt=torch.int8), e(4, dt=F32), e(32, dt=F32), None, e(4, 32), 4, 32, 64)
    assert err.value.status == 3
    torch.cuda.synchronize()
