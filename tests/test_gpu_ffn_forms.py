"""Every kernel form of the feed-forward operators (ffn_forms.py) in every
type and activation, against the 64-bit definitions and their derived bounds
(ffn_ref.py), and bit for bit where small integers make every sum exact."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import ffn_forms as F
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


class Guarded:
    """A tensor between two stretches of sentinels."""

    def __init__(self, shape, dt, fill=77):
        n, self.pad, self.fill = torch.Size(shape).numel(), 1024, fill
        self.buf = torch.full((n + 2 * self.pad,), fill, dtype=dt, device=DEV)
        self.t = self.buf[self.pad:self.pad + n].view(shape)

    def check(self):
        p = self.pad
        assert bool((self.buf[:p] == self.fill).all()) and bool((self.buf[-p:] == self.fill).all()), "wrote past the end"


def call(op, m, n, k, outs, *args, **kw):
    """An operator on guarded outputs and a workspace of the exact size, full
    of the bytes of NaN, between sentinels."""
    ws = Guarded((bsg.workspace_bytes(op, m, n, k),), torch.uint8, 255)
    getattr(bsg, op)(*args, m, n, k, workspace=ws.t, **kw)
    ws.check()
    for o in outs:
        o.check()


@pytest.mark.parametrize("name", F.PRODUCTS["gemm_i8"])
def test_gemm_i8(name):
    m, n, k = F.PRODUCTS["gemm_i8"][name]
    g = gen(m)
    a, b = ints(g, m, k), ints(g, n, k)
    sa, sb = torch.rand(m, generator=g, device=DEV) * 0.01, torch.rand(n, generator=g, device=DEV) * 0.01
    ref, err = R.i8_64(a, b, sa, sb)
    for dt, bdt in ((BF, F32), (HF, BF), (F32, HF), (F32, None), (BF, None)):
        say("gemm_i8", name, (m, n, k), dt, bdt)
        bias = None if bdt is None else rnd(g, n, dt=bdt)
        c = Guarded((m, n), dt)
        call("gemm_i8", m, n, k, [c], a, b, sa, sb, bias, c.t)
        r = ref if bias is None else ref + bias.double()
        R.check("c", c.t, r, err if bias is None else err + R.E * (r.abs() + err), dt)


def glu_small_integers(op, name, m, n, k, dt):
    """Small integers: G, U and ReLU(G) U are exact."""
    g = gen(k)
    x, wg, wu = ints(g, m, k, lo=-2, hi=2), ints(g, n, k, lo=-2, hi=2), ints(g, n, k, lo=-2, hi=2)
    gr, ur = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    out = [Guarded((m, n), dt) for _ in range(3)]
    if op == "gemm_glu":
        call(op, m, n, k, out, x.to(dt), wg.to(dt), wu.to(dt), *(o.t for o in out), act="relu")
        assert torch.equal(out[1].t, gr.to(dt)) and torch.equal(out[2].t, ur.to(dt)), name
    else:
        one = torch.ones(max(m, n), device=DEV)
        call(op, m, n, k, out[:1], x, wg, wu, one[:m], one[:n], one[:n], out[0].t, act="relu")
    assert torch.equal(out[0].t, (gr.clamp(min=0) * ur).float().to(dt)), name


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("name", F.PRODUCTS["gemm_glu"])
def test_gemm_glu(name, dt):
    m, n, k = F.PRODUCTS["gemm_glu"][name]
    g = gen(m + n)
    x, wg, wu = rnd(g, m, k, dt=dt), rnd(g, n, k, dt=dt, std=2 * k ** -0.5), rnd(g, n, k, dt=dt, std=k ** -0.5)
    for kind in R.ACTS:
        h, eh, gr, ur, eg, eu = R.glu64(x, wg, wu, kind)
        for save in (True, False):
            say("gemm_glu", name, (m, n, k), dt, kind, save)
            out = [Guarded((m, n), dt) for _ in range(3 if save else 1)]
            call("gemm_glu", m, n, k, out, x, wg, wu, *(o.t for o in out), *([] if save else [None, None]), act=kind)
            for o, what, r, e in zip(out, "hgu", (h, gr, ur), (eh, eg, eu)):
                R.check(what, o.t, r, e, dt)
    glu_small_integers("gemm_glu", name, m, n, k, dt)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("name", F.PRODUCTS["gemm_glu_i8"])
def test_gemm_glu_i8(name, dt):
    m, n, k = F.PRODUCTS["gemm_glu_i8"][name]
    g = gen(m + n)
    a, wg, wu = ints(g, m, k), ints(g, n, k), ints(g, n, k)
    sa = (0.5 + torch.rand(m, generator=g, device=DEV)) / 73
    sg, su = ((0.5 + torch.rand(n, generator=g, device=DEV)) * k ** -0.5 / 73 for _ in range(2))
    gr, eg = R.i8_64(a, wg, sa, sg)
    ur, eu = R.i8_64(a, wu, sa, su)
    for kind in R.ACTS:
        say("gemm_glu_i8", name, (m, n, k), dt, kind)
        h = Guarded((m, n), dt)
        call("gemm_glu_i8", m, n, k, [h], a, wg, wu, sa, sg, su, h.t, act=kind)
        ref, err = R._gate(gr, ur, eg, eu, kind)
        R.check("h", h.t, ref, err, dt)
    glu_small_integers("gemm_glu_i8", name, m, n, k, dt)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("name", F.BACKWARD)
def test_gemm_glu_bwd(name, dt):
    m, n, k = F.BACKWARD[name]
    g = gen(m + n)
    t = (rnd(g, m, n, dt=dt), rnd(g, m, k, dt=dt), rnd(g, n, k, dt=dt, std=k ** -0.5), rnd(g, n, k, dt=dt, std=k ** -0.5),
         rnd(g, m, n, dt=dt, std=2.0), rnd(g, m, n, dt=dt))

    def run(t, kind):
        out = [Guarded((m, k), dt), Guarded((n, k), dt), Guarded((n, k), dt)]
        call("gemm_glu_bwd", m, n, k, out, *t, *(o.t for o in out), act=kind)
        return [o.t for o in out]

    for kind in R.ACTS:
        say("gemm_glu_bwd", name, (m, n, k), dt, kind)
        for what, y, (r, e) in zip(("dx", "dwg", "dwu"), run(t, kind), R.glu_bwd64(*t, kind, dt)):
            R.check(what, y, r, e, dt)
    # ReLU and small integers: dG, dU and every sum are exact
    dh, x, wg, wu, gg, uu = (ints(g, *v.shape, lo=-2, hi=2, dt=dt) for v in t)
    dx, dwg, dwu = run((dh, x, wg, wu, gg, uu), "relu")
    on = (gg > 0).double()
    dg, du = dh.double() * uu.double() * on, dh.double() * gg.double() * on
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).to(dt))
    assert torch.equal(dwg, (dg.t() @ x.double()).to(dt)) and torch.equal(dwu, (du.t() @ x.double()).to(dt))


class Block:
    """A block's training pass and serving pass, each output and workspace
    between sentinels."""

    def __init__(self, m, n, k):
        g = gen(m + n + k)
        self.size = m, n, k
        self.x, self.dh = rnd(g, m, k, dt=BF), rnd(g, m, n, dt=BF)
        self.wg, self.wu = rnd(g, n, k, dt=BF, std=k ** -0.5), rnd(g, n, k, dt=BF, std=k ** -0.5)
        self.qg, self.qu, self.qd = ints(g, n, k), ints(g, n, k), ints(g, k, n)
        self.sn, self.sk = torch.full((n,), 1e-2 * k ** -0.5, device=DEV), torch.full((k,), 1e-2, device=DEV)
        i8 = torch.int8
        self.out = {name: Guarded(s, dt) for name, (s, dt) in dict(
            h=((m, n), BF), g=((m, n), BF), u=((m, n), BF), dx=((m, k), BF), dwg=((n, k), BF), dwu=((n, k), BF),
            q=((m, k), i8), s=((m,), F32), h8=((m, n), BF), qh=((m, n), i8), sh=((m,), F32), y=((m, k), BF)).items()}
        self.ws = {op: Guarded((bsg.workspace_bytes(op, m, *((k, n) if op == "gemm_i8" else (n, k))),), torch.uint8, 255)
                   for op in ("gemm_glu", "gemm_glu_bwd", "gemm_glu_i8", "gemm_i8")}

    def __call__(self):
        (m, n, k), o, w = self.size, {a: b.t for a, b in self.out.items()}, {a: b.t for a, b in self.ws.items()}
        bsg.gemm_glu(self.x, self.wg, self.wu, o["h"], o["g"], o["u"], m, n, k, workspace=w["gemm_glu"])
        bsg.gemm_glu_bwd(self.dh, self.x, self.wg, self.wu, o["g"], o["u"], o["dx"], o["dwg"], o["dwu"], m, n, k,
                         workspace=w["gemm_glu_bwd"])
        bsg.quant_i8(self.x, o["q"], o["s"], m, k)
        bsg.gemm_glu_i8(o["q"], self.qg, self.qu, o["s"], self.sn, self.sn, o["h8"], m, n, k, workspace=w["gemm_glu_i8"])
        bsg.quant_i8(o["h8"], o["qh"], o["sh"], m, n)
        bsg.gemm_i8(o["qh"], self.qd, o["sh"], self.sk, None, o["y"], m, k, n, workspace=w["gemm_i8"])

    def same(self, ref, what):
        for name, o in self.out.items():
            o.check()
            assert torch.equal(o.t.view(torch.uint8), ref.out[name].t.view(torch.uint8)), (what, name)
        for w in self.ws.values():
            w.check()


@pytest.mark.parametrize("size", F.PARTS)
def test_parts_of_k_repeated_on_streams_and_in_a_graph(size):
    """The tiles' partial sums and the kernels that join them: calls one after
    another on one workspace, on two streams at once (a workspace each), and
    replays of a graph between eager work give the first call's bits."""
    say("parts of K", size)
    ref = Block(*size)
    ref()
    torch.cuda.synchronize()
    again = Block(*size)
    for _ in range(3):
        again()
    torch.cuda.synchronize()
    again.same(ref, "in a row")
    runs = [(Block(*size), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(2):
        for b, st in runs:
            with torch.cuda.stream(st):
                b()
    torch.cuda.synchronize()
    for b, _ in runs:
        b.same(ref, "streams")
    b, side = Block(*size), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b()
    torch.cuda.synchronize()
    for r in range(3):
        for o in b.out.values():
            o.t.fill_(3)
        graph.replay()
        again()
        torch.cuda.synchronize()
        b.same(ref, f"replay {r}")
        again.same(ref, f"beside replay {r}")
