"""GPU tests of the expert operators together: a mixture-of-experts layer
forward and backward as a program runs it, from a graph, on two streams and
on workspaces that are shared or hold garbage."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
DEV = "cuda"


def say(*a):
    print(*a, flush=True)


def empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=DEV)


def codes(*shape, fmt="e4m3"):
    return empty(*shape, dtype=R.FP8[fmt])


class Quant:
    """What quant_fp8 makes of x (l, m, k): rows, and columns if asked."""

    def __init__(self, x, l, m, k, fmt="e4m3", tile=False, cols=False):
        mb, kb = -(-m // 128), -(-k // 128)
        self.q, self.s = codes(l, m, k, fmt=fmt), empty(*((l, mb, kb) if tile else (l, kb, m)))
        self.qt = codes(l, k, m, fmt=fmt) if cols else None
        self.st = empty(*((l, kb, mb) if tile else (l, mb, k))) if cols else None
        bsg.quant_fp8(x, self.q, self.s, self.qt, self.st, m, k, l=l, tile=tile, q_dtype=fmt)


class Layer:
    """out = sum_j weight_j W2_e relu(W1_e x): experts' weights quantised once, both ways."""

    def __init__(self, tokens, hidden, inner, experts, top_k, seed, masked=0.1):
        g = torch.Generator().manual_seed(seed)
        self.t, self.h, self.f, self.e, self.k = tokens, hidden, inner, experts, top_k
        self.x = torch.randn(tokens, hidden, generator=g).to(BF).to(DEV)
        self.ids = torch.randint(0, experts, (tokens, top_k), generator=g, dtype=torch.int32)
        self.ids[torch.rand(tokens, generator=g) < masked] = -1
        self.ids = self.ids.to(DEV)
        self.w = torch.rand(tokens, top_k, generator=g).to(DEV)
        self.w1 = (torch.randn(experts, inner, hidden, generator=g) * hidden ** -0.5).to(BF).to(DEV)
        self.w2 = (torch.randn(experts, hidden, inner, generator=g) * inner ** -0.5).to(BF).to(DEV)
        self.q1 = Quant(self.w1, experts, inner, hidden, tile=True, cols=True)
        self.q2 = Quant(self.w2, experts, hidden, inner, tile=True, cols=True)
        self.m = bsg.moe_rows(tokens, top_k, experts)
        i32 = lambda *s: empty(*s, dtype=torch.int32)  # noqa: E731
        self.ends, self.rows, self.row_of, self.pair_of = i32(experts), i32(experts), i32(tokens, top_k), i32(self.m)
        self.ws = empty(bsg.workspace_bytes("moe_sort", tokens, top_k, experts), dtype=torch.uint8)

    def sort(self):
        bsg.moe_sort(self.ids, self.ends, self.rows, self.row_of, self.pair_of, self.t, self.k, self.e, self.m,
                     workspace=self.ws)

    def forward(self):
        t, h, f, e, k, m = self.t, self.h, self.f, self.e, self.k, self.m
        self.sort()
        self.xs = torch.zeros(m, h, dtype=BF, device=DEV)
        bsg.moe_gather(self.x, self.row_of, self.ends, self.rows, None, self.xs, None, None, t, h, k, e, m)
        self.qx = Quant(self.xs, 1, m, h)
        self.y1, self.y2 = torch.zeros(m, f, dtype=BF, device=DEV), torch.zeros(m, h, dtype=BF, device=DEV)
        bsg.grouped_gemm_fp8(self.qx.q, self.q1.q, self.qx.s, self.q1.s, self.ends, None, self.y1, m, f, h, e)
        self.hs = torch.relu(self.y1)
        self.qh = Quant(self.hs, 1, m, f)
        bsg.grouped_gemm_fp8(self.qh.q, self.q2.q, self.qh.s, self.q2.s, self.ends, None, self.y2, m, h, f, e)
        out = empty(t, h, dtype=BF)
        bsg.moe_combine(self.y2, self.row_of, self.w, out, t, h, k, m)
        return out

    def backward(self, dout):
        t, h, f, e, k, m = self.t, self.h, self.f, self.e, self.k, self.m
        dy2, dw = torch.zeros(m, h, dtype=BF, device=DEV), empty(t, k)
        bsg.moe_combine_bwd(dout, self.y2, self.row_of, self.ends, self.rows, self.w, dy2, dw, t, h, k, e, m)
        g2 = Quant(dy2, 1, m, h, fmt="e5m2", cols=True)
        ht, xt = Quant(self.hs, 1, m, f, tile=True, cols=True), Quant(self.xs, 1, m, h, tile=True, cols=True)
        dw2, dw1 = empty(e, h, f, dtype=BF), empty(e, f, h, dtype=BF)
        bsg.grouped_gemm_fp8_wgrad(g2.qt, ht.qt, g2.st, ht.st, self.ends, dw2, m, h, f, e, a_dtype="e5m2")
        dh = torch.zeros(m, f, dtype=BF, device=DEV)
        bsg.grouped_gemm_fp8(g2.q, self.q2.qt, g2.s, self.q2.st, self.ends, None, dh, m, f, h, e, a_dtype="e5m2")
        dy1 = torch.where(self.y1 > 0, dh, torch.zeros_like(dh))
        g1 = Quant(dy1, 1, m, f, fmt="e5m2", cols=True)
        bsg.grouped_gemm_fp8_wgrad(g1.qt, xt.qt, g1.st, xt.st, self.ends, dw1, m, f, h, e, a_dtype="e5m2")
        dxs, dx = torch.zeros(m, h, dtype=BF, device=DEV), empty(t, h, dtype=BF)
        bsg.grouped_gemm_fp8(g1.q, self.q1.qt, g1.s, self.q1.st, self.ends, None, dxs, m, h, f, e, a_dtype="e5m2")
        bsg.moe_gather_bwd(dxs, None, self.row_of, dx, None, t, h, k, m)
        return dx, dw, dw1, dw2

    def plain(self, dout):
        """The layer in 64 bits on the CPU, without any quantisation, and its gradients by torch's autograd."""
        x, w, w1, w2 = (v.cpu().double().requires_grad_() for v in (self.x, self.w, self.w1, self.w2))
        ids = self.ids.cpu()
        out = torch.zeros(self.t, self.h, dtype=torch.float64)
        for e in range(self.e):
            for j in range(self.k):
                at = torch.nonzero(ids[:, j] == e).reshape(-1)
                y = torch.relu(x[at] @ w1[e].t()) @ w2[e].t()
                out = out.index_add(0, at, w[at, j, None] * y)
        out.backward(dout.cpu().double())
        return out.detach(), x.grad, w.grad, w1.grad, w2.grad


def off(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,hidden,inner,experts,top_k", [(300, 512, 384, 5, 2), (1024, 256, 640, 16, 4), (7, 256, 256, 3, 1)])
def test_layer(tokens, hidden, inner, experts, top_k):
    """A code is off by at most 2^-4 (E4M3) or 2^-3 (E5M2) of its value, evenly
    spread: 0.036 and 0.072 rms at most.  Errors of different operands add as
    squares.  The output passes two products with two E4M3 operands each:
    0.036 * 2 = 0.072.  dweight meets the second product's output: 0.072.  dx
    passes two products with an E5M2 and an E4M3 operand each, and dW1 one more
    E4M3 one: sqrt(2) * 0.080 = 0.114; dW2 has an E5M2 and an (itself inexact)
    E4M3 operand: sqrt(0.072^2 + 0.036^2 + 0.051^2) = 0.096.  Twice that leaves
    room for the signs that rounding turns at the ReLU."""
    say("layer", tokens, hidden, inner, experts, top_k)
    p = Layer(tokens, hidden, inner, experts, top_k, seed=tokens)
    dout = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    out = p.forward()
    got = (out, *p.backward(dout))
    names = ("out", "dx", "dweight", "dw1", "dw2")
    for name, a, b, most in zip(names, got, p.plain(dout), (0.144, 0.228, 0.144, 0.228, 0.192)):
        err = off(a, b)
        say(name, err)
        assert err < most, (name, err)
    # the same from call to call, bit for bit
    again = (p.forward(), *p.backward(dout))
    for name, a, b in zip(names, got, again):
        assert torch.equal(a, b), name


class Serve:
    """The serving path: quantised on the way in, only rows that hold a pair are computed."""

    def __init__(self, tokens, seed):
        self.p = Layer(tokens, 512, 256, 8, 2, seed)
        p = self.p
        self.xq, self.xs = torch.zeros(p.m, p.h, dtype=torch.float8_e4m3fn, device=DEV), torch.zeros(p.h // 128, p.m, device=DEV)
        self.prob = torch.zeros(p.m, device=DEV)
        self.y = torch.zeros(p.m, p.f, dtype=F16, device=DEV)
        self.out = torch.zeros(p.t, p.f, dtype=F16, device=DEV)

    def run(self):
        p = self.p
        p.sort()
        bsg.moe_gather(p.x, p.row_of, p.ends, p.rows, p.w, self.xq, self.xs, self.prob, p.t, p.h, p.k, p.e, p.m, zero_pad=False)
        bsg.grouped_gemm_fp8(self.xq, p.q1.q, self.xs, p.q1.s, p.ends, p.rows, self.y, p.m, p.f, p.h, p.e, max_rows=p.t)
        bsg.moe_combine(self.y, p.row_of, p.w, self.out, p.t, p.f, p.k, p.m)
        return self.out


@pytest.mark.parametrize("tokens", [1, 33, 2500])
def test_serving_path_from_a_graph(tokens):
    """Captured once, replayed on other tokens and another routing, with eager
    work between the replays; every replay has the eager call's bits."""
    say("graph", tokens)
    s = Serve(tokens, 3)
    others = [Layer(tokens, 512, 256, 8, 2, seed) for seed in (4, 5, 6)]
    want = []
    for o in others:
        for name in ("x", "ids", "w"):
            getattr(s.p, name).copy_(getattr(o, name))
        want.append(s.run().clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for o, w in list(zip(others, want)) * 2:
        for name in ("x", "ids", "w"):
            getattr(s.p, name).copy_(getattr(o, name))
        s.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out, w)
        assert float((torch.ones(1000, device=DEV) * 2).sum()) == 2000


def test_two_streams_at_once():
    """Calls that run at the same time, with a workspace each, do not meet."""
    a, b = Serve(900, 7), Serve(1100, 8)
    want = a.run().clone(), b.run().clone()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.out.zero_()
                s.run()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_explicit_stream():
    s = Serve(40, 9)
    want = s.run().clone()
    torch.cuda.synchronize()
    st, p = torch.cuda.Stream(), s.p
    s.out.zero_()
    torch.cuda.synchronize()
    bsg.moe_combine(s.y, p.row_of, p.w, s.out, p.t, p.f, p.k, p.m, stream=st)
    st.synchronize()
    assert torch.equal(s.out, want)


@pytest.mark.parametrize("m,n,k", [(130, 2048, 7168), (260, 520, 2048)])
def test_products_in_parts_share_a_workspace(m, n, k):
    """K in parts: two graphs on one workspace, replayed in turn, and a workspace full of NaN."""
    assert "/" in bsg.plan_string("gemm_fp8", m, n, k)
    ws = torch.full((bsg.workspace_bytes("gemm_fp8", m, n, k) // 4,), float("nan"), device=DEV)
    g = torch.Generator().manual_seed(m)
    sets = []
    for _ in range(2):
        a = Quant(torch.randn(m, k, generator=g).to(DEV), 1, m, k)
        b = Quant(torch.randn(n, k, generator=g).to(DEV), 1, n, k, tile=True)
        c = empty(m, n, dtype=BF)
        sets.append((a, b, c))

    def run(i):
        a, b, c = sets[i]
        bsg.gemm_fp8(a.q, b.q, a.s, b.s, c, m, n, k, workspace=ws)

    want = []
    for i in (0, 1):
        run(i)
        want.append(sets[i][2].clone())
        ref, err = R.gemm64(sets[i][0].q[0].cpu(), sets[i][1].q[0].cpu(), sets[i][0].s[0].cpu(), sets[i][1].s[0].cpu())
        R.check("c", want[i].cpu(), ref, err, BF)
    graphs = []
    for i in (0, 1):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(i)
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        sets[i][2].zero_()
        ws.fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(sets[i][2], want[i])


def test_tensors_that_do_not_fit_are_refused():
    s = Serve(8, 1)
    p = s.p
    args = dict(y=s.y, row_of=p.row_of, weight=p.w, out=s.out, tokens=p.t, hidden=p.f, top_k=p.k, m=p.m)
    for bad, status in ((dict(y=s.y[:-1]), 2), (dict(out=s.out.float()), 3), (dict(weight=p.w.cpu()), 6),
                        (dict(y=s.y.t()), 4), (dict(row_of=p.row_of.long()), 3)):
        with pytest.raises(bsg.BsgError) as e:
            bsg.moe_combine(**{**args, **bad})
        assert e.value.status == status, bad
    args = dict(a=s.xq, b=p.q1.q, a_scale=s.xs, b_scale=p.q1.s, padded_offsets=p.ends, expert_rows=p.rows, c=s.y, m=p.m, n=p.f,
                k=p.h, num_experts=p.e)
    for bad, status in ((dict(a=s.xq.float()), 3), (dict(b=p.q1.q[:-1]), 2), (dict(b_scale=p.q1.s[:, :-1].contiguous()), 2),
                        (dict(a_scale=s.xs.t()), 4), (dict(c=s.y.float()), 5), (dict(padded_offsets=p.ends[:-1]), 2),
                        (dict(a_dtype="e5m2"), 3)):
        with pytest.raises(bsg.BsgError) as e:
            bsg.grouped_gemm_fp8(**{**args, **bad})
        assert e.value.status == status, bad
    bsg.grouped_gemm_fp8(**{**args, "a": s.xq.view(torch.uint8), "b": p.q1.q.view(torch.uint8)})    # codes as bytes
