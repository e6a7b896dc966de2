"""GPU tests of the expert operators at the ends of their sizes: buffers whose
offsets pass 32 bits, and sums of no or few elements in the largest tiles."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
DEV = "cuda"


def test_rows_past_four_gib():
    """Rows of 8 KB up to number 599999: 4.9 GB."""
    t, k, h, m = 40, 2, 4096, 600064
    print("rows past 4 GiB", flush=True)
    g = torch.Generator().manual_seed(1)
    x, w, d = torch.randn(t, h, generator=g).to(BF), torch.rand(t, k, generator=g), torch.randn(t, h, generator=g).to(BF)
    rows = torch.randperm(m, generator=g)[: t * k].to(torch.int32).reshape(t, k)
    rows[0, 0], rows[0, 1] = m - 1, 524288 + 7          # the last row, and one just past 4 GiB
    assert len(set(rows.reshape(-1).tolist())) == t * k
    ends, held = torch.tensor([m], dtype=torch.int32, device=DEV), torch.tensor([m], dtype=torch.int32, device=DEV)
    y = torch.zeros(m, h, dtype=BF, device=DEV)
    bsg.moe_gather(x.cuda(), rows.cuda(), ends, held, None, y, None, None, t, h, k, 1, m)
    at = rows.reshape(-1).long().cuda()
    assert torch.equal(y[at].cpu(), x.repeat_interleave(k, 0)) and int((y != 0).any(1).sum()) == t * k
    out = torch.empty(t, h, dtype=BF, device=DEV)
    bsg.moe_combine(y, rows.cuda(), w.cuda(), out, t, h, k, m)
    small = torch.arange(t * k, dtype=torch.int32).reshape(t, k)       # the same rows by themselves
    yr = x.repeat_interleave(k, 0)
    ref, mag = R.combine64(yr, small, w)
    R.check("out", out.cpu(), ref, (k + 2) * R.E * mag, BF)
    dw = torch.empty(t, k, device=DEV)
    bsg.moe_combine_bwd(d.cuda(), y, rows.cuda(), ends, held, w.cuda(), y, dw, t, h, k, 1, m)
    ref_y, ref_w, mag = R.combine_bwd64(d, yr, small, w)
    R.check("dy", y[at].cpu(), ref_y, R.E * ref_y.abs(), BF)
    R.check("dweight", dw.cpu(), ref_w, (h + 1) * R.E * mag, torch.float32)


def whole(rows, k, tile, g):
    """Small whole numbers with scales of powers of two: sums are exact (tests/test_gpu_fp8.py)."""
    kb = -(-k // 128)
    q = torch.randint(-4, 5, (rows, k), generator=g).float().to(torch.float8_e4m3fn)
    return q, torch.exp2(torch.randint(-1, 2, (-(-rows // 128), kb) if tile else (kb, rows), generator=g).float())


@pytest.mark.parametrize("max_rows", [0, 64])
def test_grouped_product_past_four_gib(max_rows):
    """The last expert's rows and weight begin past 4 GiB of A, of B and of C."""
    m, n, k, experts, last = 589824, 4096, 8192, 160, 60
    print("grouped past 4 GiB", max_rows, flush=True)
    g = torch.Generator().manual_seed(2)
    a, b = (torch.zeros(*s, dtype=torch.float8_e4m3fn, device=DEV) for s in ((m, k), (experts, n, k)))
    c = torch.full((m, n), 5.0, dtype=BF, device=DEV)
    sa, sb = torch.zeros(k // 128, m, device=DEV), torch.zeros(experts, n // 128, k // 128, device=DEV)
    x, sx = whole(256, k, False, g)
    w, sw = whole(n, k, True, g)
    a[m - 256:], sa[:, m - 256:], b[-1], sb[-1] = x.cuda(), sx.cuda(), w.cuda(), sw.cuda()
    ends = torch.full((experts,), m - 256, dtype=torch.int32)
    ends[-1] = m
    rows = torch.zeros(experts, dtype=torch.int32)
    rows[0], rows[-1] = 1, last
    bsg.grouped_gemm_fp8(a, b, sa, sb, ends.cuda(), rows.cuda(), c, m, n, k, experts, max_rows=max_rows)
    want = (R.values(x, sx, False)[:last].cuda() @ R.values(w, sw, True).cuda().t()).to(BF)
    assert torch.equal(c[m - 256:m - 256 + last], want)
    assert bool((c[0] == 0).all()) and bool((c[m - 256 + last:] == 5).all()) and bool((c[1:4097] == 5).all())


@pytest.mark.parametrize("k", [0, 16, 128, 144, 256])
@pytest.mark.parametrize("m,n", [(5000, 4096), (8192, 8192), (1500, 1032)])
def test_short_sums_in_large_tiles(m, n, k):
    """Fewer blocks than the ring has slots."""
    print("short sums", m, n, k, bsg.plan_string("gemm_fp8", m, n, k), flush=True)
    g = torch.Generator().manual_seed(k)
    a, sa = whole(m, k, False, g)
    b, sb = whole(n, k, True, g)
    c = torch.full((m + 2, n), 5.0, dtype=BF, device=DEV)
    a, sa, b, sb = (v.cuda() for v in (a, sa, b, sb))
    ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device=DEV)
    bsg.gemm_fp8(a, b, sa, sb, c[1:-1], m, n, k, workspace=ws)
    want = (R.values(a, sa, False) @ R.values(b, sb, True).t()).to(BF) if k else torch.zeros(m, n, dtype=BF, device=DEV)
    assert torch.equal(c[1:-1], want) and bool((c[0] == 5).all()) and bool((c[-1] == 5).all())


def test_grouped_short_sums_in_large_tiles():
    m, n, k, experts = 16384, 4096, 48, 3
    g = torch.Generator().manual_seed(4)
    counts, ends = [5000, 0, 11000], torch.tensor([5120, 5120, 16128], dtype=torch.int32)
    a, sa = (v.cuda() for v in whole(m, k, False, g))
    bs = [[v.cuda() for v in whole(n, k, True, g)] for _ in range(experts)]
    c = torch.full((m, n), 5.0, dtype=F16, device=DEV)
    print("grouped short sums", flush=True)
    bsg.grouped_gemm_fp8(a, torch.stack([x[0] for x in bs]), sa, torch.stack([x[1] for x in bs]), ends.cuda(),
                         torch.tensor(counts, dtype=torch.int32, device=DEV), c, m, n, k, experts)
    for e, first in ((0, 0), (2, 5120)):
        x = slice(first, first + counts[e])
        want = (R.values(a[x], sa[:, x], False) @ R.values(*bs[e], True).t()).to(F16)
        assert torch.equal(c[x], want)
        assert bool((c[first + counts[e]:int(ends[e])] == 5).all())
    assert bool((c[16128:] == 5).all())


@pytest.mark.parametrize("dt", [torch.float32, BF, F16])
@pytest.mark.parametrize("t,k", [(1, 1), (37, 11), (9, 64)])
def test_combine_bwd_without_weights(t, k, dt):
    """Weights of one, and more choices than a lane holds in one batch."""
    print("combine_bwd without weights", t, k, dt, flush=True)
    hidden, m = 264, 768
    g = torch.Generator().manual_seed(t + k)
    dout, y = torch.randn(t, hidden, generator=g).to(dt), torch.randn(m, hidden, generator=g).to(dt)
    rows = torch.randperm(m, generator=g)[: t * k].to(torch.int32).reshape(t, k)
    rows[torch.rand(t, k, generator=g) < 0.2] = -1
    ref_y, ref_w, mag = R.combine_bwd64(dout, y, rows, None)
    dy, dw = torch.zeros(m, hidden, dtype=dt, device=DEV), torch.full((t, k), 7.0, device=DEV)
    bsg.moe_combine_bwd(dout.cuda(), y.cuda(), rows.cuda(), None, None, None, dy, dw, t, hidden, k, 1, m, zero_pad=False)
    R.check("dy", dy.cpu(), ref_y, 0 * ref_y, dt)         # a copy
    R.check("dweight", dw.cpu(), ref_w, (hidden + 1) * R.E * mag, torch.float32)


def test_rows_of_no_tokens_are_padding():
    """Without tokens each range is padding alone: zeros, and nothing behind the last range."""
    print("no tokens", flush=True)
    m, hidden, experts = 768, 128, 3
    ends = torch.tensor([256, 256, 512], dtype=torch.int32, device=DEV)
    held = torch.zeros(experts, dtype=torch.int32, device=DEV)
    x, rows = torch.empty(0, hidden, dtype=BF, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    for call in (lambda y: bsg.moe_gather(x, rows, ends, held, None, y, None, None, 0, hidden, 2, experts, m),
                 lambda y: bsg.moe_combine_bwd(x, None, rows, ends, held, None, y, None, 0, hidden, 2, experts, m)):
        y = torch.full((m, hidden), 5.0, dtype=BF, device=DEV)
        call(y)
        assert bool((y[:512] == 0).all()) and bool((y[512:] == 5).all())


def test_two_streams_at_once():
    """Two products of K in parts at once, each with its own workspace."""
    print("two streams", flush=True)
    m, n, k = 130, 2048, 7168
    g = torch.Generator().manual_seed(6)
    sides = []
    for _ in range(2):
        a, sa = (v.cuda() for v in whole(m, k, False, g))
        b, sb = (v.cuda() for v in whole(n, k, True, g))
        want = (R.values(a, sa, False) @ R.values(b, sb, True).t()).to(BF)
        ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device=DEV)
        sides.append((a, b, sa, sb, want, torch.zeros(m, n, dtype=BF, device=DEV), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        for a, b, sa, sb, want, c, ws, stream in sides:
            bsg.gemm_fp8(a, b, sa, sb, c, m, n, k, workspace=ws, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    for side in sides:
        assert torch.equal(side[5], side[4])


def test_wgrad_of_the_most_rows():
    """Operands with 2^22 bytes between their rows; the last expert's range is at their end."""
    m, n, k, last = 1 << 22, 264, 520, 512
    print("wgrad of 2^22 rows", flush=True)
    g = torch.Generator().manual_seed(7)
    a, b = (torch.zeros(r, m, dtype=torch.float8_e4m3fn, device=DEV) for r in (n, k))
    sa, sb = torch.zeros(m // 128, n, device=DEV), torch.zeros(-(-k // 128), m // 128, device=DEV)
    x, sx = whole(n, last, False, g)
    w, sw = whole(k, last, True, g)
    a[:, m - last:], sa[-last // 128:], b[:, m - last:], sb[:, -last // 128:] = x.cuda(), sx.cuda(), w.cuda(), sw.cuda()
    ends = torch.tensor([m - last, m - last, m], dtype=torch.int32, device=DEV)
    c = torch.full((4, n, k), 5.0, dtype=BF, device=DEV)
    bsg.grouped_gemm_fp8_wgrad(a, b, sa, sb, ends, c[:3], m, n, k, 3)
    want = (R.values(x, sx, False).cuda() @ R.values(w, sw, True).cuda().t()).to(BF)
    assert bool((c[:2] == 0).all()) and torch.equal(c[2], want) and bool((c[3] == 5).all())


def test_product_of_the_most_rows():
    """2^22 rows: the last begin past 4 GiB of A and of C."""
    m, n, k, last = 1 << 22, 1032, 1040, 300
    print("product of 2^22 rows", bsg.plan_string("gemm_fp8", m, n, k), flush=True)
    g = torch.Generator().manual_seed(8)
    a, sa = torch.zeros(m, k, dtype=torch.float8_e4m3fn, device=DEV), torch.zeros(-(-k // 128), m, device=DEV)
    x, sx = whole(last, k, False, g)
    b, sb = whole(n, k, True, g)
    a[m - last:], sa[:, m - last:] = x.cuda(), sx.cuda()
    c = torch.full((m, n), 5.0, dtype=BF, device=DEV)
    ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device=DEV)
    bsg.gemm_fp8(a, b.cuda(), sa, sb.cuda(), c, m, n, k, workspace=ws)
    want = (R.values(x, sx, False).cuda() @ R.values(b, sb, True).cuda().t()).to(BF)
    assert torch.equal(c[m - last:], want) and not bool(c[:m - last].any())
