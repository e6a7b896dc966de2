"""GPU tests of the products of 8-bit floats with a scale for each block of
128, against the 64-bit reference of moe_ref.py.

"whole" operands are small whole numbers with power-of-two scales: every
product and every partial sum is a whole multiple of one power of two that fp32
holds, the matrix instruction drops nothing (products lie within 13 bits), and
C has to be the exact sum rounded once, bit for bit.  "random" ones are what
quant_fp8 makes of normal numbers."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def say(*a):
    print(*a, flush=True)


def operand(rows, k, kind, fmt, tile, g):
    kb = -(-k // 128)
    shape = (-(-rows // 128), kb) if tile else (kb, rows)
    if kind == "whole":
        q = torch.randint(-4, 5, (rows, k), generator=g).float().to(R.FP8[fmt])
        return q, torch.exp2(torch.randint(-1, 2, shape, generator=g).float())
    x = torch.randn(1, rows, k, generator=g) * torch.exp(torch.randn(1, rows, 1, generator=g))
    q, s = R.quant(x, fmt, tile)
    return q[0], s[0]


def compare(got, a, b, sa, sb, kind, dt, name="c"):
    ref, err = R.gemm64(a, b, sa, sb)
    if kind == "whole":
        assert torch.equal(got, ref.to(dt)), (name, (got.double() - ref.to(dt).double()).abs().max())
    else:
        if dt == F16:
            # fp16's largest value is 65504 and its step there 32: what lies at 65520 or past it rounds to
            # infinity, whatever the sum's error if that leaves it there
            past = ref.abs() - err >= 65520
            assert torch.equal(got[past].double(), ref[past].sign() * float("inf"))
            got, ref = torch.where(past, torch.zeros_like(got), got), torch.where(past, torch.zeros_like(ref), ref)
        R.check(name, got, ref, err, dt)
        if ref.numel() >= 4096:
            # and as a whole: the roundings of C, uniform in a step, and the dropped bits, together far less
            # than twice half a step
            off = (got.double() - ref).norm() / ref.norm()
            assert float(off) < {BF: 2.0 ** -8, F16: 2.0 ** -11}[dt], float(off)


SIZES = [(1, 8, 16), (1, 7168, 2048), (5, 64, 128), (16, 136, 144), (17, 256, 400), (33, 128, 4096), (64, 1000, 272),
         (67, 4096, 512), (128, 128, 128), (200, 264, 1040), (256, 256, 2048), (300, 520, 640), (513, 1032, 384),
         (1003, 776, 208), (130, 2048, 7168)]


@pytest.mark.parametrize("kind", ["whole", "random"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm_fp8(m, n, k, kind):
    g = torch.Generator().manual_seed(m + n + k)
    for fmt, dt in ((("e4m3", BF), ("e5m2", F16)) if (m + n) % 2 else (("e5m2", BF), ("e4m3", F16))):
        say("gemm_fp8", m, n, k, kind, fmt, dt)
        a, sa = operand(m, k, kind, fmt, False, g)
        b, sb = operand(n, k, kind, "e4m3", True, g)
        # the output between guard rows, which stay as they are
        c = torch.full((m + 2, n), 5.0, dtype=dt, device="cuda")
        ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device="cuda")
        bsg.gemm_fp8(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), c[1:-1], m, n, k, a_dtype=fmt, workspace=ws)
        c = c.cpu()
        assert bool((c[0] == 5).all()) and bool((c[-1] == 5).all())
        compare(c[1:-1], a, b, sa, sb, kind, dt)


# Large enough for each shape of tile in turn, whole and ragged, one round of
# them and several, a last round that goes out in halves; checked on the GPU.
LARGE = {(5000, 4096, 400): "Mid", (2049, 1032, 1040): "Mid", (4200, 4104, 1040): "Mid", (4096, 4096, 1024): "Big",
         (2500, 4096, 1040): "Big", (4200, 4104, 2064): "Big", (5100, 4104, 2064): "Big", (64, 512, 512): "few 64",
         (17, 256, 400): "few 32", (16, 136, 144): "few 16", (67, 4096, 512): "Small", (40, 512, 4096): "Small / 8",
         (130, 2048, 7168): "Small / 5"}


@pytest.mark.parametrize("kind", ["whole", "random"])
@pytest.mark.parametrize("m,n,k", LARGE)
def test_gemm_fp8_in_every_form(m, n, k, kind):
    assert bsg.plan_string("gemm_fp8", m, n, k) == LARGE[m, n, k]
    say("gemm_fp8", m, n, k, kind, LARGE[m, n, k])
    g = torch.Generator().manual_seed(m + n + k)
    fmt, dt = ("e5m2", BF) if m % 2 else ("e4m3", F16)
    a, sa = (v.cuda() for v in operand(m, k, kind, fmt, False, g))
    b, sb = (v.cuda() for v in operand(n, k, kind, "e4m3", True, g))
    c = torch.full((m + 2, n), 5.0, dtype=dt, device="cuda")
    ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device="cuda")
    bsg.gemm_fp8(a, b, sa, sb, c[1:-1], m, n, k, a_dtype=fmt, workspace=ws)
    assert bool((c[0] == 5).all()) and bool((c[-1] == 5).all())
    compare(c[1:-1], a, b, sa, sb, kind, dt)


@pytest.mark.parametrize("kind", ["whole", "random"])
def test_grouped_gemm_fp8_in_large_tiles(kind):
    """256 x 256 tiles, in two rounds and a part, of uneven experts."""
    counts, m, n, k = [3000, 0, 1, 257, 5000, 128, 129, 2600, 4000], 17408, 2048, 2064
    g = torch.Generator().manual_seed(5)
    ends, rows = offsets_of(counts, m)
    a, sa = (v.cuda() for v in operand(m, k, kind, "e4m3", False, g))
    bs = [[v.cuda() for v in operand(n, k, kind, "e4m3", True, g)] for _ in counts]
    b, sb = torch.stack([x[0] for x in bs]), torch.stack([x[1] for x in bs])
    for use_rows in (True, False):
        say("grouped_gemm_fp8 large", kind, use_rows)
        c = torch.full((m, n), 5.0, dtype=BF, device="cuda")
        bsg.grouped_gemm_fp8(a, b, sa, sb, ends.cuda(), rows.cuda() if use_rows else None, c, m, n, k, len(counts),
                             max_rows=max(counts))
        at = 0
        for e, (x, s) in enumerate(bs):
            end = int(ends[e])
            last = at + counts[e] if use_rows else end
            if last > at:
                compare(c[at:last], a[at:last], x, sa[:, at:last], s, kind, BF, f"expert {e}")
            assert bool((c[last:end] == 5).all())
            at = end
        assert bool((c[at:] == 5).all())


@pytest.mark.parametrize("kind", ["whole", "random"])
def test_grouped_gemm_fp8_wgrad_in_large_tiles(kind):
    counts, m, n, k = [3000, 0, 700, 256, 1500, 40], 6400, 2056, 2064
    g = torch.Generator().manual_seed(6)
    ends, rows = offsets_of(counts, m)
    a, sa = operand(n, m, kind, "e5m2", False, g)
    b, sb = operand(k, m, kind, "e4m3", True, g)
    a.view(torch.uint8)[:, R.held_rows(ends, rows, m) == 1] = 0
    a, sa, b, sb = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    say("wgrad large", kind)
    c = torch.full((len(counts), n, k), 5.0, dtype=BF, device="cuda")
    bsg.grouped_gemm_fp8_wgrad(a, b, sa, sb, ends.cuda(), c, m, n, k, len(counts), a_dtype="e5m2")
    at = 0
    for e, end in enumerate(ends.tolist()):
        if end == at:
            assert bool((c[e] == 0).all())
        else:
            compare(c[e], a[:, at:end], b[:, at:end], sa[at // 128:end // 128], sb[:, at // 128:end // 128], kind, BF)
        at = end


def test_gemm_fp8_long_k():
    """More than 64 blocks, whose scales of B a wave holds, twice over."""
    for m, n, k in ((3, 128, 20000), (300, 264, 20000)):
        say("gemm_fp8", m, n, k)
        g = torch.Generator().manual_seed(k)
        a, sa = operand(m, k, "whole", "e4m3", False, g)
        b, sb = operand(n, k, "whole", "e4m3", True, g)
        c = torch.empty(m, n, dtype=BF, device="cuda")
        ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device="cuda")
        bsg.gemm_fp8(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), c, m, n, k, workspace=ws)
        compare(c.cpu(), a, b, sa, sb, "whole", BF)


def test_grouped_long_k_large_tiles():
    m, n, k = 8192, 4096, 9232
    g = torch.Generator().manual_seed(8)
    ends, rows = offsets_of([8000], m)
    a, sa = (v.cuda() for v in operand(m, k, "whole", "e4m3", False, g))
    b, sb = (v.cuda() for v in operand(n, k, "whole", "e4m3", True, g))
    c = torch.full((m, n), 5.0, dtype=F16, device="cuda")
    say("grouped long k")
    bsg.grouped_gemm_fp8(a, b[None], sa, sb[None], ends.cuda(), rows.cuda(), c, m, n, k, 1)
    compare(c[:8000], a[:8000], b, sa[:, :8000], sb, "whole", F16)
    assert bool((c[8000:] == 5).all())


def test_gemm_fp8_of_nothing():
    c = torch.full((4, 16), 5.0, dtype=BF, device="cuda")
    e = torch.empty(0, device="cuda", dtype=torch.uint8)
    f = torch.empty(0, device="cuda")
    ws = torch.empty(bsg.workspace_bytes("gemm_fp8", 4, 16, 0), dtype=torch.uint8, device="cuda")
    bsg.gemm_fp8(e, e, f, f, c, 4, 16, 0, workspace=ws)
    assert bool((c == 0).all())
    some, scales = torch.zeros(512, dtype=torch.uint8, device="cuda"), torch.ones(8, device="cuda")
    bsg.gemm_fp8(e, some, f, scales, c[:0], 0, 16, 32)
    bsg.gemm_fp8(some, e, scales, f, c[:, :0].contiguous(), 4, 0, 32)


@pytest.mark.parametrize("m", [3, 40, 300])
def test_gemm_fp8_infinite_scales_stay_in_their_rows(m):
    """A row of A whose scale is not finite, as quant_fp8 leaves one, gives NaN
    in its row of C alone; a tile of B in its 128 columns alone."""
    n, k = 384, 512
    g = torch.Generator().manual_seed(m)
    a, sa = operand(m, k, "whole", "e4m3", False, g)
    b, sb = operand(n, k, "whole", "e4m3", True, g)
    ref = (R.values(a, sa, False) @ R.values(b, sb, True).t()).to(BF)
    a[1, 128:256] = 0
    sa[1, 1] = float("nan")
    sb[1, 2] = float("inf")
    b[128:256, 256:384] = 0
    c = torch.empty(m, n, dtype=BF, device="cuda")
    ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device="cuda")
    bsg.gemm_fp8(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), c, m, n, k, workspace=ws)
    c = c.cpu()
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[1] = True
    bad[:, 128:256] = True
    assert bool(torch.isnan(c[bad]).all()) and torch.equal(c[~bad], ref[~bad])


def offsets_of(counts, m):
    ends = torch.cumsum((torch.tensor(counts) + 255) // 256 * 256, 0).to(torch.int32)
    assert int(ends[-1]) <= m
    return ends, torch.tensor(counts, dtype=torch.int32)


GROUPS = [([1], 256, 128, 128), ([0, 3, 0], 512, 136, 272), ([7, 0, 300, 16, 33], 1536, 256, 512), ([256, 512], 1024, 1032, 144),
          ([64, 65, 1, 2, 0, 129], 2048, 392, 2048), ([1] * 70, 70 * 256, 64, 256), ([40, 0, 900], 1280, 520, 7168)]


@pytest.mark.parametrize("kind", ["whole", "random"])
@pytest.mark.parametrize("counts,m,n,k", GROUPS)
def test_grouped_gemm_fp8(counts, m, n, k, kind):
    g = torch.Generator().manual_seed(m + n)
    experts = len(counts)
    ends, rows = offsets_of(counts, m)
    fmt, dt = ("e4m3", BF) if n % 16 else ("e5m2", F16)
    a, sa = operand(m, k, kind, fmt, False, g)
    bs = [operand(n, k, kind, "e4m3", True, g) for _ in counts]
    b, sb = torch.stack([x[0] for x in bs]).cuda(), torch.stack([x[1] for x in bs]).cuda()
    held = R.held_rows(ends, rows, m)
    # rows that hold no pair are not read where expert_rows is given
    dirty, dirty_s = a.clone(), sa.clone()
    dirty.view(torch.uint8)[held != 0] = 0x7F
    dirty_s[:, held != 0] = float("nan")
    for use_rows, max_rows in ((True, 0), (True, max(counts)), (True, 1), (False, 0), (False, max(counts))):
        say("grouped_gemm_fp8", counts[:6], m, n, k, kind, use_rows, max_rows)
        c = torch.full((m, n), 5.0, dtype=dt, device="cuda")
        bsg.grouped_gemm_fp8((dirty if use_rows else a).cuda(), b, (dirty_s if use_rows else sa).cuda(), sb, ends.cuda(),
                             rows.cuda() if use_rows else None, c, m, n, k, experts, max_rows=max_rows, a_dtype=fmt)
        c, at = c.cpu(), 0
        for e, (x, s) in enumerate(bs):
            last, end = at + (counts[e] if use_rows else int(ends[e]) - at), int(ends[e])
            if last > at:
                compare(c[at:last], a[at:last], x, sa[:, at:last], s, kind, dt, f"expert {e}")
            assert bool((c[last:end] == 5).all())       # rows that hold no pair stay as they are
            at = end
        assert bool((c[at:] == 5).all())


@pytest.mark.parametrize("kind", ["whole", "random"])
@pytest.mark.parametrize("counts,m,n,k", [([1], 256, 128, 128), ([0, 3, 0], 512, 136, 272), ([256, 512], 1024, 264, 520),
                                          ([7, 0, 300, 16, 33], 1536, 130, 256), ([900, 2, 0, 700], 2304, 520, 1032),
                                          ([1] * 70, 70 * 256 + 256, 64, 64)])
def test_grouped_gemm_fp8_wgrad(counts, m, n, k, kind):
    g = torch.Generator().manual_seed(m + n)
    experts = len(counts)
    ends, rows = offsets_of(counts, m)
    held = R.held_rows(ends, rows, m)
    fmt, dt = ("e5m2", BF) if n % 16 else ("e4m3", F16)
    a, sa = operand(n, m, kind, fmt, False, g)
    b, sb = operand(k, m, kind, "e4m3", True, g)
    a.view(torch.uint8)[:, held == 1] = 0
    a.view(torch.uint8)[:, held == 2] = 0x7F            # rows behind the last expert are not read
    b.view(torch.uint8)[:, held == 2] = 0x7F
    sa[held[::128] == 2] = float("nan")
    say("wgrad", counts[:6], m, n, k, kind)
    c = torch.full((experts, n, k), 5.0, dtype=dt, device="cuda")
    bsg.grouped_gemm_fp8_wgrad(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), ends.cuda(), c, m, n, k, experts, a_dtype=fmt)
    c, at = c.cpu(), 0
    for e in range(experts):
        end = int(ends[e])
        if end == at:
            assert bool((c[e] == 0).all())
        else:
            compare(c[e], a[:, at:end], b[:, at:end], sa[at // 128:end // 128], sb[:, at // 128:end // 128], kind, dt)
        at = end
