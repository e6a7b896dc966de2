"""GPU tests of kernel forms of the 8-bit float products that take large or
particular sizes, each held to the form that the launch chooses: the kernel of
up to 32 rows of an expert, and the largest tile with sums of fewer blocks than
its ring has slots.  References and bounds as in test_gpu_fp8.py."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R
from test_gpu_fp8 import BF, F16, compare, offsets_of, operand, say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def experts_of(count, n, k, kind, g):
    each = [[v.cuda() for v in operand(n, k, kind, "e4m3", True, g)] for _ in range(count)]
    return each, torch.stack([x[0] for x in each]), torch.stack([x[1] for x in each])


def compare_experts(c, counts, ends, each, a, sa, kind, dt):
    """The rows of each expert, and that the others are as they were."""
    at = 0
    for e, (x, s) in enumerate(each):
        last, end = at + counts[e], int(ends[e])
        if counts[e]:
            compare(c[at:last], a[at:last], x, sa[:, at:last], s, kind, dt, f"expert {e}")
        assert bool((c[last:end] == 5).all())
        at = end
    assert bool((c[at:] == 5).all())


@pytest.mark.parametrize("kind", ["whole", "random"])
@pytest.mark.parametrize("counts,m", [([40, 0, 35], 768), ([33, 0, 64, 17, 1, 40], 1536), ([64] * 9, 2304),
                                      ([20, 32, 0, 31, 0, 0, 47, 1, 60, 64, 33], 2816), ([256, 100], 512)])
@pytest.mark.parametrize("n,k", [(1032, 1040), (136, 272), (520, 7168), (24, 16)])
def test_grouped_few_rows_by_32(counts, m, n, k, kind):
    """Experts of up to 32 rows, of more, and of more than the caller said."""
    experts = len(counts)
    g = torch.Generator().manual_seed(m + n)
    ends, rows = offsets_of(counts, m)
    fmt, dt = ("e4m3", BF) if (experts + n) % 16 else ("e5m2", F16)
    a, sa = (v.cuda() for v in operand(m, k, kind, fmt, False, g))
    each, b, sb = experts_of(experts, n, k, kind, g)
    held = R.held_rows(ends, rows, m).cuda()
    # rows that hold no pair are not read
    dirty, dirty_s = a.clone(), sa.clone()
    dirty.view(torch.uint8)[held != 0] = 0x7F
    dirty_s[:, held != 0] = float("nan")
    for max_rows in (17, 33, 64):
        assert bsg.plan_string("grouped_gemm_fp8", m, n, k, num_experts=experts, max_rows=max_rows) == "few 32"
        say("few 32", counts[:6], m, n, k, kind, max_rows)
        c = torch.full((m, n), 5.0, dtype=dt, device=DEV)
        bsg.grouped_gemm_fp8(dirty, b, dirty_s, sb, ends.cuda(), rows.cuda(), c, m, n, k, experts, max_rows=max_rows, a_dtype=fmt)
        compare_experts(c, counts, ends, each, a, sa, kind, dt)


@pytest.mark.parametrize("max_rows", [12, 40])
@pytest.mark.parametrize("n,k", [(264, 16416), (8216, 16)])
def test_grouped_few_rows_past_four_gib(n, k, max_rows):
    """The last expert's rows begin past 4 GiB of A and its weight past 4 GiB of B, or its rows past 4 GiB of C."""
    m, experts = 1 << 18, 1024
    assert bsg.plan_string("grouped_gemm_fp8", m, n, k, num_experts=experts, max_rows=max_rows) == ("few 16" if max_rows < 17 else "few 32")
    assert (m - 256) * k > 1 << 32 and (experts - 1) * n * k > 1 << 32 or (m - 256) * n * 2 > 1 << 32
    say("few rows past 4 GiB", n, k, max_rows)
    g = torch.Generator().manual_seed(9)
    a, b = (torch.zeros(*s, dtype=torch.float8_e4m3fn, device=DEV) for s in ((m, k), (experts, n, k)))
    kb = -(-k // 128)
    sa, sb = torch.zeros(kb, m, device=DEV), torch.zeros(experts, -(-n // 128), kb, device=DEV)
    c = torch.full((m, n), 5.0, dtype=BF, device=DEV)
    rows = torch.zeros(experts, dtype=torch.int32)
    want = {}
    for e, count in ((0, 1), (511, min(max_rows, 33)), (experts - 1, max_rows)):
        x, sx = (v.cuda() for v in operand(count, k, "whole", "e4m3", False, g))
        w, sw = (v.cuda() for v in operand(n, k, "whole", "e4m3", True, g))
        at = slice(256 * e, 256 * e + count)
        a[at], sa[:, at], b[e], sb[e], rows[e] = x, sx, w, sw, count
        want[e] = (R.values(x, sx, False) @ R.values(w, sw, True).t()).to(BF)
    ends = 256 * torch.arange(1, experts + 1, dtype=torch.int32)
    bsg.grouped_gemm_fp8(a, b, sa, sb, ends.cuda(), rows.cuda(), c, m, n, k, experts, max_rows=max_rows)
    for e, y in want.items():
        at = slice(256 * e, 256 * e + len(y))
        assert torch.equal(c[at], y)
        c[at] = 5.0
    assert bool((c == 5).all())


@pytest.mark.parametrize("fmt,dt", [("e4m3", BF), ("e5m2", F16)])
@pytest.mark.parametrize("m,n,k", [(65536, 4096, 144), (65505, 4072, 240), (64001, 4080, 256)])
def test_short_sums_in_the_largest_tile(m, n, k, fmt, dt):
    """Two blocks, the second short or whole; one round of tiles follows the other in the ring.  (One block
    takes the smaller tiles: test_moe_plan.py.)"""
    assert bsg.plan_string("gemm_fp8", m, n, k) == "Big"
    say("short sums in the largest tile", m, n, k, fmt, dt)
    g = torch.Generator().manual_seed(k)
    a, sa = (v.cuda() for v in operand(m, k, "whole", fmt, False, g))
    b, sb = (v.cuda() for v in operand(n, k, "whole", "e4m3", True, g))
    c = torch.full((m + 2, n), 5.0, dtype=dt, device=DEV)
    bsg.gemm_fp8(a, b, sa, sb, c[1:-1], m, n, k, a_dtype=fmt)
    assert torch.equal(c[1:-1], (R.values(a, sa, False) @ R.values(b, sb, True).t()).to(dt))
    assert bool((c[0] == 5).all()) and bool((c[-1] == 5).all())


@pytest.mark.parametrize("use_rows", [True, False])
@pytest.mark.parametrize("fmt,dt", [("e4m3", F16), ("e5m2", BF)])
def test_grouped_short_sums_in_the_largest_tile(fmt, dt, use_rows):
    m, n, k, counts = 65536, 4096, 144, [20000, 0, 1, 44000, 300]
    assert bsg.plan_string("grouped_gemm_fp8", m, n, k, num_experts=5, expert_rows=use_rows) == "Big"
    say("grouped short sums in the largest tile", fmt, dt, use_rows)
    g = torch.Generator().manual_seed(11)
    ends, rows = offsets_of(counts, m)
    a, sa = (v.cuda() for v in operand(m, k, "whole", fmt, False, g))
    each, b, sb = experts_of(5, n, k, "whole", g)
    c = torch.full((m, n), 5.0, dtype=dt, device=DEV)
    bsg.grouped_gemm_fp8(a, b, sa, sb, ends.cuda(), rows.cuda() if use_rows else None, c, m, n, k, 5, a_dtype=fmt)
    have = counts if use_rows else [int(e) - int(s) for s, e in zip([0, *ends[:-1]], ends)]
    compare_experts(c, have, ends, each, a, sa, "whole", dt)


@pytest.mark.parametrize("kind", ["whole", "random"])
@pytest.mark.parametrize("fmt,dt", [("e4m3", BF), ("e4m3", F16), ("e5m2", F16)])
def test_wgrad_of_few_blocks_in_the_largest_tile(fmt, dt, kind):
    """Sums of 2, 0, 6 and 8 blocks, and rows behind the last expert."""
    counts, m, n, k = [256, 0, 700, 900], 2304, 4104, 4088
    assert bsg.plan_string("grouped_gemm_fp8_wgrad", m, n, k, num_experts=4) == "Big"
    say("wgrad of few blocks", fmt, dt, kind)
    g = torch.Generator().manual_seed(12)
    ends, rows = offsets_of(counts, m)
    held = R.held_rows(ends, rows, m)
    a, sa = operand(n, m, kind, fmt, False, g)
    b, sb = operand(k, m, kind, "e4m3", True, g)
    a.view(torch.uint8)[:, held == 1] = 0
    a.view(torch.uint8)[:, held == 2] = 0x7F            # rows behind the last expert are not read
    b.view(torch.uint8)[:, held == 2] = 0x7F
    sa[held[::128] == 2] = float("nan")
    a, sa, b, sb = a.cuda(), sa.cuda(), b.cuda(), sb.cuda()
    c = torch.full((len(counts), n, k), 5.0, dtype=dt, device=DEV)
    bsg.grouped_gemm_fp8_wgrad(a, b, sa, sb, ends.cuda(), c, m, n, k, len(counts), a_dtype=fmt)
    at = 0
    for e, end in enumerate(ends.tolist()):
        if end == at:
            assert bool((c[e] == 0).all())
        else:
            compare(c[e], a[:, at:end], b[:, at:end], sa[at // 128:end // 128], sb[:, at // 128:end // 128], kind, dt)
        at = end
