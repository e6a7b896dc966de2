"""GPU tests of ranges of rows that a program lays out itself, longer than an
expert's pairs by more than 256: every row behind the pairs is padding."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R

pytestmark = pytest.mark.gpu
BF, E4M3, DEV = torch.bfloat16, torch.float8_e4m3fn, "cuda"
T, K, E = 300, 2, 4
HELD, ENDS, M = [299, 1, 0, 300], [1024, 1280, 2048, 3328], 3584


def layout():
    """row_of of T tokens for experts of HELD rows from each range's beginning."""
    begin = [0, *ENDS[:-1]]
    rows = torch.tensor([b + i for b, n in zip(begin, HELD) for i in range(n)], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    row_of = rows[torch.randperm(T * K, generator=g)].reshape(T, K)
    ends, held = torch.tensor(ENDS, dtype=torch.int32), torch.tensor(HELD, dtype=torch.int32)
    return row_of, ends, held, R.held_rows(ends, held, M), g


@pytest.mark.parametrize("hidden", [16, 1032, 7168])
@pytest.mark.parametrize("dt", [torch.float32, BF])
def test_padding_behind_the_pairs(hidden, dt):
    print("capacity", hidden, dt, flush=True)
    row_of, ends, held, kind, g = layout()
    x, w = torch.randn(T, hidden, generator=g).to(dt), torch.rand(T, K, generator=g)
    token = torch.zeros(M, dtype=torch.long)
    token[row_of.reshape(-1).long()] = torch.arange(T).repeat_interleave(K)
    prob = torch.where(kind == 0, 0.0, torch.where(kind == 1, 0.0, 5.0))
    prob[row_of.reshape(-1).long()] = w.reshape(-1)
    want = torch.where((kind == 0)[:, None], x[token], torch.where(kind == 1, 0.0, 5.0)[:, None].to(dt))
    y, p = torch.full((M, hidden), 5.0, dtype=dt, device=DEV), torch.full((M,), 5.0, device=DEV)
    dev = [v.cuda() for v in (row_of, ends, held, w)]
    bsg.moe_gather(x.cuda(), *dev, y, None, p, T, hidden, K, E, M)
    assert torch.equal(y.cpu(), want) and torch.equal(p.cpu(), prob)
    dy = torch.full((M, hidden), 5.0, dtype=dt, device=DEV)
    bsg.moe_combine_bwd(x.cuda(), None, *dev[:3], None, dy, None, T, hidden, K, E, M)
    assert torch.equal(dy.cpu(), want)
    if hidden % 16 == 0:
        q, s = torch.full((M, hidden), 5.0, device=DEV).to(E4M3), torch.full((-(-hidden // 128), M), 5.0, device=DEV)
        bsg.moe_gather(x.cuda(), *dev, q, s, p, T, hidden, K, E, M)
        cq, cs = R.quant(x[None], "e4m3", False)
        wq = torch.where((kind == 0)[:, None], cq[0][token].float(), torch.where(kind == 1, 0.0, 5.0)[:, None])
        ws = torch.where((kind == 0)[None], cs[0][:, token], torch.where(kind == 1, torch.tensor(2.0 ** -100) / 448, 5.0)[None])
        assert torch.equal(q.cpu().float(), wq) and torch.equal(s.cpu(), ws) and torch.equal(p.cpu(), prob)


@pytest.mark.parametrize("max_rows", [0, 16, 64])
def test_products_of_long_ranges(max_rows):
    """The grouped product takes the pairs' rows and leaves the others; the weights' gradient adds zeros."""
    n, k = 264, 400
    print("products of long ranges", max_rows, bsg.plan_string("grouped_gemm_fp8", M, n, k, num_experts=E, max_rows=max_rows), flush=True)
    _, ends, held, kind, g = layout()
    code = lambda *s: torch.randint(-4, 5, s, generator=g).float().to(E4M3)  # noqa: E731
    power = lambda *s: torch.exp2(torch.randint(-1, 2, s, generator=g).float())  # noqa: E731
    a, sa, b, sb = code(M, k), power(4, M), code(E, n, k), power(E, 3, 4)
    c = torch.full((M, n), 5.0, dtype=BF, device=DEV)
    bsg.grouped_gemm_fp8(a.cuda(), b.cuda(), sa.cuda(), sb.cuda(), ends.cuda(), held.cuda(), c, M, n, k, E, max_rows=max_rows)
    dy, sdy, x, sx = code(n, M), power(M // 128, n), code(k, M), power(4, M // 128)
    dy.view(torch.uint8)[:, kind == 1] = 0
    dw = torch.empty(E, n, k, dtype=BF, device=DEV)
    bsg.grouped_gemm_fp8_wgrad(dy.cuda(), x.cuda(), sdy.cuda(), sx.cuda(), ends.cuda(), dw, M, n, k, E)
    c, dw, at = c.cpu(), dw.cpu(), 0
    for e, (end, rows) in enumerate(zip(ENDS, HELD)):
        r = slice(at, at + rows)
        assert torch.equal(c[r], R.gemm64(a[r], b[e], sa[:, r], sb[e])[0].to(BF)) and bool((c[at + rows:end] == 5).all())
        r = slice(at, end)
        assert torch.equal(dw[e], R.gemm64(dy[:, r], x[:, r], sdy[at // 128:end // 128], sx[:, at // 128:end // 128])[0].to(BF))
        at = end
    assert bool((c[at:] == 5).all())
