"""GPU tests of the expert operators on a batch without tokens, as a rank that
is sent none runs them: every tensor at its size, some without elements."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg

pytestmark = pytest.mark.gpu
BF, F32, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
K, E, H = 2, 3, 256


def full(*shape, dtype=F32, value=5.0):
    return torch.full(shape, value, device="cuda").to(dtype)


@pytest.mark.parametrize("m", [0, 512])
def test_layer_of_no_tokens(m):
    """m = 0 is what moe_rows asks for; a program may hold more."""
    print("no tokens", m, flush=True)
    assert bsg.moe_rows(0, K, E) == 0
    x, ids, w = full(0, H, dtype=BF), full(0, K, dtype=I32), full(0, K)
    ends, held, row_of, pair_of = full(E, dtype=I32), full(E, dtype=I32), full(0, K, dtype=I32), full(m, dtype=I32)
    bsg.moe_sort(ids, ends, held, row_of, pair_of, 0, K, E, m)
    assert bool((ends == 0).all()) and bool((held == 0).all()) and bool((pair_of == -1).all())
    y, prob = full(m, H, dtype=BF), full(m)
    bsg.moe_gather(x, row_of, ends, held, w, y, None, prob, 0, H, K, E, m)
    q, scale = full(m, H, dtype=E4M3), full(H // 128, m)
    bsg.moe_gather(x, row_of, ends, held, w, q, scale, prob, 0, H, K, E, m)
    b, sb, c = full(E, 64, H, dtype=E4M3), full(E, 1, H // 128), full(m, 64, dtype=BF)
    bsg.grouped_gemm_fp8(q, b, scale, sb, ends, held, c, m, 64, H, E, max_rows=0)
    out = full(0, H, dtype=BF)
    bsg.moe_combine(y, row_of, w, out, 0, H, K, m)
    dy, dw = full(m, H, dtype=BF), full(0, K)
    bsg.moe_combine_bwd(out, y, row_of, ends, held, w, dy, dw, 0, H, K, E, m)
    bsg.moe_gather_bwd(dy, prob, row_of, x, dw, 0, H, K, m)
    grad = full(E, 64, H, dtype=BF)
    bsg.grouped_gemm_fp8_wgrad(full(64, m, dtype=E4M3), full(H, m, dtype=E4M3), full(m // 128, 64), full(H // 128, m // 128), ends,
                               grad, m, 64, H, E)
    assert bool((grad == 0).all())
    # no range has rows: what lies behind them all stays
    assert all(bool((t.float() == 5).all()) for t in (y, prob, q, scale, c, dy))


def test_padding_of_no_tokens():
    """Ranges of padding alone, with weights and codes."""
    m, ends, held = 768, torch.tensor([256, 256, 512], dtype=I32, device="cuda"), full(E, dtype=I32, value=0)
    x, row_of, w = full(0, H, dtype=BF), full(0, K, dtype=I32), full(0, K)
    q, scale, prob = full(m, H, dtype=E4M3), full(H // 128, m), full(m)
    print("padding of no tokens", flush=True)
    bsg.moe_gather(x, row_of, ends, held, w, q, scale, prob, 0, H, K, E, m)
    least = torch.tensor(2.0 ** -100) / 448
    assert bool((q[:512].float() == 0).all()) and bool((scale[:, :512] == least.cuda()).all()) and bool((prob[:512] == 0).all())
    assert bool((q[512:].float() == 5).all()) and bool((scale[:, 512:] == 5).all()) and bool((prob[512:] == 5).all())


def test_tokens_without_rows():
    """A rank whose experts nobody asked for, with no rows at all: zeros."""
    t, y, row_of = 3, full(0, H, dtype=BF), full(3, K, dtype=I32, value=-1)
    dx, dw, out = full(t, H, dtype=BF), full(t, K), full(t, H, dtype=BF)
    print("no rows", flush=True)
    bsg.moe_gather(full(t, H, dtype=BF), row_of, None, None, full(t, K), y, None, full(0), t, H, K, E, 0)
    bsg.moe_combine(y, row_of, full(t, K), out, t, H, K, 0)
    bsg.moe_gather_bwd(y, full(0), row_of, dx, dw, t, H, K, 0)
    assert bool((out == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all())
    dw.fill_(5)
    bsg.moe_combine_bwd(out, y, row_of, None, None, full(t, K), y, dw, t, H, K, E, 0)
    assert bool((dw == 0).all())
