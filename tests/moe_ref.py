"""Plain implementation of the expert operators in 64 bits, and the error
bounds that their kernels have to keep.  Tensors live on the CPU.

Bounds, with E = 2^-24 (one fp32 rounding):
  * an fp32 sum of K products, fused or not, is off by at most (K + 1) E
    sum|products|, whatever its order;
  * an output is that sum rounded once (ffn_ref.out_bound);
  * the 8-bit matrix instruction drops, of each 8 products, the bits below
    2^-13 of the largest (tests/test_gpu_mfma_precision.py): under 7 * 2^-13 of
    the 8's sum of magnitudes.  Both scales are multiplied in fp32 (one
    rounding), a block's sum meets them and the accumulator in a fused step:
    with B blocks (B + 3) E of the sum of magnitudes.
quant_fp8 is defined by three fp32 operations and a cast, which the reference
repeats: its results are equal bit for bit.
"""
import torch

from ffn_ref import E, check, out_bound  # noqa: F401

MAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def moe_rows(tokens, top_k, experts):
    pairs = tokens * top_k
    return (pairs + 255 * min(experts, pairs)) // 256 * 256


def sort(ids, experts, m):
    """(padded_offsets, expert_rows, row_of, pair_of) by lists."""
    flat = ids.reshape(-1).tolist()
    held = [[p for p, e in enumerate(flat) if e == x] for x in range(experts)] if experts < 40 else None
    if held is None:
        held = [[] for _ in range(experts)]
        for p, e in enumerate(flat):
            if 0 <= e < experts:
                held[e].append(p)
    row_of, pair_of, ends, at = [-1] * len(flat), [-1] * m, [], 0
    for pairs in held:
        for i, p in enumerate(pairs):
            row_of[p], pair_of[at + i] = at + i, p
        at += -(-len(pairs) // 256) * 256
        ends.append(at)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(ends), i32([len(v) for v in held]), i32(row_of).reshape(ids.shape), i32(pair_of)


def held_rows(ends, rows, m):
    """0 for a row that holds a pair, 1 for one of an expert's range that does not, 2 behind them all."""
    kind, at = torch.full((m,), 2, dtype=torch.int64), 0
    for end, n in zip(ends.tolist(), rows.tolist()):
        kind[at:end] = 1
        kind[at:at + n] = 0
        at = end
    return kind


def on(row_of, m):
    return (row_of >= 0) & (row_of < m)


def combine64(y, row_of, weight):
    """sum_j weight y[row], and the sum of magnitudes."""
    m, (t, k) = y.shape[0], row_of.shape
    out = torch.zeros(t, y.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for j in range(k):
        use = on(row_of[:, j], m)
        v = y[row_of[use, j].long()].double()
        if weight is not None:
            v = v * weight[use, j].double()[:, None]
        out[use] += v
        mag[use] += v.abs()
    return out, mag


def combine_bwd64(dout, y, row_of, weight):
    """(dy, dweight, sum of magnitudes of dweight); dy is 0 where no pair is."""
    m, (t, k) = y.shape[0], row_of.shape
    dy = torch.zeros(m, dout.shape[1], dtype=torch.float64)
    dw = torch.zeros(t, k, dtype=torch.float64)
    mag = torch.zeros_like(dw)
    for j in range(k):
        use = on(row_of[:, j], m)
        r, d = row_of[use, j].long(), dout[use].double()
        w = torch.ones(len(r), dtype=torch.float64) if weight is None else weight[use, j].double()
        dy[r] = w[:, None] * d
        p = d * y[r].double()
        dw[use, j], mag[use, j] = p.sum(1), p.abs().sum(1)
    return dy, dw, mag


def quant(x, fmt, tile):
    """(codes, scale) of x (l, m, k), along k or for each 128 x 128."""
    l, m, k = x.shape
    mb, kb = -(-m // 128), -(-k // 128)
    x = x.float()
    big = torch.zeros(l, 128 * mb, 128 * kb)
    big[:, :m, :k] = x.abs()
    g = big.reshape(l, mb, 128, kb, 128)
    top = g.amax((2, 4)) if tile else g.amax(4).reshape(l, 128 * mb, kb)[:, :m]
    top = torch.maximum(top, torch.tensor(2.0 ** -100))             # (NaN stays)
    scale, inv = top / MAX[fmt], torch.full_like(top, MAX[fmt]) / top      # (a number over a tensor would take two roundings)
    if tile:
        each = lambda v: v.repeat_interleave(128, 1)[:, :m].repeat_interleave(128, 2)[:, :, :k]  # noqa: E731
    else:
        each = lambda v: v.repeat_interleave(128, 2)[:, :, :k]  # noqa: E731
    # |x inv| is the largest code or a rounding past it
    q = torch.where(torch.isfinite(each(top)), (x * each(inv)).clamp(-MAX[fmt], MAX[fmt]), torch.zeros(())).to(FP8[fmt])
    return q, scale if tile else scale.transpose(1, 2).contiguous()


def values(q, scale, tile):
    """Codes (m, k) times their scales, in float64."""
    m, k = q.shape
    s = scale.double()
    s = s.repeat_interleave(128, 0)[:m].repeat_interleave(128, 1)[:, :k] if tile else s.repeat_interleave(128, 0)[:k].t()
    return q.double() * s


def gemm64(a, b, a_scale, b_scale):
    """a b^T in float64 and its bound before the output's rounding."""
    x, y = values(a, a_scale, False), values(b, b_scale, True)
    mag = x.abs() @ y.abs().t()
    return x @ y.t(), (7 * 2.0 ** -13 + (a.shape[1] // 128 + 4) * E) * mag
