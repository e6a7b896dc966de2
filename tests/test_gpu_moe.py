"""GPU tests of the operators that put rows into expert order and back and
quantise them, against the 64-bit references of moe_ref.py."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF, F16, F32]
GARBAGE = -77


def say(*a):
    print(*a, flush=True)


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def routed(t, k, experts, seed, masked=0.2):
    """Uneven expert ids; some pairs name no expert, by values on both sides of the range."""
    g = gen_of(seed)
    ids = (torch.rand(t, k, generator=g) ** 2 * experts).to(torch.int32).clamp(max=experts - 1)
    off = torch.rand(t, k, generator=g) < masked
    wrong = torch.where(torch.rand(t, k, generator=g) < 0.5, torch.tensor(-1), torch.tensor(experts)).to(torch.int32)
    return torch.where(off, wrong, ids)


def sort_gpu(ids, experts, m, pair_of=True, extra_ws=0):
    t, k = ids.shape
    dev = dict(device="cuda", dtype=torch.int32)
    out = [torch.full((experts,), GARBAGE, **dev), torch.full((experts,), GARBAGE, **dev), torch.full((t, k), GARBAGE, **dev),
           torch.full((m,), GARBAGE, **dev) if pair_of else None]
    ws = torch.empty(bsg.workspace_bytes("moe_sort", t, k, experts) + extra_ws, dtype=torch.uint8, device="cuda")
    bsg.moe_sort(ids.cuda(), *out, t, k, experts, m, workspace=ws)
    return out


@pytest.mark.parametrize("t,k,experts", [
    (0, 2, 3), (1, 1, 1), (1, 8, 64), (16, 8, 64), (33, 3, 5), (257, 2, 1), (256, 1, 2), (100, 64, 1024), (4096, 2, 7),
    (2049, 4, 33), (4097, 1, 1),
    (8193, 1, 256), (4001, 8, 64), (20000, 8, 128), (70001, 2, 1024), (66000, 2, 2), (300001, 1, 600)])
def test_sort(t, k, experts):
    say("sort", t, k, experts)
    ids = routed(t, k, experts, seed=t + k)
    m = bsg.moe_rows(t, k, experts) + 256
    want = R.sort(ids, experts, m)
    got = sort_gpu(ids, experts, m)
    for name, a, b in zip(("padded_offsets", "expert_rows", "row_of", "pair_of"), got, want):
        assert torch.equal(a.cpu(), b), name
    if t:
        for a, b in zip(sort_gpu(ids, experts, m, pair_of=False)[:3], want):
            assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("t,k,experts,kind", [(5000, 4, 16, "one"), (5000, 4, 16, "none"), (1, 4, 4, "twice"), (9000, 1, 3, "last")])
def test_sort_of_uneven_ids(t, k, experts, kind):
    """Every pair to one expert, no pair at all, a token that names an expert
    more than once, and the pairs at the end alone."""
    ids = torch.full((t, k), {"one": 5, "none": -1, "twice": 2, "last": 7}[kind], dtype=torch.int32)
    if kind == "last":
        ids[-1] = experts - 1
    m = bsg.moe_rows(t, k, experts)
    for a, b in zip(sort_gpu(ids, experts, m), R.sort(ids, experts, m)):
        assert torch.equal(a.cpu(), b)


def problem(t, k, experts, hidden, dt, seed):
    g = gen_of(seed)
    ids = routed(t, k, experts, seed)
    m = R.moe_rows(t, k, experts) + 256
    ends, rows, row_of, _ = R.sort(ids, experts, m)
    return dict(g=g, m=m, ends=ends, rows=rows, row_of=row_of, kind=R.held_rows(ends, rows, m),
                x=torch.randn(t, hidden, generator=g).to(dt), w=torch.rand(t, k, generator=g))


SHAPES = [(1, 1, 1, 16), (1, 8, 64, 256), (16, 8, 64, 7168), (33, 3, 5, 48), (300, 2, 4, 4096 + 16), (1003, 4, 9, 128),
          (130, 64, 1024, 64)]


@pytest.mark.parametrize("pad", [True, False])
@pytest.mark.parametrize("out", ["same", "e4m3"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,k,experts,hidden", SHAPES)
def test_gather(t, k, experts, hidden, dt, out, pad):
    say("gather", t, k, experts, hidden, dt, out, pad)
    p = problem(t, k, experts, hidden, dt, seed=t)
    m, kind = p["m"], p["kind"]
    if out == "same":
        y = torch.full((m, hidden), 3.0, dtype=dt, device="cuda")
        scale = None
    else:
        y = torch.full((m, hidden), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scale = torch.full((-(-hidden // 128), m), 3.0, device="cuda")
    prob = torch.full((m,), 3.0, device="cuda")
    old_y, old_s, old_p = y.cpu().clone(), None if scale is None else scale.cpu().clone(), prob.cpu().clone()
    bsg.moe_gather(p["x"].cuda(), p["row_of"].cuda(), p["ends"].cuda(), p["rows"].cuda(), p["w"].cuda(), y, scale, prob, t,
                   hidden, k, experts, m, zero_pad=pad)
    pairs = p["row_of"].reshape(-1)
    use = pairs >= 0
    rows, tok = pairs[use].long(), (torch.arange(t * k) // k)[use]
    if pad:
        old_p[kind == 1] = 0
    old_p[rows] = p["w"].reshape(-1)[use]
    assert torch.equal(prob.cpu(), old_p)
    if out == "same":
        if pad:
            old_y[kind == 1] = 0
        old_y[rows] = p["x"][tok]
        assert torch.equal(y.cpu(), old_y)
        return
    q, s = R.quant(p["x"][None], "e4m3", False)
    bytes_ = old_y.view(torch.uint8)
    if pad:
        bytes_[kind == 1] = 0
        old_s[:, kind == 1] = float(R.quant(torch.zeros(1, 1, 16), "e4m3", False)[1])
    bytes_[rows] = q[0].view(torch.uint8)[tok]
    old_s[:, rows] = s[0][:, tok]
    assert torch.equal(y.cpu().view(torch.uint8), bytes_) and torch.equal(scale.cpu(), old_s)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,k,experts,hidden", SHAPES)
def test_combine_and_gather_bwd(t, k, experts, hidden, dt):
    say("combine", t, k, experts, hidden, dt)
    p = problem(t, k, experts, hidden, dt, seed=t + 1)
    m = p["m"]
    y = torch.randn(m, hidden, generator=p["g"]).to(dt)
    y[p["kind"] != 0] = float("nan")             # rows that no pair has are not read
    dprob = torch.randn(m, generator=p["g"])
    yg, rows = y.cuda(), p["row_of"].cuda()
    for w in (p["w"], None):
        out = torch.full((t, hidden), GARBAGE, dtype=dt, device="cuda")
        bsg.moe_combine(yg, rows, None if w is None else w.cuda(), out, t, hidden, k, m)
        ref, mag = R.combine64(y, p["row_of"], w)
        R.check("out", out.cpu(), ref, (k + 2) * R.E * mag, dt)
    dx = torch.full((t, hidden), GARBAGE, dtype=dt, device="cuda")
    dw = torch.full((t, k), GARBAGE, device="cuda", dtype=F32)
    bsg.moe_gather_bwd(yg, dprob.cuda(), rows, dx, dw, t, hidden, k, m)
    assert torch.equal(dx, out)
    use = p["row_of"] >= 0
    assert torch.equal(dw.cpu(), torch.where(use, dprob[p["row_of"].clamp(min=0).long()], torch.zeros(())))
    dx2, dw2 = torch.zeros_like(dx), torch.zeros_like(dw)
    bsg.moe_gather_bwd(yg, None, rows, dx2, None, t, hidden, k, m)
    bsg.moe_gather_bwd(None, dprob.cuda(), rows, None, dw2, t, hidden, k, m, dtype=dt)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,k,experts,hidden", SHAPES)
def test_combine_bwd(t, k, experts, hidden, dt):
    say("combine_bwd", t, k, experts, hidden, dt)
    p = problem(t, k, experts, hidden, dt, seed=t + 2)
    m, kind = p["m"], p["kind"]
    y = torch.randn(m, hidden, generator=p["g"]).to(dt)
    y[kind != 0] = float("nan")
    dout, rows = p["x"], p["row_of"].cuda()
    ref_y, ref_w, mag = R.combine_bwd64(dout, y, p["row_of"], p["w"])
    for pad in (True, False):
        dy = torch.full((m, hidden), 3.0, dtype=dt, device="cuda")
        dw = torch.full((t, k), GARBAGE, device="cuda", dtype=F32)
        bsg.moe_combine_bwd(dout.cuda(), y.cuda(), rows, p["ends"].cuda(), p["rows"].cuda(), p["w"].cuda(), dy, dw, t,
                            hidden, k, experts, m, zero_pad=pad)
        R.check("dweight", dw.cpu(), ref_w, (hidden + 1) * R.E * mag, F32)
        want = ref_y.clone()
        want[kind == 2 if pad else kind != 0] = 3.0
        R.check("dy", dy.cpu(), want, R.E * want.abs(), dt)
    # each half alone, and the gradient in place of the rows, have the same bits
    alone_y, alone_w, place = torch.full_like(dy, 3.0), torch.zeros_like(dw), y.cuda()
    args = (rows, p["ends"].cuda(), p["rows"].cuda(), p["w"].cuda())
    bsg.moe_combine_bwd(dout.cuda(), None, *args, alone_y, None, t, hidden, k, experts, m, zero_pad=False)
    bsg.moe_combine_bwd(dout.cuda(), y.cuda(), *args, None, alone_w, t, hidden, k, experts, m)
    assert torch.equal(alone_y, dy) and torch.equal(alone_w, dw)
    bsg.moe_combine_bwd(dout.cuda(), place, *args, place, alone_w.zero_(), t, hidden, k, experts, m, zero_pad=False)
    assert torch.equal(place[kind.cuda() == 0], dy[kind.cuda() == 0]) and torch.equal(alone_w, dw)


def test_maps_that_point_outside_are_no_rows():
    """Values past m, as an offset map of a larger buffer may hold, are no rows."""
    t, k, h, m = 5, 2, 64, 256
    rows = torch.tensor([[0, 256], [1 << 30, -5], [7, 255], [-(1 << 31), 3], [2147483647, 8]], dtype=torch.int32)
    y = torch.randn(m, h, generator=gen_of(1))
    w = torch.rand(t, k, generator=gen_of(2))
    out = torch.empty(t, h, device="cuda")
    bsg.moe_combine(y.cuda(), rows.cuda(), w.cuda(), out, t, h, k, m)
    ref, mag = R.combine64(y, rows, w)
    R.check("out", out.cpu(), ref, (k + 2) * R.E * mag, F32)
    got = torch.zeros(m, h, device="cuda")
    ends = torch.tensor([256], dtype=torch.int32, device="cuda")
    bsg.moe_gather(y[:t].cuda().contiguous(), rows.cuda(), ends, ends, None, got, None, None, t, h, k, 1, m, zero_pad=False)
    want = torch.zeros(m, h)
    for i, r in enumerate(rows.reshape(-1).tolist()):
        if 0 <= r < m:
            want[r] = y[i // k]
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("l,m,k", [(1, 1, 16), (1, 16, 128), (2, 144, 272), (1, 128, 4096), (3, 16, 2048), (1, 1008, 400),
                                   (1, 7, 7168)])
def test_quant_fp8(l, m, k, dt, fmt, tile):
    say("quant_fp8", l, m, k, dt, fmt, tile)
    g = gen_of(m + k)
    x = torch.randn(l, m, k, generator=g) * torch.exp(4 * torch.randn(l, m, 1, generator=g))
    x[:, :, :: max(1, k // 5)] *= 30
    x[0, m // 2] = 0                                 # a row of zeros
    if dt == F16:
        x = x.clamp(-60000, 60000)
    x = x.to(dt)
    dev = dict(device="cuda")
    mb, kb = -(-m // 128), -(-k // 128)
    cols = m % 16 == 0
    q = torch.full((l, m, k), 1, dtype=torch.uint8, **dev).view(R.FP8[fmt])
    scale = torch.full((l, mb, kb) if tile else (l, kb, m), 3.0, **dev)
    q_t = torch.full((l, k, m), 1, dtype=torch.uint8, **dev) if cols else None
    scale_t = torch.full((l, kb, mb) if tile else (l, mb, k), 3.0, **dev) if cols else None
    bsg.quant_fp8(x.cuda(), q, scale, q_t, scale_t, m, k, l=l, tile=tile, q_dtype=fmt)
    want_q, want_s = R.quant(x, fmt, tile)
    assert torch.equal(scale.cpu(), want_s) and torch.equal(q.cpu().view(torch.uint8), want_q.view(torch.uint8))
    if not cols:
        return
    want_q, want_s = R.quant(x.transpose(1, 2).contiguous(), fmt, tile)
    assert torch.equal(scale_t.cpu(), want_s) and torch.equal(q_t.cpu(), want_q.view(torch.uint8))
    # either output alone
    for one in (0, 1):
        a, b = torch.zeros_like(q_t if one else q), torch.zeros_like(scale_t if one else scale)
        args = (None, None, a, b) if one else (a, b, None, None)
        bsg.quant_fp8(x.cuda(), *args, m, k, l=l, tile=tile, q_dtype=fmt)
        assert torch.equal(a.view(torch.uint8), (q_t if one else q).view(torch.uint8)) and torch.equal(b, scale_t if one else scale)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quant_fp8_of_every_value_of_a_type(fmt):
    """All finite fp16 values, beside a largest one that scales them so that
    they meet the codes' steps and borders from both sides."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(F16)
    v = bits[torch.isfinite(bits)]
    v = v[: len(v) // 127 * 127].reshape(1, -1, 127)
    for top in (65504.0, 448.0, 57344.0, 1.0, 0.3333):
        x = torch.cat([torch.full((1, v.shape[1], 1), top, dtype=F16), v], 2).clamp(-top, top)
        x = torch.cat([x, x.new_zeros(1, -x.shape[1] % 16, 128)], 1)
        m = x.shape[1]
        q = torch.empty(1, m, 128, dtype=R.FP8[fmt], device="cuda")
        s = torch.empty(1, 1, m, device="cuda")
        bsg.quant_fp8(x.cuda(), q, s, None, None, m, 128, q_dtype=fmt)
        want_q, want_s = R.quant(x, fmt, False)
        assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu().view(torch.uint8), want_q.view(torch.uint8))


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_quant_fp8_of_infinities(value, tile):
    """A group that holds one has codes 0 and a scale that is not finite; the other groups keep theirs."""
    x = torch.randn(1, 144, 272, generator=gen_of(9))
    x[0, 130, 5] = value
    q, q_t = (torch.empty(1, 144, 272, dtype=torch.float8_e4m3fn, device="cuda"),
              torch.empty(1, 272, 144, dtype=torch.float8_e4m3fn, device="cuda"))
    s, s_t = ((torch.empty(1, 2, 3, device="cuda"), torch.empty(1, 3, 2, device="cuda")) if tile else
              (torch.empty(1, 3, 144, device="cuda"), torch.empty(1, 2, 272, device="cuda")))
    bsg.quant_fp8(x.cuda(), q, s, q_t, s_t, 144, 272, tile=tile)
    for got_q, got_s, src in ((q, s, x), (q_t, s_t, x.transpose(1, 2).contiguous())):
        want_q, want_s = R.quant(src, "e4m3", tile)
        assert torch.equal(got_q.cpu().view(torch.uint8), want_q.view(torch.uint8))
        bad = ~torch.isfinite(want_s)
        assert int(bad.sum()) == 1 and torch.equal(got_s.cpu()[~bad], want_s[~bad])
        odd = got_s.cpu()[bad]
        assert bool(torch.isnan(odd).all()) if value != value else bool((odd == float("inf")).all())
