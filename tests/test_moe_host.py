"""CPU tests of the expert operators: the host-side checks of arguments, the
sizes, and the 64-bit references against their definitions and differences
(the formulas that the GPU tests compare the kernels with)."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R

OK, NULLPTR, SHAPE, DTYPE, ALIGN, UNSUP = 0, 1, 2, 3, 4, 5
P = 0x10000   # a 16-byte aligned fake device address (validation never dereferences)
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def call(name, base):
    return lambda **kw: getattr(bsg, name)(**{**base, **kw}, validate_only=True)


sort = call("moe_sort", dict(expert=P, padded_offsets=P, expert_rows=P, row_of=P, pair_of=P, tokens=7, top_k=2,
                             num_experts=4, m=1024, workspace=P))
gather = call("moe_gather", dict(x=P, row_of=P, padded_offsets=P, expert_rows=P, weight=P, y=P, scale=None, prob=P,
                                 tokens=7, hidden=64, top_k=2, num_experts=4, m=1024, x_dtype=BF))
gather_bwd = call("moe_gather_bwd", dict(dy=P, dprob=P, row_of=P, dx=P, dweight=P, tokens=7, hidden=64, top_k=2, m=1024,
                                         dtype=BF))
combine = call("moe_combine", dict(y=P, row_of=P, weight=P, out=P, tokens=7, hidden=64, top_k=2, m=1024, dtype=F16))
combine_bwd = call("moe_combine_bwd", dict(dout=P, y=P, row_of=P, padded_offsets=P, expert_rows=P, weight=P, dy=P,
                                           dweight=P, tokens=7, hidden=64, top_k=2, num_experts=4, m=1024, dtype=F32))
quant = call("quant_fp8", dict(x=P, q=P, scale=P, q_t=P, scale_t=P, m=32, k=64, x_dtype=BF))
gemm = call("gemm_fp8", dict(a=P, b=P, a_scale=P, b_scale=P, c=P, m=5, n=64, k=64, c_dtype=BF, workspace=P))
grouped = call("grouped_gemm_fp8", dict(a=P, b=P, a_scale=P, b_scale=P, padded_offsets=P, expert_rows=P, c=P, m=1024,
                                        n=64, k=64, num_experts=4, c_dtype=BF))
wgrad = call("grouped_gemm_fp8_wgrad", dict(a=P, b=P, a_scale=P, b_scale=P, padded_offsets=P, c=P, m=1024, n=64, k=64,
                                            num_experts=4, c_dtype=F16))


@pytest.mark.parametrize("tokens,top_k,experts", [(0, 1, 1), (1, 1, 1), (1, 8, 64), (16, 8, 64), (257, 1, 2), (1000, 3, 7),
                                                  (33, 64, 1024)])
def test_moe_rows_is_the_worst_routing(tokens, top_k, experts):
    """As many experts as possible with one pair past a multiple of 256."""
    pairs = tokens * top_k
    some = min(experts, pairs)
    each = [1] * some
    left = pairs - some
    if some:
        each[0] += left // 256 * 256
        each[-1] += left % 256
    worst = sum(-(-n // 256) * 256 for n in each)
    m = bsg.moe_rows(tokens, top_k, experts)
    assert m == R.moe_rows(tokens, top_k, experts) and m % 256 == 0 and worst <= m < worst + 512


def test_moe_rows_refusals():
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1025), (1 << 23, 1, 1), (1, 65, 4)):
        with pytest.raises(bsg.BsgError):
            bsg.moe_rows(*bad)


def test_moe_sort_validation():
    assert sort() == OK and sort(pair_of=None) == OK and sort(workspace=None) == OK
    assert sort(tokens=0, expert=0, row_of=0, m=0) == OK
    assert sort(m=bsg.moe_rows(7, 2, 4)) == OK and sort(m=bsg.moe_rows(7, 2, 4) - 256) == SHAPE
    assert sort(m=1000) == SHAPE and sort(tokens=-1) == SHAPE and sort(top_k=0) == SHAPE
    assert sort(num_experts=0) == SHAPE and sort(num_experts=1025) == SHAPE
    assert sort(top_k=65, m=1 << 20) == UNSUP and sort(tokens=(1 << 22) + 1, m=1 << 29) == UNSUP and sort(m=1 << 31) == UNSUP
    assert sort(expert=0) == NULLPTR and sort(row_of=0) == NULLPTR and sort(padded_offsets=0) == NULLPTR
    assert sort(expert_rows=0) == NULLPTR
    assert sort(expert=P + 2) == ALIGN and sort(pair_of=P + 1) == ALIGN
    big = dict(tokens=1 << 16, top_k=8, m=1 << 20)
    assert bsg.workspace_bytes("moe_sort", 1 << 16, 8, 4) > 0
    assert sort(**big) == OK and sort(**big, workspace=None) == NULLPTR and sort(**big, workspace=P + 4) == ALIGN


def test_moe_gather_validation():
    assert gather() == OK and gather(weight=None, prob=None) == OK and gather(tokens=0, x=0, row_of=0) == OK
    assert gather(y_dtype="e4m3", scale=P) == OK and gather(y_dtype="e4m3") == NULLPTR and gather(scale=P) == NULLPTR
    assert gather(y_dtype=F32) == DTYPE and gather(y_dtype="e5m2", scale=P) == DTYPE and gather(x_dtype=bsg.E4M3) == DTYPE
    assert gather(weight=None) == NULLPTR and gather(prob=None) == NULLPTR
    assert gather(hidden=12) == ALIGN and gather(hidden=12, x_dtype=F32) == OK and gather(hidden=10, x_dtype=F32) == ALIGN
    assert gather(hidden=24) == OK and gather(hidden=24, y_dtype="e4m3", scale=P) == ALIGN
    assert gather(hidden=0) == SHAPE and gather(hidden=1 << 21) == UNSUP and gather(m=100) == SHAPE
    assert gather(x=0) == NULLPTR and gather(y=0) == NULLPTR and gather(row_of=0) == NULLPTR
    assert gather(expert_rows=0) == NULLPTR and gather(expert_rows=0, padded_offsets=0, zero_pad=False) == OK
    assert gather(x=P + 8) == ALIGN and gather(prob=P + 2) == ALIGN
    assert gather(m=0, y=0, x=0) == OK


def test_moe_gather_bwd_validation():
    assert gather_bwd() == OK and gather_bwd(dprob=None, dweight=None) == OK and gather_bwd(dx=None, dy=None) == OK
    assert gather_bwd(dprob=None) == NULLPTR and gather_bwd(dy=None) == NULLPTR and gather_bwd(row_of=0) == NULLPTR
    assert gather_bwd(dx=None, dprob=None, dweight=None) == NULLPTR
    assert gather_bwd(hidden=4) == ALIGN and gather_bwd(dx=P + 8) == ALIGN and gather_bwd(dweight=P + 2) == ALIGN
    assert gather_bwd(dtype=bsg.E4M3) == DTYPE and gather_bwd(m=-256) == SHAPE and gather_bwd(tokens=0, dy=0, row_of=0) == OK


def test_moe_combine_validation():
    assert combine() == OK and combine(weight=None) == OK and combine(tokens=0, y=0, out=0, row_of=0) == OK
    assert combine(m=0, y=0) == OK                       # every token becomes zero
    assert combine(y=0) == NULLPTR and combine(out=0) == NULLPTR and combine(row_of=0) == NULLPTR
    assert combine(y=P + 4) == ALIGN and combine(weight=P + 2) == ALIGN and combine(hidden=20) == ALIGN
    assert combine(dtype=bsg.E5M2) == DTYPE and combine(top_k=0) == SHAPE and combine(m=8) == SHAPE


def test_moe_combine_bwd_validation():
    assert combine_bwd() == OK and combine_bwd(dy=None) == OK and combine_bwd(dweight=None, y=None) == OK
    assert combine_bwd(dy=None, dweight=None) == NULLPTR and combine_bwd(y=None) == NULLPTR and combine_bwd(dout=0) == NULLPTR
    assert combine_bwd(weight=None) == OK
    assert combine_bwd(expert_rows=0) == NULLPTR and combine_bwd(expert_rows=0, padded_offsets=0, zero_pad=False) == OK
    assert combine_bwd(expert_rows=0, padded_offsets=0, dy=None) == OK
    assert combine_bwd(hidden=6) == ALIGN and combine_bwd(dy=P + 8) == ALIGN and combine_bwd(num_experts=2000) == SHAPE


def test_quant_fp8_validation():
    assert quant() == OK and quant(q=None, scale=None) == OK and quant(q_t=None, scale_t=None) == OK and quant(tile=True) == OK
    assert quant(l=0) == OK and quant(m=0, x=0) == OK and quant(q_dtype="e5m2") == OK
    assert quant(q=None) == NULLPTR and quant(scale_t=None) == NULLPTR and quant(x=0) == NULLPTR
    assert quant(q=None, scale=None, q_t=None, scale_t=None) == NULLPTR
    assert quant(k=40) == ALIGN and quant(m=40) == ALIGN and quant(m=40, q_t=None, scale_t=None) == OK
    assert quant(x=P + 8) == ALIGN and quant(scale=P + 2) == ALIGN and quant(q_t=P + 4) == ALIGN
    assert quant(x_dtype=bsg.E4M3) == DTYPE and quant(l=-1) == SHAPE and quant(l=1025) == UNSUP and quant(m=1 << 23) == UNSUP
    with pytest.raises(ValueError):
        quant(q_dtype="int8")
    assert bsg.lib().bsg_validate_quant_fp8(P, P, P, P, P, 1, 32, 64, 0, bsg.BF16, bsg.BF16) == DTYPE


@pytest.mark.parametrize("f", [gemm, grouped, wgrad])
def test_fp8_product_validation(f):
    assert f() == OK and f(a_dtype="e5m2") == OK and f(c_dtype=F16) == OK and f(n=0) == OK
    assert f(c_dtype=F32) == UNSUP and f(c_dtype=bsg.E4M3) == DTYPE
    for name in ("a", "b", "a_scale", "b_scale", "c"):
        assert f(**{name: 0}) == NULLPTR
    assert f(a=P + 8) == ALIGN and f(c=P + 8) == ALIGN and f(a_scale=P + 2) == ALIGN and f(b_scale=P + 1) == ALIGN
    assert f(m=-256) == SHAPE and f(n=1 << 21) == UNSUP and f(m=1 << 23) == UNSUP
    with pytest.raises(ValueError):
        f(a_dtype="e3m4")


def test_fp8_product_sizes():
    assert gemm(k=24) == ALIGN and gemm(n=12) == ALIGN and gemm(n=8, k=16) == OK and gemm(k=0, a=0, b=0, a_scale=0) == OK
    assert gemm(m=1 << 22, n=1 << 20) == UNSUP
    assert gemm(m=(1 << 22) + 1, n=8) == UNSUP and gemm(k=(1 << 20) + 16) == UNSUP and grouped(m=(1 << 22) + 256) == UNSUP
    parts = dict(m=130, n=2048, k=7168)                   # K in parts: a workspace is needed
    assert gemm(**parts) == OK and gemm(**parts, workspace=None) == NULLPTR and gemm(**parts, workspace=P + 4) == ALIGN
    assert grouped(k=24) == ALIGN and grouped(n=12) == ALIGN and grouped(m=1000) == SHAPE and grouped(num_experts=0) == SHAPE
    assert grouped(padded_offsets=0) == NULLPTR and grouped(expert_rows=None) == OK and grouped(expert_rows=P + 2) == ALIGN
    assert grouped(max_rows=-1) == SHAPE and grouped(max_rows=1 << 40) == OK and grouped(m=0, a=0, c=0) == OK
    assert wgrad(k=12) == ALIGN and wgrad(n=3) == OK and wgrad(m=1000) == SHAPE and wgrad(padded_offsets=0) == NULLPTR
    assert wgrad(m=0, a=0, b=0, a_scale=0, b_scale=0) == OK          # zeros
    assert wgrad(n=1 << 18, k=1 << 18, num_experts=1024) == UNSUP


def test_workspace_bytes():
    for t in (1, 1 << 10, 1 << 14, 1 << 22):
        assert 0 <= bsg.workspace_bytes("moe_sort", t, 8, 64) < 1 << 20
    for bad in ((-1, 8, 64), (4, 0, 64), (4, 8, 0), (4, 65, 8)):
        with pytest.raises(bsg.BsgError):
            bsg.workspace_bytes("moe_sort", *bad)
    assert bsg.workspace_bytes("gemm_fp8", 4, 64, 64) >= 0
    with pytest.raises(bsg.BsgError):
        bsg.workspace_bytes("gemm_fp8", 4, -64, 64)


def test_binding_refuses_tensors_that_do_not_fit():
    cpu = torch.zeros(4, 64, dtype=BF)
    with pytest.raises(bsg.BsgError) as e:
        gather(x=cpu)
    assert e.value.status == 6


# ---------------------------------------------------------------------------
# The references
# ---------------------------------------------------------------------------
def test_reference_sort_is_a_stable_order():
    gen = torch.Generator().manual_seed(5)
    ids = torch.randint(-2, 9, (301, 3), generator=gen, dtype=torch.int32)
    m = R.moe_rows(301, 3, 7)
    ends, rows, row_of, pair_of = R.sort(ids, 7, m)
    flat, key = row_of.reshape(-1), ids.reshape(-1)
    assert bool(((flat >= 0) == ((key >= 0) & (key < 7))).all()) and int(rows.sum()) == int((flat >= 0).sum())
    assert torch.equal(pair_of[flat[flat >= 0].long()].long(), torch.nonzero(flat >= 0).reshape(-1))
    for e in range(7):
        mine = flat[key == e].long()
        begin = int(ends[e - 1]) if e else 0
        assert torch.equal(mine, torch.arange(begin, begin + len(mine))) and int(ends[e]) % 256 == 0


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_reference_quant_is_near(fmt):
    """Half a step of the format: 2^-4 (e4m3) or 2^-3 (e5m2) of a value, and of
    the smallest step for small ones."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(2, 144, 272, generator=gen)
    for tile in (False, True):
        q, s = R.quant(x, fmt, tile)
        step = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}[fmt]
        for i in range(2):
            v = R.values(q[i], s[i], tile)
            scale = R.values(torch.ones_like(q[i]), s[i], tile)
            assert bool(((v - x[i].double()).abs() <= torch.maximum(step[0] * x[i].double().abs() * (1 + 1e-6), step[1] * scale)).all())


def test_reference_gradients_match_differences():
    """Both operators are linear in every argument: differences are exact up
    to rounding."""
    gen = torch.Generator().manual_seed(3)
    t, k, h, experts = 9, 2, 16, 3
    ids = torch.randint(-1, experts, (t, k), generator=gen, dtype=torch.int32)
    m = R.moe_rows(t, k, experts)
    _, _, row_of, _ = R.sort(ids, experts, m)
    r64 = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    y, w, dout, x, dy, dprob = r64(m, h), r64(t, k), r64(t, h), r64(t, h), r64(m, h), r64(m)
    gy, gw, _ = R.combine_bwd64(dout, y, row_of, w)
    f = lambda y, w: float((dout * R.combine64(y, row_of, w)[0]).sum())  # noqa: E731

    def gather(x, w):
        use = row_of >= 0
        r = row_of[use].long()
        tok = torch.arange(t)[:, None].expand(t, k)[use]
        return float((dy[r] * x[tok]).sum() + (dprob[r] * w[use]).sum())

    gx = R.combine64(dy, row_of, None)[0]
    gd = torch.where(row_of >= 0, dprob[row_of.clamp(min=0).long()], torch.zeros((), dtype=torch.float64))
    r0 = int(row_of[row_of >= 0][0])
    for fun, args, which, grad, at in ((f, [y, w], 0, gy, (r0, 5)), (f, [y, w], 0, gy, (m - 1, 0)), (f, [y, w], 1, gw, (4, 1)),
                                       (gather, [x, w], 0, gx, (3, 7)), (gather, [x, w], 1, gd, (8, 0))):
        v = args[which]
        old = float(v[at])
        v[at] = old + 1
        hi = fun(*args)
        v[at] = old - 1
        lo = fun(*args)
        v[at] = old
        assert abs((hi - lo) / 2 - float(grad[at])) < 1e-9


@pytest.mark.parametrize("m", [1, 2, 16, 17, 40, 64, 65, 300, 1000, 4096, 8192])
def test_gemm_fp8_plan(m):
    """Every size has a form; parts of K have room for their sums and none is too short."""
    seen = set()
    for n in (8, 128, 1000, 4096, 8192):
        for k in (0, 16, 512, 2048, 7168, 16384):
            text = bsg.plan_string("gemm_fp8", m, n, k)
            form, _, parts = text.partition(" / ")
            assert form in ("few 16", "few 32", "few 64", "Small", "Mid", "Big")
            if form.startswith("few"):
                assert m <= int(form[4:]) <= max(16, 2 * m)
            need = bsg.workspace_bytes("gemm_fp8", m, n, k)
            assert need == (4 * m * n * int(parts) if parts else 0)
            assert not parts or (form == "Small" and k >= 128 * 4 * int(parts) - 127)
            seen.add(form)
    assert ("Big" in seen) == (m >= 1000) or m == 1000
    assert bsg.plan_string("gemm_fp8", 0, 64, 64) == "none"
    with pytest.raises(ValueError):
        bsg.plan_string("moe_sort", 1, 1, 1)
