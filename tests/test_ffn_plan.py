"""CPU tests: the sizes of ffn_forms.py reach every kernel form that the
operators' calls can take, so that a change of the choice between forms cannot
leave one without a GPU test."""
import math
import random
import re

import pytest

import block_scaled_gemm_02_amd as bsg
import ffn_forms as F

PARTS = re.compile(r"/ \d+")
# the sizes of the table of measurements, and the forms that they have had
LARGE = [("gemm_i8", (8192, 8192, 8192)), ("gemm_glu_i8", (4001, 8192, 4096)), ("gemm_glu", (8192, 8192, 4096))]


def form(op, size):
    return PARTS.sub("/ P", bsg.plan_string(op, *size))


def products(text):
    """The forms of a backward call, one a launch."""
    return [text] if "+" in text else text.split(", ")


def draws(op, count):
    rng = random.Random(op)
    for _ in range(count):
        m, n, k = (math.exp(rng.uniform(math.log(lo), math.log(16384))) for lo in (1, 8, 16))
        yield int(m), max(8, int(n) // 8 * 8), max(16, int(k) // 16 * 16)


@pytest.mark.parametrize("op", F.PRODUCTS)
def test_product_sizes_reach_every_form(op):
    for name, size in F.PRODUCTS[op].items():
        assert form(op, size) == name, size
    assert {form(op, s) for s in draws(op, 6000)} == set(F.PRODUCTS[op])


def test_backward_sizes_reach_every_form():
    for name, size in F.BACKWARD.items():
        assert form("gemm_glu_bwd", size) == name, size
    reached = {p for name in F.BACKWARD for p in products(name)}
    assert {p for s in draws("gemm_glu_bwd", 20000) for p in products(form("gemm_glu_bwd", s))} == reached


@pytest.mark.parametrize("op,size", LARGE)
def test_large_products_take_the_largest_tile(op, size):
    assert form(op, size) == "Big"
    assert form("gemm_glu_bwd", (8192, 8192, 4096)) == "dX + dW: Big"


def test_plan_string():
    for op in F.PRODUCTS:
        assert bsg.plan_string(op, 0, 64, 64) == "none" and bsg.plan_string(op, 3, 0, 64) == "none"
    assert bsg.plan_string("gemm_glu_bwd", 0, 64, 64).startswith("dW: ")
    assert bsg.plan_string("gemm_glu_bwd", 5, 0, 64).startswith("dX: ")
    assert bsg.plan_string("gemm_glu_bwd", 5, 64, 0) == "none"
    assert re.fullmatch(r"Mid / [2-8]", bsg.plan_string("gemm_i8", 69, 136, 4112))
    with pytest.raises(ValueError):
        bsg.plan_string("quant_i8", 1, 1, 1)
    with pytest.raises(bsg.BsgError):
        bsg.plan_string("gemm_i8", -1, 8, 8)
    assert bsg.lib().bsg_plan_string(9, 1, 1, 1) is None


def test_sizes_with_k_in_parts():
    """What the GPU test of repeats, streams and graphs relies on."""
    (a, b, c) = F.PARTS
    assert form("gemm_glu", a) == form("gemm_glu_i8", a) == "Mid / P"
    assert form("gemm_i8", (b[0], b[2], b[1])) == "Mid / P" and form("gemm_glu_bwd", b).startswith("dX: Mid / P")
    assert form("gemm_glu_bwd", c).endswith("dW: Mid / P")


@pytest.mark.parametrize("size", [((1 << 22) + 1, 8, 16), (8, (1 << 20) + 8, 16), (8, 8, (1 << 20) + 16), (1 << 40, 1 << 30, 8),
                                  (1 << 31, 1 << 30, 8), ((1 << 63) - 1, 8, 16)])
def test_sizes_that_calls_refuse_have_no_workspace(size):
    """Past the limits on sizes the bytes would wrap around: to 0 at the
    fourth of these."""
    for op in (*F.PRODUCTS, "gemm_glu_bwd"):
        with pytest.raises(bsg.BsgError) as err:
            bsg.workspace_bytes(op, *size)
        assert err.value.status == 5
        with pytest.raises(bsg.BsgError) as err:
            bsg.plan_string(op, *size)
        assert err.value.status == 5
