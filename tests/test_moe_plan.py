"""CPU tests of which kernel the 8-bit float products take: the forms that the
GPU tests of the grouped ones mean to run, by the rule that the launch asks."""
import pytest

import block_scaled_gemm_02_amd as bsg
import test_gpu_fp8 as T


def grouped(m, n, k, experts, max_rows=0, expert_rows=True):
    return bsg.plan_string("grouped_gemm_fp8", m, n, k, num_experts=experts, max_rows=max_rows, expert_rows=expert_rows)


def wgrad(m, n, k, experts):
    return bsg.plan_string("grouped_gemm_fp8_wgrad", m, n, k, num_experts=experts)


def test_forms_of_the_grouped_cases():
    """Those of test_gpu_fp8.py."""
    for counts, m, n, k in T.GROUPS:
        assert grouped(m, n, k, len(counts)) == grouped(m, n, k, len(counts), max(counts), False) == "Mid"
        assert grouped(m, n, k, len(counts), max(counts)) == ("few 16" if max(counts) <= 3 else "Mid")
        assert grouped(m, n, k, len(counts), 1) == "few 16"
    assert grouped(17408, 2048, 2064, 9, 5000) == grouped(17408, 2048, 2064, 9, 5000, False) == "Big"
    assert grouped(8192, 4096, 9232, 1) == "Big"
    assert wgrad(6400, 2056, 2064, 6) == "Big" and wgrad(1024, 264, 520, 2) == wgrad(2304, 520, 1032, 4) == "Mid"


def test_decode_batches_take_the_kernel_of_few_rows():
    for tokens in range(1, 65):
        m = bsg.moe_rows(tokens, 2, 8)
        assert grouped(m, 1024, 1024, 8, tokens) == ("few 16" if tokens <= 16 else "few 32")
    assert grouped(m, 1024, 1024, 8, 65) == grouped(m, 1024, 1024, 8, 0) == "Mid"
    assert grouped(m, 1024, 1024, 8, 64, False) == "Mid"       # without expert_rows every row counts


@pytest.mark.parametrize("k", [16, 112, 128])
def test_one_block_takes_the_smaller_tiles(k):
    """A largest tile's way out costs more than one block of K gains, whatever the size."""
    for m in [*range(1, 1500, 83), *(2 ** i + d for i in range(11, 22) for d in (-1, 0, 300)), 1 << 22]:
        for n in (8, 256, 520, 1032, 4096, 8192, 1 << 14):
            if -(-m // 64) * -(-n // 64) < 1 << 23:
                assert bsg.plan_string("gemm_fp8", m, n, k) != "Big", (m, n, k)


def test_grouped_plan_refusals():
    for bad in (dict(m=-256), dict(m=100), dict(n=-1), dict(k=1 << 21), dict(num_experts=0), dict(num_experts=1025),
                dict(max_rows=-1), dict(m=1 << 23)):
        for name in ("grouped_gemm_fp8", "grouped_gemm_fp8_wgrad"):
            with pytest.raises(bsg.BsgError):
                bsg.plan_string(name, **{**dict(m=512, n=64, k=64, num_experts=2), **bad})
    assert grouped(0, 64, 64, 2) == grouped(512, 0, 64, 2) == wgrad(512, 0, 64, 2) == wgrad(512, 64, 0, 2) == "none"
    assert wgrad(0, 64, 64, 2) == "Mid" and grouped(512, 64, 0, 2, 1 << 40) == "Mid"
