"""What the 8-bit matrix instruction drops, through gemm_fp8, at its worst: of
each 8 consecutive products it aligns all to 2^-13 of the largest's power of two
and drops the bits below, towards zero (tests/test_gpu_mfma_precision.py).

A group here is 256 = 2^8 and seven products below 2^(8-13), which vanish: 8.0e-4
of the sum in E4M3, more than half a step of fp16 (2^-11 = 4.9e-4) and under the
stated 7 * 2^-13 = 8.5e-4 of the sum of magnitudes.  With 256 and -256 and six
small products nothing is left of the sum."""
import pytest
import torch

import block_scaled_gemm_02_amd as bsg
import moe_ref as R

pytestmark = pytest.mark.gpu
SMALL = {"e4m3": 1.875 * 2.0 ** -6, "e5m2": 1.75 * 2.0 ** -6}       # the largest codes below 2^-5
DEV = "cuda"


@pytest.mark.parametrize("fmt,dt", [("e4m3", torch.float16), ("e5m2", torch.float16), ("e4m3", torch.bfloat16)])
@pytest.mark.parametrize("m,n,k", [(2, 8, 128), (40, 264, 1024), (130, 2048, 7168), (300, 520, 640), (5000, 4096, 400),
                                   (4096, 4096, 1024)])
def test_loss_at_its_worst(m, n, k, fmt, dt):
    print("dropped bits", m, n, k, bsg.plan_string("gemm_fp8", m, n, k), fmt, dt, flush=True)
    a = torch.full((m, k), SMALL[fmt])
    a[:, ::8] = 256.0
    a[1::2, 1::8] = -256.0
    q, b = a.to(R.FP8[fmt]), torch.ones(n, k).to(torch.float8_e4m3fn)
    assert torch.equal(q.float(), a)
    kb, nb = -(-k // 128), -(-n // 128)
    sa, sb = torch.full((kb, m), 2.0 ** -8), torch.ones(nb, kb)
    c = torch.empty(m, n, dtype=dt, device=DEV)
    ws = torch.empty(bsg.workspace_bytes("gemm_fp8", m, n, k), dtype=torch.uint8, device=DEV)
    bsg.gemm_fp8(q.cuda(), b.cuda(), sa.cuda(), sb.cuda(), c, m, n, k, a_dtype=fmt, workspace=ws)
    groups, c = k // 8, c.cpu().double()
    assert bool((c[::2] == groups).all()) and bool((c[1::2] == 0).all())
    # the loss against the stated bound and fp16's half step
    ref, err = R.gemm64(q[:2], b[:1], sa[:, :2], sb[:1])
    lost = ref[:, 0] - torch.tensor([groups, 0.0])
    assert bool((lost > 0).all()) and bool((lost < err[:, 0]).all())
    assert float(lost[0] / ref[0, 0]) > 2.0 ** -11 and float(lost[1]) == float(ref[1, 0])
