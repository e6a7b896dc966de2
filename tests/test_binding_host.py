"""CPU tests of the binding on a torch without GPU support: the package
imports, every host-only check works, and the device and stream are asked for
through torch's public functions."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_RAW_QUERIES = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import block_scaled_gemm_02_amd as bsg

P = 0x10000
assert bsg.quant_i8(P, P, P, 5, 64, x_dtype=torch.bfloat16, validate_only=True) == 0
assert bsg.gemm_glu(P, P, P, P, None, None, 5, 64, 64, dtype=torch.float16, workspace=P, validate_only=True) == 0
assert bsg.gemm_amax(a=P, b=P, sfa=P, sfb=P, c=P, amax=P, m=256, n=256, k=256, l=1, ab_dtype="e4m3",
                     c_dtype=bsg.F32, sf_vec_size=32, validate_only=True) == 0


class Stream:
    cuda_stream = 1234


class Tensor:
    dtype, nbytes = torch.int8, 64
    def get_device(self): return 3
    def is_contiguous(self): return True
    def data_ptr(self): return P


torch.cuda.current_stream = lambda device=None: Stream
torch.cuda.current_device = lambda: 3
assert bsg._stream(None) == 1234 and bsg._stream(7) == 7 and bsg._stream(Stream) == 1234
assert bsg._addresses((Tensor(), "q", 64, torch.int8), (None, "bias", 4, torch.float32)) == [P, None]
"""


def test_torch_without_raw_device_queries():
    r = subprocess.run([sys.executable, "-c", WITHOUT_RAW_QUERIES], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
