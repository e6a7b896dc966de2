"""Python binding of the gfx950 block-scaled GEMM library (libbsg.so).

Argument marshalling only: torch tensors become device pointers, the current
torch stream becomes the hipStream_t, and every step runs inside the HIP
kernels behind the C ABI declared in include/bsg.h.  There is no fallback:
if libbsg.so is missing or a call fails, a RuntimeError is raised.

Entry points keep the C names:
    gemm_amax, grouped_gemm, grouped_gemm_srelu, grouped_gemm_dswiglu,
    gemm_proj_rope_mxfp8, grouped_gemm_discrete, grouped_gemm_srelu_discrete,
    quant_i8, gemm_i8, gemm_glu, gemm_glu_i8, gemm_glu_bwd,
    moe_sort, moe_gather, moe_gather_bwd, moe_combine, moe_combine_bwd,
    quant_fp8, gemm_fp8, grouped_gemm_fp8, grouped_gemm_fp8_wgrad
and validate_only=True calls the host-only check bsg_validate_<name>.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsg.so")

# bsg_dtype
F32, F16, BF16, E4M3, E5M2, E2M1X2, E8M0 = range(7)
_TORCH_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
STATUS = {0: "OK", 1: "NULLPTR", 2: "SHAPE", 3: "DTYPE", 4: "ALIGN", 5: "UNSUPPORTED",
          6: "DEVICE", 7: "LAUNCH"}

# the feed-forward operators, bsg_act and bsg_op
_FFN_OPS = ["quant_i8", "gemm_i8", "gemm_glu", "gemm_glu_i8", "gemm_glu_bwd"]
_ACTS = {"silu": 0, "gelu_tanh": 1, "relu": 2}
_WS_OPS = {"gemm_i8": 0, "gemm_glu": 1, "gemm_glu_i8": 2, "gemm_glu_bwd": 3, "moe_sort": 4, "gemm_fp8": 5}
# the expert operators
_MOE_OPS = ["moe_sort", "moe_gather", "moe_gather_bwd", "moe_combine", "moe_combine_bwd", "quant_fp8", "gemm_fp8",
            "grouped_gemm_fp8", "grouped_gemm_fp8_wgrad"]


class BsgError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib():
    """Load libbsg.so (built by block_scaled_gemm_02_amd/build.py); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m block_scaled_gemm_02_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        sigs = {
            "gemm_amax": [p] * 6 + [i64] * 4 + [i32] * 6 + [p],
            "grouped_gemm": [p] * 8 + [i64] * 4 + [i32] * 3 + [p],
            "grouped_gemm_srelu": [p] * 14 + [i64] * 4 + [i32] * 4 + [f32, p],
            "gemm_proj_rope_mxfp8": [p] * 10 + [i64] * 5 + [i32, i32, p],
            "grouped_gemm_dswiglu": [p] * 16 + [i64] * 4 + [i32] * 5 + [p],
            "bsg_validate_grouped_gemm_dswiglu": [p] * 16 + [i64] * 4 + [i32] * 5,
            "grouped_gemm_discrete": [p] * 8 + [i64] * 4 + [i32] * 3 + [p],
            "grouped_gemm_srelu_discrete": [p] * 14 + [i64] * 4 + [i32] * 4 + [f32, p],
            "bsg_validate_grouped_gemm_discrete": [p] * 8 + [i64] * 4 + [i32] * 3,
            "bsg_validate_grouped_gemm_srelu_discrete": [p] * 14 + [i64] * 4 + [i32] * 4 + [f32],
            "bsg_validate_gemm_amax": [p] * 6 + [i64] * 4 + [i32] * 6,
            "bsg_validate_grouped_gemm": [p] * 8 + [i64] * 4 + [i32] * 3,
            "bsg_validate_grouped_gemm_srelu": [p] * 14 + [i64] * 4 + [i32] * 4 + [f32],
            "bsg_validate_gemm_proj_rope_mxfp8": [p] * 10 + [i64] * 5 + [i32, i32],
            "bsg_check_padded_offsets": [p, i64, i64, p],
            "quant_i8": [p] * 3 + [i64] * 2 + [i32, p],
            "gemm_i8": [p] * 7 + [i64] * 4 + [i32, i32, p],
            "gemm_glu": [p] * 7 + [i64] * 4 + [i32, i32, p],
            "gemm_glu_i8": [p] * 8 + [i64] * 4 + [i32, i32, p],
            "gemm_glu_bwd": [p] * 10 + [i64] * 4 + [i32, i32, p],
            "moe_sort": [p] * 6 + [i64] * 5 + [p],
            "moe_gather": [p] * 8 + [i64] * 5 + [i32] * 3 + [p],
            "moe_gather_bwd": [p] * 5 + [i64] * 4 + [i32, p],
            "moe_combine": [p] * 4 + [i64] * 4 + [i32, p],
            "moe_combine_bwd": [p] * 8 + [i64] * 5 + [i32] * 2 + [p],
            "quant_fp8": [p] * 5 + [i64] * 3 + [i32] * 3 + [p],
            "gemm_fp8": [p] * 6 + [i64] * 4 + [i32] * 2 + [p],
            "grouped_gemm_fp8": [p] * 7 + [i64] * 5 + [i32] * 2 + [p],
            "grouped_gemm_fp8_wgrad": [p] * 6 + [i64] * 4 + [i32] * 2 + [p],
        }
        for name in _FFN_OPS + _MOE_OPS:
            sigs["bsg_validate_" + name] = sigs[name][:-1]
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = i32
        L.bsg_workspace_bytes.restype = i64
        L.bsg_workspace_bytes.argtypes = [i32, i64, i64, i64]
        L.bsg_moe_rows.restype = i64
        L.bsg_moe_rows.argtypes = [i64] * 3
        L.bsg_plan_string.restype = ctypes.c_char_p
        L.bsg_plan_string.argtypes = [i32, i64, i64, i64]
        L.bsg_grouped_plan_string.restype = ctypes.c_char_p
        L.bsg_grouped_plan_string.argtypes = [i32] + [i64] * 5 + [i32]
        L.bsg_status_string.restype = ctypes.c_char_p
        L.bsg_status_string.argtypes = [i32]
        L.bsg_last_error.restype = ctypes.c_char_p
        L.bsg_last_error.argtypes = []
        L.bsg_version.restype = i32
        _lib = L
    return _lib


def symbols():
    """Names of the C entry points this binding expects libbsg.so to export."""
    return ["gemm_amax", "grouped_gemm", "grouped_gemm_srelu", "gemm_proj_rope_mxfp8",
            "grouped_gemm_discrete", "grouped_gemm_srelu_discrete", "grouped_gemm_dswiglu",
            "bsg_validate_gemm_amax", "bsg_validate_grouped_gemm",
            "bsg_validate_grouped_gemm_srelu", "bsg_validate_gemm_proj_rope_mxfp8",
            "bsg_validate_grouped_gemm_dswiglu",
            "bsg_validate_grouped_gemm_discrete", "bsg_validate_grouped_gemm_srelu_discrete",
            "bsg_check_padded_offsets", "bsg_status_string", "bsg_last_error", "bsg_version",
            *_FFN_OPS, *("bsg_validate_" + n for n in _FFN_OPS), "bsg_workspace_bytes",
            "bsg_plan_string", "bsg_grouped_plan_string", *_MOE_OPS, *("bsg_validate_" + n for n in _MOE_OPS), "bsg_moe_rows"]


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# ---------------------------------------------------------------------------
# Tensor checks.  The C ABI receives bare pointers and cannot see how large a
# buffer is, so the binding checks every torch tensor it is handed against
# what the kernels will read or write for the given sizes: device, dense
# row-major layout, element type and byte count.  Plain integers are device
# addresses; their extent is the caller's contract.
# ---------------------------------------------------------------------------
_OUT_TORCH = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
_BYTES = {F32: 4.0, F16: 2.0, BF16: 2.0, E4M3: 1.0, E5M2: 1.0, E2M1X2: 0.5}


def _cdiv(a, b):
    return -(-a // b)


def sf_atom_bytes(mn: int, k: int, l: int = 1) -> int:
    """Bytes of a (32, 4, ceil(MN/128), 4, ceil(K/128), L) E8M0 scale-atom buffer."""
    return 512 * _cdiv(mn, 128) * _cdiv(_cdiv(k, 32), 4) * l


def _need(t, name, nbytes, kind=None):
    """Reject a tensor that the kernel cannot use as `name`: kind is a
    bsg_dtype code (a float dtype must match exactly; FP8 / FP4 codes need
    one-byte elements), a torch dtype, or None (any element type)."""
    if t is None or isinstance(t, int):
        return
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise BsgError(6, f"{name} must be on the current CUDA device (got {t.device})")
    if not t.is_contiguous():
        raise BsgError(4, f"{name} must be contiguous")
    if isinstance(kind, torch.dtype):
        # 8-bit floats may come as plain bytes
        if t.dtype != kind and not (t.dtype == torch.uint8 and kind in (torch.float8_e4m3fn, torch.float8_e5m2)):
            raise BsgError(3, f"{name} must be {kind} (got {t.dtype})")
    elif kind in _OUT_TORCH:
        if t.dtype != _OUT_TORCH[kind]:
            raise BsgError(3, f"{name} must be {_OUT_TORCH[kind]} for dtype code {kind} (got {t.dtype})")
    elif kind is not None and t.element_size() != 1:
        raise BsgError(3, f"{name} holds one-byte codes (got {t.dtype})")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise BsgError(2, f"{name} holds {have} bytes; these sizes need {int(nbytes)}")


def _out_bytes(code, count):
    return int(_BYTES.get(code, 1.0) * count)


def _ab_row_bytes(ab, k):
    return k // 2 if ab == E2M1X2 else k


def _grouped_common_need(padded_offsets, alpha, prob, m, num_experts):
    _need(padded_offsets, "padded_offsets", 4 * num_experts, torch.int32)
    _need(alpha, "alpha", 4 * num_experts, torch.float32)
    _need(prob, "prob", 4 * m, torch.float32)


# The current device and its stream.  torch.cuda.current_stream() makes a Stream
# object, 2.8 us a call; the queries beneath it are not public, and a torch
# without GPU support lacks them: there the public functions answer.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _stream(stream):
    if stream is None:
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != 0:
        raise BsgError(rc, lib().bsg_last_error().decode())


def dtype_code(x) -> int:
    """torch dtype or tensor -> bsg_dtype code (float outputs only)."""
    if isinstance(x, int):
        return x
    if isinstance(x, torch.Tensor):
        x = x.dtype
    return _TORCH_DT[x]


def _ab_code(fmt) -> int:
    return {"e4m3": E4M3, "e5m2": E5M2, "e2m1": E2M1X2, E4M3: E4M3, E2M1X2: E2M1X2, E5M2: E5M2}[fmt]


def _d_code(d_dtype, d) -> int:
    """Output dtype code: "e4m3" / "e5m2" (or torch's float8_e4m3fn /
    float8_e5m2) for FP8 outputs, else a torch float dtype (taken from the
    tensor d when d_dtype is None)."""
    x = d_dtype if d_dtype is not None else d
    if isinstance(x, torch.Tensor):
        x = x.dtype
    if x in ("e4m3", E4M3, torch.float8_e4m3fn):
        return E4M3
    if x in ("e5m2", E5M2, torch.float8_e5m2):
        return E5M2
    if x in ("e2m1", E2M1X2):
        return E2M1X2
    return dtype_code(x)


# ---------------------------------------------------------------------------
def _major(x, allowed, name):
    """A major argument as the character code the C ABI takes."""
    if not isinstance(x, str) or len(x) != 1:
        raise ValueError(f"{name} must be one of {allowed!r}, got {x!r}")
    return ord(x)


def gemm_amax(a, b, sfa, sfb, c, amax, m, n, k, l, ab_dtype="e4m3", c_dtype=None,
              sf_vec_size=32, a_major="k", b_major="k", c_major="n", stream=None, validate_only=False):
    """C = sum_k A_hat B_hat per batch and Amax = max |C| (see include/bsg.h).
    c_dtype: a torch float dtype, "e4m3" / "e5m2" (FP8 C) or "e2m1" (packed
    FP4 C, (M, N/2, L) bytes); the last three with FP4 operands only.
    a_major "k" (memory [L][M][K]) or "m" ([L][K][M]); b_major "k" or "n"
    ([L][K][N]); c_major "n" ([L][M][N]) or "m" ([L][N][M])."""
    cd = _d_code(c_dtype, c)
    ab = _ab_code(ab_dtype)
    if m * n * l > 0:
        rb = _ab_row_bytes(ab, k)
        _need(a, "a", l * m * rb, ab); _need(b, "b", l * n * rb, ab)
        _need(sfa, "sfa", sf_atom_bytes(m, k, l), E8M0); _need(sfb, "sfb", sf_atom_bytes(n, k, l), E8M0)
        _need(c, "c", _out_bytes(cd, l * m * n), cd)
    _need(amax, "amax", 4, torch.float32)
    args = [_ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb), _ptr(c), _ptr(amax), m, n, k, l,
            ab, cd, sf_vec_size, _major(a_major, "km", "a_major"), _major(b_major, "kn", "b_major"),
            _major(c_major, "nm", "c_major")]
    if validate_only:
        return lib().bsg_validate_gemm_amax(*args)
    _check(lib().gemm_amax(*args, _stream(stream)))


def check_padded_offsets(padded_offsets, m, num_experts=None, stream=None):
    """Opt-in debug check of the routing offsets' values on the device
    (bsg_check_padded_offsets: multiples of 256 in [0, m], nondecreasing);
    waits for the stream.  Raises BsgError naming the first violation."""
    if num_experts is None:
        num_experts = padded_offsets.numel()
    _need(padded_offsets, "padded_offsets", 4 * num_experts, torch.int32)
    _check(lib().bsg_check_padded_offsets(_ptr(padded_offsets), num_experts, m, _stream(stream)))


def grouped_gemm(a, b, padded_offsets, alpha, prob, bias, c, d, m, n, k, num_experts,
                 bias_dtype=None, c_dtype=None, d_dtype=None, stream=None, validate_only=False):
    """BF16 grouped GEMM with alpha / prob / bias epilogue (see include/bsg.h)."""
    bd = dtype_code(bias_dtype if bias_dtype is not None else (bias if bias is not None else torch.bfloat16))
    cd = dtype_code(c_dtype if c_dtype is not None else (c if c is not None else torch.bfloat16))
    dd = dtype_code(d_dtype if d_dtype is not None else d)
    _grouped_common_need(padded_offsets, alpha, prob, m, num_experts)
    if m * n > 0:
        _need(a, "a", 2 * m * k, torch.bfloat16); _need(b, "b", 2 * num_experts * n * k, torch.bfloat16)
        _need(bias, "bias", _out_bytes(bd, n * num_experts), bd)
        _need(c, "c", _out_bytes(cd, m * n), cd); _need(d, "d", _out_bytes(dd, m * n), dd)
    args = [_ptr(a), _ptr(b), _ptr(padded_offsets), _ptr(alpha), _ptr(prob), _ptr(bias),
            _ptr(c), _ptr(d), m, n, k, num_experts, bd, cd, dd]
    if validate_only:
        return lib().bsg_validate_grouped_gemm(*args)
    _check(lib().grouped_gemm(*args, _stream(stream)))


def grouped_gemm_srelu(a, b, sfa, sfb, padded_offsets, alpha, prob, norm_const, c, d, d_col,
                       sfd_row, sfd_col, amax, m, n, k, num_experts, ab_dtype="e4m3",
                       c_dtype=None, d_dtype=None, sf_vec_size=32, tanh_clamp_scale=0.0,
                       stream=None, validate_only=False):
    """Grouped block-scaled GEMM + prob-gated squared ReLU (see include/bsg.h).

    d_dtype: a torch float dtype, or "e4m3" / "e5m2" / "e2m1" for MX-quantised
    output with SFD_row/col.  c_dtype: a torch float dtype, or "e4m3" /
    "e5m2" / "e2m1" for an unscaled saturating cast of C (E2M1 packed two
    per byte)."""
    cd = _d_code(c_dtype if c_dtype is not None else (c if c is not None else torch.bfloat16), None)
    dd = _d_code(d_dtype, d)
    s = float(tanh_clamp_scale) if tanh_clamp_scale is not None else 0.0
    ab = _ab_code(ab_dtype)
    _grouped_common_need(padded_offsets, alpha, prob, m, num_experts)
    _need(amax, "amax", 4 * num_experts, torch.float32)
    if m * n > 0:
        rb = _ab_row_bytes(ab, k)
        _need(a, "a", m * rb, ab); _need(sfa, "sfa", sf_atom_bytes(m, k, 1), E8M0)
        _need(b, "b", num_experts * n * rb, ab)
        _need(sfb, "sfb", sf_atom_bytes(n, k, num_experts), E8M0)
        _need(c, "c", _out_bytes(cd, m * n), cd)
        _need(d, "d", _out_bytes(dd, m * n), dd); _need(d_col, "d_col", _out_bytes(dd, m * n), dd)
        _need(norm_const, "norm_const", 4, torch.float32)
        _need(sfd_row, "sfd_row", sf_atom_bytes(m, n, 1), E8M0)
        _need(sfd_col, "sfd_col", sf_atom_bytes(n, m, 1), E8M0)
    args = [_ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb), _ptr(padded_offsets), _ptr(alpha),
            _ptr(prob), _ptr(norm_const), _ptr(c), _ptr(d), _ptr(d_col), _ptr(sfd_row),
            _ptr(sfd_col), _ptr(amax), m, n, k, num_experts, ab, cd, dd,
            sf_vec_size, s]
    if validate_only:
        return lib().bsg_validate_grouped_gemm_srelu(*args)
    _check(lib().grouped_gemm_srelu(*args, _stream(stream)))


def pointer_array(tensors):
    """(L,) int64 device tensor of the tensors' data pointers, for the
    discrete-weight calls (b_ptrs / sfb_ptrs).  The caller keeps the tensors
    alive until the stream has finished with them."""
    ptrs = [t.data_ptr() for t in tensors]
    return torch.tensor(ptrs, dtype=torch.int64).to(tensors[0].device)


def grouped_gemm_discrete(a, b_ptrs, padded_offsets, alpha, prob, bias, c, d, m, n, k, num_experts,
                          bias_dtype=None, c_dtype=None, d_dtype=None, stream=None, validate_only=False):
    """grouped_gemm with per-expert weight allocations: b_ptrs is an (L,)
    int64 device tensor of (N,K) bf16 matrices (see include/bsg.h)."""
    bd = dtype_code(bias_dtype if bias_dtype is not None else (bias if bias is not None else torch.bfloat16))
    cd = dtype_code(c_dtype if c_dtype is not None else (c if c is not None else torch.bfloat16))
    dd = dtype_code(d_dtype if d_dtype is not None else d)
    _grouped_common_need(padded_offsets, alpha, prob, m, num_experts)
    if m * n > 0:
        _need(a, "a", 2 * m * k, torch.bfloat16); _need(b_ptrs, "b_ptrs", 8 * num_experts, torch.int64)
        _need(bias, "bias", _out_bytes(bd, n * num_experts), bd)
        _need(c, "c", _out_bytes(cd, m * n), cd); _need(d, "d", _out_bytes(dd, m * n), dd)
    args = [_ptr(a), _ptr(b_ptrs), _ptr(padded_offsets), _ptr(alpha), _ptr(prob), _ptr(bias),
            _ptr(c), _ptr(d), m, n, k, num_experts, bd, cd, dd]
    if validate_only:
        return lib().bsg_validate_grouped_gemm_discrete(*args)
    _check(lib().grouped_gemm_discrete(*args, _stream(stream)))


def grouped_gemm_srelu_discrete(a, b_ptrs, sfa, sfb_ptrs, padded_offsets, alpha, prob, norm_const, c, d,
                                d_col, sfd_row, sfd_col, amax, m, n, k, num_experts, ab_dtype="e4m3",
                                c_dtype=None, d_dtype=None, sf_vec_size=32, tanh_clamp_scale=0.0,
                                stream=None, validate_only=False):
    """grouped_gemm_srelu with per-expert weight and scale allocations:
    b_ptrs / sfb_ptrs are (L,) int64 device tensors (see include/bsg.h)."""
    cd = _d_code(c_dtype if c_dtype is not None else (c if c is not None else torch.bfloat16), None)
    dd = _d_code(d_dtype, d)
    s = float(tanh_clamp_scale) if tanh_clamp_scale is not None else 0.0
    ab = _ab_code(ab_dtype)
    _grouped_common_need(padded_offsets, alpha, prob, m, num_experts)
    _need(amax, "amax", 4 * num_experts, torch.float32)
    if m * n > 0:
        rb = _ab_row_bytes(ab, k)
        _need(a, "a", m * rb, ab); _need(sfa, "sfa", sf_atom_bytes(m, k, 1), E8M0)
        _need(b_ptrs, "b_ptrs", 8 * num_experts, torch.int64)
        _need(sfb_ptrs, "sfb_ptrs", 8 * num_experts, torch.int64)
        _need(c, "c", _out_bytes(cd, m * n), cd)
        _need(d, "d", _out_bytes(dd, m * n), dd); _need(d_col, "d_col", _out_bytes(dd, m * n), dd)
        _need(norm_const, "norm_const", 4, torch.float32)
        _need(sfd_row, "sfd_row", sf_atom_bytes(m, n, 1), E8M0)
        _need(sfd_col, "sfd_col", sf_atom_bytes(n, m, 1), E8M0)
    args = [_ptr(a), _ptr(b_ptrs), _ptr(sfa), _ptr(sfb_ptrs), _ptr(padded_offsets), _ptr(alpha),
            _ptr(prob), _ptr(norm_const), _ptr(c), _ptr(d), _ptr(d_col), _ptr(sfd_row),
            _ptr(sfd_col), _ptr(amax), m, n, k, num_experts, ab, cd, dd,
            sf_vec_size, s]
    if validate_only:
        return lib().bsg_validate_grouped_gemm_srelu_discrete(*args)
    _check(lib().grouped_gemm_srelu_discrete(*args, _stream(stream)))


def grouped_gemm_dswiglu(a, b, sfa, sfb, c, padded_offsets, alpha, beta, prob, norm_const, d_row, d_col,
                         sfd_row, sfd_col, dprob, m, n, k, num_experts, ab_dtype="e4m3", c_dtype=None,
                         d_dtype="e4m3", sf_vec_size=32, amax=None, b_major="k", stream=None,
                         validate_only=False):
    """Grouped GEMM + dSwiGLU backward (see include/bsg.h): MXFP8 D for FP8
    inputs, bf16/fp32 D with amax (L, 2) for FP4 inputs.  dprob is accumulated:
    zero-fill it first.  b_major "k" (B memory [L][N][K]) or "n" ([L][K][N],
    FP8 only)."""
    cd = BF16 if c_dtype is None else (_TORCH_DT[c_dtype] if c_dtype in _TORCH_DT else c_dtype)
    dd = _d_code(d_dtype, d_row)
    ab = _ab_code(ab_dtype)
    _grouped_common_need(padded_offsets, alpha, prob, m, num_experts)
    _need(beta, "beta", 4 * num_experts, torch.float32)
    _need(amax, "amax", 8 * num_experts, torch.float32)
    if m * n > 0:
        rb = _ab_row_bytes(ab, k)
        _need(a, "a", m * rb, ab); _need(b, "b", num_experts * n * rb, ab)
        _need(sfa, "sfa", sf_atom_bytes(m, k, 1), E8M0); _need(sfb, "sfb", sf_atom_bytes(n, k, num_experts), E8M0)
        _need(c, "c", 2 * m * 2 * n, torch.bfloat16)
        _need(d_row, "d_row", _out_bytes(dd, m * 2 * n), dd); _need(d_col, "d_col", _out_bytes(dd, m * 2 * n), dd)
        _need(norm_const, "norm_const", 4, torch.float32)
        _need(sfd_row, "sfd_row", sf_atom_bytes(m, 2 * n, 1), E8M0)
        _need(sfd_col, "sfd_col", sf_atom_bytes(2 * n, m, 1), E8M0)
        _need(dprob, "dprob", 4 * m, torch.float32)
    args = [_ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb), _ptr(c), _ptr(padded_offsets), _ptr(alpha), _ptr(beta),
            _ptr(prob), _ptr(norm_const), _ptr(d_row), _ptr(d_col), _ptr(sfd_row), _ptr(sfd_col), _ptr(dprob),
            _ptr(amax), m, n, k, num_experts, ab, cd, dd, sf_vec_size, _major(b_major, "kn", "b_major")]
    if validate_only:
        return lib().bsg_validate_grouped_gemm_dswiglu(*args)
    _check(lib().grouped_gemm_dswiglu(*args, _stream(stream)))


def gemm_proj_rope_mxfp8(x, w, x_scale, w_scale, cos, sin, out_fp8_row, out_scales_row,
                         out_fp8_col, out_scales_col, tokens, q_lora, num_heads=128,
                         head_dim=192, qk_rope=64, in_dtype=BF16, w_out_in=1, stream=None,
                         validate_only=False):
    """Projection GEMM + per-head RoPE + dual MXFP8 quantisation (see include/bsg.h)."""
    if tokens * num_heads > 0:
        nout = num_heads * head_dim
        es = 1 if in_dtype == E4M3 else 2
        kind = E4M3 if in_dtype == E4M3 else torch.bfloat16
        _need(x, "x", es * tokens * q_lora, kind); _need(w, "w", es * nout * q_lora, kind)
        _need(x_scale, "x_scale", tokens * (q_lora // 32), E8M0)
        _need(w_scale, "w_scale", nout * (q_lora // 32), E8M0)
        _need(cos, "cos", 2 * tokens * qk_rope, torch.bfloat16); _need(sin, "sin", 2 * tokens * qk_rope, torch.bfloat16)
        _need(out_fp8_row, "out_fp8_row", tokens * nout, E4M3); _need(out_fp8_col, "out_fp8_col", tokens * nout, E4M3)
        _need(out_scales_row, "out_scales_row", tokens * nout // 32, E8M0)
        _need(out_scales_col, "out_scales_col", (tokens // 32) * nout, E8M0)
    args = [_ptr(x), _ptr(w), _ptr(x_scale), _ptr(w_scale), _ptr(cos), _ptr(sin),
            _ptr(out_fp8_row), _ptr(out_scales_row), _ptr(out_fp8_col), _ptr(out_scales_col),
            tokens, q_lora, num_heads, head_dim, qk_rope, in_dtype, int(w_out_in)]
    if validate_only:
        return lib().bsg_validate_gemm_proj_rope_mxfp8(*args)
    _check(lib().gemm_proj_rope_mxfp8(*args, _stream(stream)))


# ---------------------------------------------------------------------------
# Feed-forward operators
# ---------------------------------------------------------------------------
def workspace_bytes(name, m, n, k) -> int:
    """Scratch bytes that operator `name` takes at these sizes (0 for
    quant_i8; moe_sort: of tokens, top_k, num_experts).  A program keeps one
    such buffer beside its layer."""
    if name == "quant_i8":
        return 0
    if name not in _WS_OPS:
        raise ValueError(f"no operator named {name!r}")
    b = lib().bsg_workspace_bytes(_WS_OPS[name], m, n, k)
    if b < 0:
        _refuse_sizes(m, n, k)
    return b


def _refuse_sizes(*sizes):
    raise BsgError(2 if min(sizes) < 0 else 5, lib().bsg_last_error().decode())


def plan_string(name, m, n, k, num_experts=1, max_rows=0, expert_rows=True) -> str:
    """How operator `name` goes out at these sizes (see include/bsg.h): for
    tests and tuning.  The last three count for the grouped products alone."""
    if name in ("grouped_gemm_fp8", "grouped_gemm_fp8_wgrad"):
        s = lib().bsg_grouped_plan_string(int(name.endswith("wgrad")), m, n, k, num_experts, max_rows, int(bool(expert_rows)))
    elif name not in _WS_OPS or name == "moe_sort":
        raise ValueError(f"no product named {name!r}")
    else:
        s = lib().bsg_plan_string(_WS_OPS[name], m, n, k)
    if s is None:
        _refuse_sizes(m, n, k)
    return s.decode()


_TORCH_OF = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
# (looked up once: an attribute of the torch module costs 50 ns a call)
_I8, _F32 = torch.int8, torch.float32


def _code(dtype, t) -> int:
    """dtype_code of a dtype argument, or of the tensor t if it is None."""
    x = t.dtype if dtype is None and isinstance(t, torch.Tensor) else dtype
    c = _TORCH_DT.get(x)
    return dtype_code(x) if c is None else c


def _addresses(*specs):
    """The addresses of several (tensor, name, bytes, torch dtype or None),
    checked as _need does.  A call for one token takes a few microseconds, and
    this one pass of quick checks takes one; what does not pass them goes to
    _need, which says what is wrong."""
    dev, out = None, []
    for t, name, nbytes, dt in specs:
        if t is None or type(t) is int:
            out.append(t)
            continue
        d = t.get_device()
        if dev is None and d >= 0:
            dev = _current_device()
        if d != dev or (dt is not None and t.dtype is not dt) or t.nbytes < nbytes or not t.is_contiguous():
            _need(t, name, nbytes, dt)
        out.append(t.data_ptr())
    return out


def _act(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return _ACTS[act]


def _ws_bytes(workspace, name, m, n, k):
    """Bytes of a workspace; a plain address is taken to be large enough."""
    if workspace is None:
        return 0
    if isinstance(workspace, int):
        return lib().bsg_workspace_bytes(_WS_OPS[name], m, n, k)
    return workspace.nbytes


def quant_i8(x, q, scale, m, k, x_dtype=None, stream=None, validate_only=False):
    """Rows of x (m, k) -> 8-bit integers q and one fp32 scale a row (see
    include/bsg.h).  x_dtype: torch.float32 / float16 / bfloat16, from x if None."""
    xd = _code(x_dtype, x)
    args = _addresses((x, "x", _out_bytes(xd, m * k), _TORCH_OF.get(xd)), (q, "q", m * k, _I8),
                      (scale, "scale", 4 * m, _F32))
    args += (m, k, xd)
    if validate_only:
        return lib().bsg_validate_quant_i8(*args)
    _check(lib().quant_i8(*args, _stream(stream)))


def gemm_i8(a, b, a_scale, b_scale, bias, c, m, n, k, bias_dtype=None, c_dtype=None, workspace=None,
            stream=None, validate_only=False):
    """c = (a b^T) * a_scale[:, None] * b_scale + bias from 8-bit integers
    (see include/bsg.h).  bias may be None."""
    cd = _code(c_dtype, c)
    bd = F32 if bias is None else _code(bias_dtype, bias)
    args = _addresses((a, "a", m * k, _I8), (b, "b", n * k, _I8), (a_scale, "a_scale", 4 * m, _F32),
                      (b_scale, "b_scale", 4 * n, _F32), (bias, "bias", _out_bytes(bd, n), _TORCH_OF.get(bd)),
                      (c, "c", _out_bytes(cd, m * n), _TORCH_OF.get(cd)),
                      (workspace, "workspace", 0, None))
    args += (_ws_bytes(workspace, "gemm_i8", m, n, k), m, n, k, bd, cd)
    if validate_only:
        return lib().bsg_validate_gemm_i8(*args)
    _check(lib().gemm_i8(*args, _stream(stream)))


def gemm_glu(x, w_gate, w_up, h, g, u, m, n, k, act="silu", dtype=None, workspace=None, stream=None,
             validate_only=False):
    """h = act(x w_gate^T) * (x w_up^T), and the two products in g and u
    unless they are None (see include/bsg.h).  act: "silu", "gelu_tanh" or
    "relu".  dtype: torch.float16 / bfloat16 of every tensor, from x if None."""
    dt = _code(dtype, x)
    mn, nk, td = _out_bytes(dt, m * n), _out_bytes(dt, n * k), _TORCH_OF.get(dt)
    args = _addresses((x, "x", _out_bytes(dt, m * k), td), (w_gate, "w_gate", nk, td), (w_up, "w_up", nk, td),
                      (h, "h", mn, td), (g, "g", mn, td), (u, "u", mn, td),
                      (workspace, "workspace", 0, None))
    args += (_ws_bytes(workspace, "gemm_glu", m, n, k), m, n, k, dt, _act(act))
    if validate_only:
        return lib().bsg_validate_gemm_glu(*args)
    _check(lib().gemm_glu(*args, _stream(stream)))


def gemm_glu_i8(a, w_gate, w_up, a_scale, gate_scale, up_scale, h, m, n, k, act="silu", h_dtype=None,
                workspace=None, stream=None, validate_only=False):
    """gemm_glu from 8-bit integers and their scales (see include/bsg.h)."""
    dt = _code(h_dtype, h)
    args = _addresses((a, "a", m * k, _I8), (w_gate, "w_gate", n * k, _I8), (w_up, "w_up", n * k, _I8),
                      (a_scale, "a_scale", 4 * m, _F32), (gate_scale, "gate_scale", 4 * n, _F32),
                      (up_scale, "up_scale", 4 * n, _F32), (h, "h", _out_bytes(dt, m * n), _TORCH_OF.get(dt)),
                      (workspace, "workspace", 0, None))
    args += (_ws_bytes(workspace, "gemm_glu_i8", m, n, k), m, n, k, dt, _act(act))
    if validate_only:
        return lib().bsg_validate_gemm_glu_i8(*args)
    _check(lib().gemm_glu_i8(*args, _stream(stream)))


def gemm_glu_bwd(dh, x, w_gate, w_up, g, u, dx, dw_gate, dw_up, m, n, k, act="silu", dtype=None,
                 workspace=None, stream=None, validate_only=False):
    """Gradients of gemm_glu from dh and the saved g and u (see include/bsg.h).
    dx, or dw_gate and dw_up together, may be None.  In fp16 dG and dU have
    that type's range, so the loss is scaled as for any fp16 gradient."""
    dt = _code(dtype, dh)
    mn, mk, nk = _out_bytes(dt, m * n), _out_bytes(dt, m * k), _out_bytes(dt, n * k)
    td = _TORCH_OF.get(dt)
    args = _addresses((dh, "dh", mn, td), (x, "x", mk, td), (w_gate, "w_gate", nk, td), (w_up, "w_up", nk, td),
                      (g, "g", mn, td), (u, "u", mn, td), (dx, "dx", mk, td), (dw_gate, "dw_gate", nk, td),
                      (dw_up, "dw_up", nk, td), (workspace, "workspace", 0, None))
    args += (_ws_bytes(workspace, "gemm_glu_bwd", m, n, k), m, n, k, dt, _act(act))
    if validate_only:
        return lib().bsg_validate_gemm_glu_bwd(*args)
    _check(lib().gemm_glu_bwd(*args, _stream(stream)))


# ---------------------------------------------------------------------------
# Expert operators
# ---------------------------------------------------------------------------
_I32 = torch.int32
_FP8 = {"e4m3": (E4M3, torch.float8_e4m3fn), "e5m2": (E5M2, torch.float8_e5m2)}


_E4M3 = torch.float8_e4m3fn
_ES = {F32: 4, F16: 2, BF16: 2}       # bytes of an element (1 for what the call will refuse)


def _fp8(fmt):
    """The bsg_dtype code and torch dtype of an 8-bit float format's name."""
    f = _FP8.get(fmt)
    if f is None:
        raise ValueError(f"an 8-bit float format is one of {sorted(_FP8)}, got {fmt!r}")
    return f


def moe_rows(tokens, top_k, num_experts) -> int:
    """Rows that any routing of these sizes fits in, each expert's range
    padded to 256 (see include/bsg.h)."""
    m = lib().bsg_moe_rows(tokens, top_k, num_experts)
    if m < 0:
        raise BsgError(2 if tokens < 0 or top_k < 1 or not 1 <= num_experts <= 1024 else 5, lib().bsg_last_error().decode())
    return m


def moe_sort(expert, padded_offsets, expert_rows, row_of, pair_of, tokens, top_k, num_experts, m, workspace=None,
             stream=None, validate_only=False):
    """Expert ids (tokens, top_k) -> the order of the rows: padded_offsets and
    expert_rows (num_experts,), row_of (tokens, top_k) and pair_of (m,), which
    may be None (see include/bsg.h).  m: at least moe_rows(...)."""
    pairs = 4 * tokens * top_k
    args = _addresses((expert, "expert", pairs, _I32), (padded_offsets, "padded_offsets", 4 * num_experts, _I32),
                      (expert_rows, "expert_rows", 4 * num_experts, _I32), (row_of, "row_of", pairs, _I32),
                      (pair_of, "pair_of", 4 * m, _I32), (workspace, "workspace", 0, None))
    args += (_ws_bytes(workspace, "moe_sort", tokens, top_k, num_experts), tokens, top_k, num_experts, m)
    if validate_only:
        return lib().bsg_validate_moe_sort(*args)
    _check(lib().moe_sort(*args, _stream(stream)))


def moe_gather(x, row_of, padded_offsets, expert_rows, weight, y, scale, prob, tokens, hidden, top_k, num_experts, m,
               zero_pad=True, x_dtype=None, y_dtype=None, stream=None, validate_only=False):
    """y[row_of[t, j]] = x[t] and prob[row_of[t, j]] = weight[t, j] (see
    include/bsg.h).  y has x's type, or 8-bit codes (y_dtype "e4m3", taken from
    a float8_e4m3fn y) with scale (ceil(hidden / 128), m).  weight and prob may
    be None.  zero_pad: rows of an expert's range without a pair become zeros."""
    xd = _code(x_dtype, x)
    if y_dtype is not None:
        yd = _d_code(y_dtype, y)
    elif isinstance(y, torch.Tensor):
        yd = xd if y.dtype is _TORCH_OF.get(xd) else _d_code(None, y)
    else:
        yd = xd
    out = _E4M3 if yd == E4M3 else _TORCH_OF.get(yd)
    pairs = 4 * tokens * top_k
    args = _addresses((x, "x", _ES.get(xd, 1) * tokens * hidden, _TORCH_OF.get(xd)), (row_of, "row_of", pairs, _I32),
                      (padded_offsets, "padded_offsets", 4 * num_experts, _I32),
                      (expert_rows, "expert_rows", 4 * num_experts, _I32), (weight, "weight", pairs, _F32),
                      (y, "y", _ES.get(yd, 1) * m * hidden, out), (scale, "scale", 4 * m * -(-hidden // 128), _F32),
                      (prob, "prob", 4 * m, _F32))
    args += (tokens, hidden, top_k, num_experts, m, int(bool(zero_pad)), xd, yd)
    if validate_only:
        return lib().bsg_validate_moe_gather(*args)
    _check(lib().moe_gather(*args, _stream(stream)))


def moe_gather_bwd(dy, dprob, row_of, dx, dweight, tokens, hidden, top_k, m, dtype=None, stream=None,
                   validate_only=False):
    """Gradients of moe_gather: dx[t] = sum_j dy[row_of[t, j]] and dweight[t, j]
    = dprob[row_of[t, j]] (see include/bsg.h).  dprob and dweight, or dy and dx,
    may be None."""
    like = dy if dx is None else dx
    dt = F32 if dtype is None and like is None else _code(dtype, like)
    td, pairs, es = _TORCH_OF.get(dt), 4 * tokens * top_k, _ES.get(dt, 1)
    args = _addresses((dy, "dy", es * m * hidden, td), (dprob, "dprob", 4 * m, _F32),
                      (row_of, "row_of", pairs, _I32), (dx, "dx", es * tokens * hidden, td),
                      (dweight, "dweight", pairs, _F32))
    args += (tokens, hidden, top_k, m, dt)
    if validate_only:
        return lib().bsg_validate_moe_gather_bwd(*args)
    _check(lib().moe_gather_bwd(*args, _stream(stream)))


def moe_combine(y, row_of, weight, out, tokens, hidden, top_k, m, dtype=None, stream=None, validate_only=False):
    """out[t] = sum_j weight[t, j] y[row_of[t, j]] (see include/bsg.h); weight
    None: ones."""
    dt = _code(dtype, out)
    td, pairs, es = _TORCH_OF.get(dt), 4 * tokens * top_k, _ES.get(dt, 1)
    args = _addresses((y, "y", es * m * hidden, td), (row_of, "row_of", pairs, _I32),
                      (weight, "weight", pairs, _F32), (out, "out", es * tokens * hidden, td))
    args += (tokens, hidden, top_k, m, dt)
    if validate_only:
        return lib().bsg_validate_moe_combine(*args)
    _check(lib().moe_combine(*args, _stream(stream)))


def moe_combine_bwd(dout, y, row_of, padded_offsets, expert_rows, weight, dy, dweight, tokens, hidden, top_k,
                    num_experts, m, zero_pad=True, dtype=None, stream=None, validate_only=False):
    """Gradients of moe_combine: dy[row_of[t, j]] = weight[t, j] dout[t] and
    dweight[t, j] = <dout[t], y[row_of[t, j]]> (see include/bsg.h).  dy, or
    dweight and y, may be None."""
    dt = _code(dtype, dout)
    td, pairs, es = _TORCH_OF.get(dt), 4 * tokens * top_k, _ES.get(dt, 1)
    rows = es * m * hidden
    args = _addresses((dout, "dout", es * tokens * hidden, td), (y, "y", rows, td),
                      (row_of, "row_of", pairs, _I32), (padded_offsets, "padded_offsets", 4 * num_experts, _I32),
                      (expert_rows, "expert_rows", 4 * num_experts, _I32), (weight, "weight", pairs, _F32),
                      (dy, "dy", rows, td), (dweight, "dweight", pairs, _F32))
    args += (tokens, hidden, top_k, num_experts, m, int(bool(zero_pad)), dt)
    if validate_only:
        return lib().bsg_validate_moe_combine_bwd(*args)
    _check(lib().moe_combine_bwd(*args, _stream(stream)))


def quant_fp8(x, q, scale, q_t, scale_t, m, k, l=1, tile=False, q_dtype="e4m3", x_dtype=None, stream=None,
              validate_only=False):
    """x (l, m, k) -> 8-bit floats with a scale for each 128 values along k (q,
    scale) and along m (q_t, transposed, and scale_t), or with tile for each 128
    x 128 (see include/bsg.h).  Either pair may be None."""
    xd, mb, kb, n = _code(x_dtype, x), -(-m // 128), -(-k // 128), l * m * k
    qd, qt = _fp8(q_dtype)
    args = _addresses((x, "x", _ES.get(xd, 1) * n, _TORCH_OF.get(xd)), (q, "q", n, qt),
                      (scale, "scale", 4 * l * kb * (mb if tile else m), _F32),
                      (q_t, "q_t", n, qt),
                      (scale_t, "scale_t", 4 * l * mb * (kb if tile else k), _F32))
    args += (l, m, k, int(bool(tile)), xd, qd)
    if validate_only:
        return lib().bsg_validate_quant_fp8(*args)
    _check(lib().quant_fp8(*args, _stream(stream)))


def gemm_fp8(a, b, a_scale, b_scale, c, m, n, k, a_dtype="e4m3", c_dtype=None, workspace=None, stream=None,
             validate_only=False):
    """c = a b^T from 8-bit floats with a scale for each 128 of k (a: each row,
    b: each 128 rows; see include/bsg.h)."""
    cd, kb = _code(c_dtype, c), -(-k // 128)
    ad, at = _fp8(a_dtype)
    args = _addresses((a, "a", m * k, at), (b, "b", n * k, _E4M3), (a_scale, "a_scale", 4 * kb * m, _F32),
                      (b_scale, "b_scale", 4 * kb * -(-n // 128), _F32),
                      (c, "c", _ES.get(cd, 1) * m * n, _TORCH_OF.get(cd)), (workspace, "workspace", 0, None))
    args += (_ws_bytes(workspace, "gemm_fp8", m, n, k), m, n, k, ad, cd)
    if validate_only:
        return lib().bsg_validate_gemm_fp8(*args)
    _check(lib().gemm_fp8(*args, _stream(stream)))


def grouped_gemm_fp8(a, b, a_scale, b_scale, padded_offsets, expert_rows, c, m, n, k, num_experts, max_rows=0,
                     a_dtype="e4m3", c_dtype=None, stream=None, validate_only=False):
    """gemm_fp8 of rows sorted by expert with a weight for each expert (see
    include/bsg.h).  expert_rows may be None; max_rows: no expert has more rows
    (0: not known), for the choice of the kernel."""
    cd, kb = _code(c_dtype, c), -(-k // 128)
    ad, at = _fp8(a_dtype)
    args = _addresses((a, "a", m * k, at), (b, "b", num_experts * n * k, _E4M3), (a_scale, "a_scale", 4 * kb * m, _F32),
                      (b_scale, "b_scale", 4 * num_experts * kb * -(-n // 128), _F32),
                      (padded_offsets, "padded_offsets", 4 * num_experts, _I32),
                      (expert_rows, "expert_rows", 4 * num_experts, _I32),
                      (c, "c", _ES.get(cd, 1) * m * n, _TORCH_OF.get(cd)))
    args += (m, n, k, num_experts, max_rows, ad, cd)
    if validate_only:
        return lib().bsg_validate_grouped_gemm_fp8(*args)
    _check(lib().grouped_gemm_fp8(*args, _stream(stream)))


def grouped_gemm_fp8_wgrad(a, b, a_scale, b_scale, padded_offsets, c, m, n, k, num_experts, a_dtype="e4m3",
                           c_dtype=None, stream=None, validate_only=False):
    """Gradient of the experts' weights, c (num_experts, n, k), from the
    transposed codes of the output's gradient, a (n, m), and of the input, b
    (k, m) (see include/bsg.h)."""
    cd, mb = _code(c_dtype, c), -(-m // 128)
    ad, at = _fp8(a_dtype)
    args = _addresses((a, "a", n * m, at), (b, "b", k * m, _E4M3), (a_scale, "a_scale", 4 * mb * n, _F32),
                      (b_scale, "b_scale", 4 * mb * -(-k // 128), _F32),
                      (padded_offsets, "padded_offsets", 4 * num_experts, _I32),
                      (c, "c", _ES.get(cd, 1) * num_experts * n * k, _TORCH_OF.get(cd)))
    args += (m, n, k, num_experts, ad, cd)
    if validate_only:
        return lib().bsg_validate_grouped_gemm_fp8_wgrad(*args)
    _check(lib().grouped_gemm_fp8_wgrad(*args, _stream(stream)))
