// quant_i8: rows of floats -> 8-bit integers and one scale a row.
//
//   t = max(max_k |x|, 2^-100), scale = t / 127, q = rint(x * (127 / t))
//
// The bound 2^-100 keeps 127 / t finite; a row below it (an empty row) gets
// codes that are 0 or next to it and a scale that says so.
#include "act.hpp"

namespace bsg {
namespace ffn {
namespace {

template <class T>
__global__ __launch_bounds__(256) void k_quant_i8(const T *__restrict__ x, int8_t *__restrict__ q,
                                                  float *__restrict__ scale, int64_t k)
{
    const int64_t row = blockIdx.x;
    const T *xr = x + row * k;
    float top = 0.0f;
    bool nan = false;
    for (int64_t i = threadIdx.x; i < k; i += 256) {
        const float v = (float)xr[i];
        top = fmaxf(top, fabsf(v));
        nan |= v != v;
    }
    __shared__ float part[4];
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    const bool bad = __syncthreads_or(nan);
    top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    top = fmaxf(top, 0x1p-100f);
    if (bad) top = __builtin_nanf("");
    const float inv = __fdiv_rn(127.0f, top);
    for (int64_t i = threadIdx.x; i < k; i += 256) {
        const float v = rintf((float)xr[i] * inv);
        q[row * k + i] = v == v ? (int8_t)fminf(fmaxf(v, -127.0f), 127.0f) : (int8_t)0;
    }
    if (threadIdx.x == 0) scale[row] = __fdiv_rn(top, 127.0f);
}

}  // namespace

hipError_t launch_quant_i8(const QuantArgs &a, hipStream_t s)
{
    if (a.m == 0) return hipSuccess;
    const dim3 grid((unsigned)a.m), block(256);
    if (a.x_dtype == DT_F32) k_quant_i8<<<grid, block, 0, s>>>((const float *)a.x, a.q, a.scale, a.k);
    else if (a.x_dtype == DT_F16) k_quant_i8<<<grid, block, 0, s>>>((const _Float16 *)a.x, a.q, a.scale, a.k);
    else k_quant_i8<<<grid, block, 0, s>>>((const __bf16 *)a.x, a.q, a.scale, a.k);
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
