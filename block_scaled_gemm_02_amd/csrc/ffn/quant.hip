// quant_i8: rows of floats -> 8-bit integers and one scale a row.
//
//   t = max(max_k |x|, 2^-100), scale = t / 127, q = rint(x * (127 / t))
//
// One pass over the row, which stays in registers between the maximum and
// the codes (up to 4 groups of 16 elements a thread of 256; the rest of a
// longer row is read a second time).  Bound by memory from about 2048 elements
// a row on: 16384 x 7168 fp16 (352 MB) takes 62 us, 5.6 TB/s (a large copy
// reaches 4.9), fp32 108 us, 5.5 TB/s; 16384 x 2048 bf16 20.9 us, 4.8 TB/s, fp32
// 30.3 us, 5.5 TB/s.  Shorter rows are bound by their number, a workgroup
// each, most of whose threads have nothing to do: 16384 rows of 256 to 1024
// elements take 12.6-14.1 us in any type, for 5.1 us of memory at 512 of bf16.
#include "act.hpp"

namespace bsg {
namespace ffn {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 consecutive elements as loaded
template <class T>
struct Group {
    u32x4 v[sizeof(T)];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) v[i] = reinterpret_cast<const u32x4 *>(p)[i];
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(v[i / 4][i % 4]);
        else {
            const uint32_t w = v[i / 8][i / 2 % 4];
            constexpr int DT = std::is_same_v<T, _Float16> ? DT_F16 : DT_BF16;
            return i % 2 ? hi16<DT>(w) : lo16<DT>(w);
        }
    }
    // the largest |x| as bits: they order like the values, with NaN on top
    __device__ __forceinline__ uint32_t top(uint32_t t) const
    {
#pragma unroll
        for (int i = 0; i < 16; ++i) t = max(t, __float_as_uint(at(i)) & 0x7FFFFFFFu);
        return t;
    }
    // 16 codes.  Adding 1.5 * 2^23 rounds to an integer, to nearest even, and
    // leaves it in the low byte; |x * inv| needs no bound, since x is at most
    // t: the product exceeds 127 by a rounding at most.  The product is
    // rounded by itself, as the definition has it (no fused multiply-add).
    __device__ __forceinline__ u32x4 codes(float inv, uint32_t keep) const
    {
#pragma clang fp contract(off)
        u32x4 q;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = at(4 * w + e) * inv;
                b[e] = __float_as_uint(p + 12582912.0f);
            }
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0C);
            q[w] = (lo | hi) & keep;
        }
        return q;
    }
};

template <class T, int NV>
__global__ __launch_bounds__(256) void k_quant_i8(const T *__restrict__ x, int8_t *__restrict__ q,
                                                  float *__restrict__ scale, int64_t k)
{
    const int64_t row = blockIdx.x;
    const T *const xr = x + row * k;
    int8_t *const qr = q + row * k;
    const int groups = (int)(k / 16), t = threadIdx.x;
    Group<T> g[NV];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (t + 256 * i < groups) g[i].load(xr + 16 * (int64_t)(t + 256 * i));
        else g[i] = Group<T>{};
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) top = g[i].top(top);
    for (int i = t + 256 * NV; i < groups; i += 256) {
        Group<T> r;
        r.load(xr + 16 * (int64_t)i);
        top = r.top(top);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    __shared__ uint32_t part[4];
    if ((t & 63) == 0) part[t >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    top = max(top, __float_as_uint(0x1p-100f));
    const float tf = __uint_as_float(top), inv = __fdiv_rn(127.0f, tf);
    const uint32_t keep = top < 0x7F800000u ? 0xFFFFFFFFu : 0u;     // a row with infinity or NaN has codes 0
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t + 256 * i < groups) *reinterpret_cast<u32x4 *>(qr + 16 * (int64_t)(t + 256 * i)) = g[i].codes(inv, keep);
    for (int i = t + 256 * NV; i < groups; i += 256) {
        Group<T> r;
        r.load(xr + 16 * (int64_t)i);
        *reinterpret_cast<u32x4 *>(qr + 16 * (int64_t)i) = r.codes(inv, keep);
    }
    if (t == 0) scale[row] = __fdiv_rn(tf, 127.0f);
}

template <class T>
void go(const QuantArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)a.m);
    const T *x = (const T *)a.x;
    // the fewest registers that hold the row (more rows at work on a CU)
    if (a.k <= 4096) k_quant_i8<T, 1><<<grid, 256, 0, s>>>(x, a.q, a.scale, a.k);
    else if (a.k <= 8192) k_quant_i8<T, 2><<<grid, 256, 0, s>>>(x, a.q, a.scale, a.k);
    else k_quant_i8<T, 4><<<grid, 256, 0, s>>>(x, a.q, a.scale, a.k);
}

}  // namespace

hipError_t launch_quant_i8(const QuantArgs &a, hipStream_t s)
{
    if (a.m == 0) return hipSuccess;
    if (a.x_dtype == DT_F32) go<float>(a, s);
    else if (a.x_dtype == DT_F16) go<_Float16>(a, s);
    else go<__bf16>(a, s);
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
