// What the operators on rows of tokens share: pieces of a row as loaded, the
// 8-bit codes of a group of 128, and how threads lie over rows.
#pragma once
#include "../ffn/act.hpp"
#include "moe.hpp"

namespace bsg {
namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int es_dt(int dt) { return dt == DT_F32 ? 4 : 2; }

// N consecutive elements as loaded (16-bit: in pairs).
template <int DT, int N>
struct Piece {
    static constexpr int W = N * es_dt(DT) / 4;
    uint32_t v[W];
    __device__ __forceinline__ void load(const void *p)
    {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const u32x4 x = ((const u32x4 *)p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = x[j];
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const
    {
        if constexpr (DT == DT_F32) return __uint_as_float(v[i]);
        else return i % 2 ? ffn::hi16<DT>(v[i / 2]) : ffn::lo16<DT>(v[i / 2]);
    }
    // the largest |x| as bits: they order like the values, with NaN on top
    __device__ __forceinline__ uint32_t top(uint32_t t) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) t = max(t, __float_as_uint(at(i)) & 0x7FFFFFFFu);
        return t;
    }
};

// 16 bytes of output from the fp32 values of an element range.
template <int DT>
__device__ __forceinline__ u32x4 pack16(const float *f)
{
    if constexpr (DT == DT_F32) return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    else return u32x4{ffn::pack2<DT>(f[0], f[1]), ffn::pack2<DT>(f[2], f[3]), ffn::pack2<DT>(f[4], f[5]), ffn::pack2<DT>(f[6], f[7])};
}

// A store of a row's piece past the L2: rows are written once, and by a
// workgroup that does not read them again.  8192 tokens of 4096 bf16 into 8 rows
// each take 113 us so and 127 us through the L2, 4001 of 7168 quantised 57 and 77.
template <class T>
__device__ __forceinline__ void store_past(T *p, T v)
{
    __builtin_nontemporal_store(v, p);
}

// The scale of a group of values and what multiplies them before the cast,
// from the bits of its largest |x|:
//   t = max(top, 2^-100),   scale = t / MAX,   inv = MAX / t
// each one fp32 operation.  keep: 0 where the group holds infinity or NaN, whose
// codes are then 0 and whose scale is not finite.
struct Scale {
    float scale, inv;
    uint32_t keep;
};
template <bool E5>
__device__ __forceinline__ Scale scale_of(uint32_t top)
{
    constexpr float M = E5 ? 57344.0f : 448.0f;
    top = max(top, __float_as_uint(0x1p-100f));
    const float t = __uint_as_float(top);
    return {__fdiv_rn(t, M), __fdiv_rn(M, t), top < 0x7F800000u ? 0xFFFFFFFFu : 0u};
}

// Four codes of x * inv, to nearest even.  |x inv| exceeds the largest code by
// a rounding at most, which the cast takes back, so it needs no bound.  The
// product is rounded by itself, as the definition has it.
template <bool E5>
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3, float inv, uint32_t keep)
{
#pragma clang fp contract(off)
    return cvt4_fp8<E5>(x0 * inv, x1 * inv, x2 * inv, x3 * inv) & keep;
}

// Threads over rows: 2^lg threads of 256 take a row, the others further rows;
// a row of more pieces than 256 goes over blockIdx.y.
struct Lay {
    int lg;
    unsigned rows, cols;        // grid
    int rows_wg() const { return 256 >> lg; }
};
inline Lay lay_of(int64_t rows, int64_t pieces, int least)
{
    int lg = least;
    while (lg < 8 && (1 << lg) < pieces) ++lg;
    const int64_t per = 256 >> lg;
    return {lg, (unsigned)((rows + per - 1) / per), (unsigned)((pieces + (1 << lg) - 1) >> lg)};
}

// f(std::integral_constant<int, DT>) for a run-time float type
template <class F>
void with_float(int dt, F &&f)
{
    if (dt == DT_F32) f(std::integral_constant<int, DT_F32>{});
    else if (dt == DT_F16) f(std::integral_constant<int, DT_F16>{});
    else f(std::integral_constant<int, DT_BF16>{});
}

}  // namespace moe
}  // namespace bsg
