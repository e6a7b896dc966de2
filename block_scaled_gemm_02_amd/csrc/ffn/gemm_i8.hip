// gemm_i8: C = (A B^T) * a_scale * b_scale + bias from 8-bit integers.
#include "few.hpp"

namespace bsg {
namespace ffn {
namespace {

__device__ __forceinline__ float load_float(const void *p, int64_t i, int dt)
{
    return dt == DT_F32 ? ((const float *)p)[i] : dt == DT_F16 ? (float)((const _Float16 *)p)[i] : (float)((const __bf16 *)p)[i];
}

// Scales four sums of row r from column c on, adds the bias and stores them.
template <int CT>
__device__ __forceinline__ void finish4(const I8Args &p, int64_t r, int64_t c, float4 s)
{
    const float rs = p.a_scale[r], *const cs = p.b_scale + c;
    float b[4] = {0, 0, 0, 0};
    if (p.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = load_float(p.bias, c + e, p.bias_dtype);
    }
    store4<CT>(p.c, r * p.n + c, make_float4(s.x * rs * cs[0] + b[0], s.y * rs * cs[1] + b[1], s.z * rs * cs[2] + b[2],
                                             s.w * rs * cs[3] + b[3]));
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
template <int CT, class S, bool SPLIT>
__global__ __launch_bounds__(256, S::kWaves) void k_i8(I8Args p, int mt, int nt, int splits)
{
    typedef typename S::template Of<IN_I8, true, true> T;
    constexpr int MI = S::MI, NB = S::NB;
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    const int lane = threadIdx.x & 63, w = wave_id();
    const auto [at, part] = tile_of_block<SPLIT>(blockIdx.x, mt, nt, splits);
    const Split sp = split_of(part, SPLIT ? splits : 1, pairs_of(p.k));
    const int64_t ld = p.k, m0 = (int64_t)S::TM * at.m, n0 = (int64_t)S::TN * at.n;
    typename T::LA la;
    typename T::LB lb;
    {
        const int64_t r = m0 + S::TM / 4 * w, c = n0 + S::TN / 4 * w;
        la.init_k((const uint8_t *)p.a + r * ld, (p.m - r) * ld, ld, ld, w, lane);
        lb.init_k((const uint8_t *)p.b + c * ld, (p.n - c) * ld, ld, ld, w, lane);
    }
    auto seek = [&](int pair) {
        la.seek(sp.at(pair));
        lb.seek(sp.at(pair));
    };
    f32x16 acc[MI][NB];
    T t;
    const int64_t r0 = m0 + 32 * MI * (w >> 1), c0 = n0 + 32 * NB * (w & 1);
    const int rows = (int)min((int64_t)32 * MI, p.m - r0), cols = (int)min((int64_t)32 * NB, p.n - c0);
    // scales and bias, in registers over the K loop: a row's for each block,
    // and columns l and l + 64 of the wave's in lane l
    constexpr int CL = (NB + 1) / 2;
    float rs[MI], sc[CL], bi[CL];
    if constexpr (!SPLIT) {
#pragma unroll
        for (int i = 0; i < MI; ++i) rs[i] = 32 * i + (lane & 31) < rows ? p.a_scale[r0 + 32 * i + (lane & 31)] : 0.0f;
#pragma unroll
        for (int h = 0; h < CL; ++h) {
            const int c = lane + 64 * h;
            sc[h] = c < cols ? p.b_scale[c0 + c] : 0.0f;
            bi[h] = c < cols && p.bias ? load_float(p.bias, c0 + c, p.bias_dtype) : 0.0f;
        }
    }
    t.run(acc, ring, la, lb, sp.count, seek);
    uint8_t *const reg = ring + w * T::kStage;
    if constexpr (SPLIT) {
        put_sums<NB, 0>(acc, reg, (float *)p.workspace + (sp.index * p.m + r0) * p.n + c0, p.n, rows, cols, lane);
    } else {
        constexpr int ES = es_of<CT>(), kReg = 32 * StageGeom<ES, NB>::RBP;
        static_assert(kReg + 8 * 64 * CL <= T::kStage, "the staging fits the wave's part of the ring");
        float *const cs = reinterpret_cast<float *>(reg + kReg), *const cb = cs + 64 * CL;   // scale and bias of the columns
#pragma unroll
        for (int h = 0; h < CL; ++h) {
            cs[lane + 64 * h] = sc[h];
            cb[lane + 64 * h] = bi[h];
        }
        static_for<MI>([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            __builtin_amdgcn_sched_barrier(0);
            pin(acc[i]);
            stage_block<CT, NB>(reg, lane, [&](auto jj, auto qq) {
                constexpr int j = decltype(jj)::value, q = decltype(qq)::value;
                const int c = 32 * j + 8 * q + 4 * (lane >> 5);
                const float4 s = *reinterpret_cast<const float4 *>(cs + c), b = *reinterpret_cast<const float4 *>(cb + c);
                return make_float4((float)__float_as_int(acc[i][j][4 * q]) * rs[i] * s.x + b.x,
                                   (float)__float_as_int(acc[i][j][4 * q + 1]) * rs[i] * s.y + b.y,
                                   (float)__float_as_int(acc[i][j][4 * q + 2]) * rs[i] * s.z + b.z,
                                   (float)__float_as_int(acc[i][j][4 * q + 3]) * rs[i] * s.w + b.w);
            });
            flush_block<ES, NB>(reg, (char *)p.c + ES * ((r0 + 32 * i) * p.n + c0), (uint32_t)(ES * p.n), rows - 32 * i,
                                ES * cols, lane);
        });
    }
}

// Joins the splits' sums: four columns a thread.
template <int CT>
__global__ __launch_bounds__(256) void k_i8_join(I8Args p, int splits)
{
    const int64_t i = 256ll * blockIdx.x + threadIdx.x, n4 = p.n / 4;
    if (i < p.m * n4) finish4<CT>(p, i / n4, i % n4 * 4, join4<IN_I8>((const float *)p.workspace + 4 * i, p.m * p.n, splits));
}

// ---------------------------------------------------------------------------
// Few tokens
// ---------------------------------------------------------------------------
template <int CT, int MB, int U>
__global__ __launch_bounds__(kFewThreads) void k_i8_few(I8Args p)
{
    __shared__ __attribute__((aligned(16))) float red[kFewWaves * 16 * MB * 16];
    const int lane = threadIdx.x & 63;
    const int64_t c0 = 16ll * blockIdx.x;
    const uint8_t *const wrow = (const uint8_t *)p.b + min(c0 + (lane & 15), p.n - 1) * p.k, *xrow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) xrow[b] = (const uint8_t *)p.a + min((int64_t)16 * b + (lane & 15), p.m - 1) * p.k;
    few_sums<IN_I8, MB, U>(red, wrow, xrow, (int)p.k);
    for (int i = threadIdx.x; i < 16 * (int)p.m; i += kFewThreads) {
        const int ch = i % 16, tk = i / 16;
        const int64_t c = c0 + ch;
        if (c >= p.n) continue;
        const float bias = p.bias ? load_float(p.bias, c, p.bias_dtype) : 0.0f;
        store_one<CT>(p.c, tk * p.n + c, few_join<IN_I8, MB>(red, tk, ch) * p.a_scale[tk] * p.b_scale[c] + bias);
    }
}

template <int CT, int MB, int U>
void go_few(const I8Args &a, hipStream_t s)
{
    k_i8_few<CT, MB, U><<<(unsigned)((a.n + 15) / 16), kFewThreads, 0, s>>>(a);
}

template <int CT>
void launch(const I8Args &a, hipStream_t s)
{
    if (few_is_cheaper(a.m, a.n, a.k)) {
        if (a.m <= 16) return go_few<CT, 1, 2>(a, s);
        if (a.m <= 32) return go_few<CT, 2, 2>(a, s);
        return go_few<CT, 4, 1>(a, s);
    }
    const Plan p = plan_of(a.m, a.n, a.k);
    with_shape(p, [&](auto shape, auto split) {
        k_i8<CT, decltype(shape), decltype(split)::value><<<p.grid(), 256, 0, s>>>(a, p.mt, p.nt, p.splits);
    });
    if (p.splits > 1) k_i8_join<CT><<<(unsigned)((a.m * a.n / 4 + 255) / 256), 256, 0, s>>>(a, p.splits);
}

}  // namespace

int64_t workspace_gemm_i8(int64_t m, int64_t n, int64_t k)
{
    if (few_is_cheaper(m, n, k)) return 0;
    const Plan p = plan_of(m, n, k);
    return p.splits > 1 ? 4 * m * n * p.splits : 0;
}

hipError_t launch_gemm_i8(const I8Args &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    if (a.c_dtype == DT_F32) launch<DT_F32>(a, s);
    else if (a.c_dtype == DT_F16) launch<DT_F16>(a, s);
    else launch<DT_BF16>(a, s);
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
