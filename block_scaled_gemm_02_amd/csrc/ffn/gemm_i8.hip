// gemm_i8: C = (A B^T) * a_scale * b_scale + bias from 8-bit integers.
#include "few.hpp"

namespace bsg {
namespace ffn {
namespace {

__device__ __forceinline__ float load_float(const void *p, int64_t i, int dt)
{
    return dt == DT_F32 ? ((const float *)p)[i] : dt == DT_F16 ? (float)((const _Float16 *)p)[i] : (float)((const __bf16 *)p)[i];
}

template <int CT, int MI, int NB, int NS, bool PF>
__global__ __launch_bounds__(256, MI *NB == 16 ? 1 : 2) void k_i8(I8Args p, int mt, int nt)
{
    typedef Tile<IN_I8, true, true, MI, NB, NS, PF> T;
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    const int lane = threadIdx.x & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
    const TileAt at = tile_at(blockIdx.x, mt, nt);
    const int64_t ld = p.k, m0 = (int64_t)T::TM * at.m, n0 = (int64_t)T::TN * at.n;
    typename T::LA la;
    typename T::LB lb;
    {
        const int64_t r = m0 + T::TM / 4 * w, c = n0 + T::TN / 4 * w;
        la.init_k((const uint8_t *)p.a + r * ld, (p.m - r) * ld, ld, ld, w, lane);
        lb.init_k((const uint8_t *)p.b + c * ld, (p.n - c) * ld, ld, ld, w, lane);
    }
    const int64_t r0 = m0 + 32 * MI * wm, c0 = n0 + 32 * NB * wn;
    const int rows = (int)min((int64_t)32 * MI, p.m - r0), cols = (int)min((int64_t)32 * NB, p.n - c0);
    // scales and bias, in registers over the K loop: a row's for each block,
    // and columns l and l + 64 of the wave's in lane l
    constexpr int CL = (NB + 1) / 2;
    float rs[MI], sc[CL], bi[CL];
#pragma unroll
    for (int i = 0; i < MI; ++i) rs[i] = 32 * i + (lane & 31) < rows ? p.a_scale[r0 + 32 * i + (lane & 31)] : 0.0f;
#pragma unroll
    for (int h = 0; h < CL; ++h) {
        const int c = lane + 64 * h;
        sc[h] = c < cols ? p.b_scale[c0 + c] : 0.0f;
        bi[h] = c < cols && p.bias ? load_float(p.bias, c0 + c, p.bias_dtype) : 0.0f;
    }
    f32x16 acc[MI][NB];
    T t;
    t.run(acc, ring, la, lb, pairs_of(ld), [&](int pair) {
        la.seek(pair);
        lb.seek(pair);
    });

    uint8_t *const reg = ring + w * T::kStage;
    constexpr int ES = es_of<CT>(), kReg = 32 * StageGeom<ES, NB>::RBP;
    float *const cs = reinterpret_cast<float *>(reg + kReg), *const cb = cs + 64 * CL;   // scale and bias of the columns
#pragma unroll
    for (int h = 0; h < CL; ++h) {
        cs[lane + 64 * h] = sc[h];
        cb[lane + 64 * h] = bi[h];
    }
    const uint32_t row_bytes = (uint32_t)(ES * p.n);
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
        flush_block<ES, NB>(reg, (char *)p.c + ES * ((r0 + 32 * i) * p.n + c0), row_bytes, rows - 32 * i, ES * cols, lane);
    });
    static_assert(kReg + 8 * 64 * CL <= T::kStage, "the staging fits the wave's part of the ring");
}

template <int CT, int RB, int MB, int U>
__global__ __launch_bounds__(kFewThreads) void k_i8_few(I8Args p)
{
    __shared__ __attribute__((aligned(16))) float red[kFewWaves * 16 * MB * 16 * RB];
    const int lane = threadIdx.x & 63;
    const int64_t c0 = 16ll * RB * blockIdx.x;
    const uint8_t *wrow[RB], *xrow[MB];
#pragma unroll
    for (int b = 0; b < RB; ++b) wrow[b] = (const uint8_t *)p.b + min(c0 + 16 * b + (lane & 15), p.n - 1) * p.k;
#pragma unroll
    for (int b = 0; b < MB; ++b) xrow[b] = (const uint8_t *)p.a + min((int64_t)16 * b + (lane & 15), p.m - 1) * p.k;
    few_sums<IN_I8, RB, MB, U>(red, wrow, xrow, (int)p.k);
    for (int i = threadIdx.x; i < 16 * RB * (int)p.m; i += kFewThreads) {
        const int ch = i % (16 * RB), tk = i / (16 * RB);
        const int64_t c = c0 + ch;
        if (c >= p.n) continue;
        const float bias = p.bias ? load_float(p.bias, c, p.bias_dtype) : 0.0f;
        store_one<CT>(p.c, tk * p.n + c, few_join<IN_I8, RB, MB>(red, tk, ch) * p.a_scale[tk] * p.b_scale[c] + bias);
    }
}

template <int CT, int RB, int MB, int U>
void go_few(const I8Args &a, hipStream_t s)
{
    k_i8_few<CT, RB, MB, U><<<(unsigned)((a.n + 16 * RB - 1) / (16 * RB)), kFewThreads, 0, s>>>(a);
}

template <int CT, int MI, int NB, int NS, bool PF>
void go(const I8Args &a, hipStream_t s)
{
    const int mt = (int)((a.m + 64 * MI - 1) / (64 * MI)), nt = (int)((a.n + 64 * NB - 1) / (64 * NB));
    k_i8<CT, MI, NB, NS, PF><<<(unsigned)mt * (unsigned)nt, 256, 0, s>>>(a, mt, nt);
}

}  // namespace

int64_t workspace_gemm_i8(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_i8(const I8Args &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    const bool big = (a.m + 255) / 256 * ((a.n + 255) / 256) >= 128;
    auto by_tile = [&](auto ct) {
        constexpr int C = decltype(ct)::value;
        if (a.m <= 16) go_few<C, 1, 1, 4>(a, s);
        else if (a.m <= 32) go_few<C, 1, 2, 2>(a, s);
        else if (a.m <= 64) go_few<C, 2, 4, 2>(a, s);
        else if (big) go<C, 4, 4, 2, true>(a, s);
        else go<C, 2, 2, 4, false>(a, s);
    };
    if (a.c_dtype == DT_F32) by_tile(std::integral_constant<int, DT_F32>{});
    else if (a.c_dtype == DT_F16) by_tile(std::integral_constant<int, DT_F16>{});
    else by_tile(std::integral_constant<int, DT_BF16>{});
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
