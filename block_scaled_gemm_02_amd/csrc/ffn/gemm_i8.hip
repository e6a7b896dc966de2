// gemm_i8: C = (A B^T) * a_scale * b_scale + bias from 8-bit integers.
//
// int32 sums; each is converted to fp32, which rounds it to 24 bits, only to
// meet its scales, and C is rounded once more to its type.  8192^3 runs in
// 374-384 us, 2860-2940 TOPS, the matrix cores 76% busy at the clock that the
// power limit leaves (on zeros 280 us); 67 x 4096, K 7168 in 4 parts in 13.2
// us, and in 16.9 from weights that no cache holds, 14 of them the tiles, on
// half of the compute units.
#include "few.hpp"

namespace bsg {
namespace ffn {
namespace {

// Element i of a float tensor of a run-time type.  No branch on the type: the
// loads of several elements then go out together (two halves of an fp32).
__device__ __forceinline__ float load_float(const void *p, int64_t i, int dt)
{
    const bool f32 = dt == DT_F32;
    const uint16_t *const h = (const uint16_t *)p + (f32 ? 2 * i : i);
    const uint32_t lo = h[0], hi = h[f32 ? 1 : 0];
    const float half = (float)__builtin_bit_cast(_Float16, (uint16_t)lo), wide = __uint_as_float(hi << 16 | (f32 ? lo : 0u));
    return dt == DT_F16 ? half : wide;
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
    f32x4 acc[2 * MI][2 * NB];
    T t;
    const int64_t r0 = m0 + 32 * MI * (w >> 1), c0 = n0 + 32 * NB * (w & 1);
    const int rows = (int)min((int64_t)32 * MI, p.m - r0), cols = (int)min((int64_t)32 * NB, p.n - c0);
    // scales and bias, in registers over the K loop: a row's for each 16-row block,
    // and columns l and l + 64 of the wave's in lane l
    constexpr int CL = (NB + 1) / 2;
    float rs[2 * MI], sc[CL], bi[CL];
    if constexpr (!SPLIT) {
#pragma unroll
        for (int i = 0; i < 2 * MI; ++i) rs[i] = 16 * i + (lane & 15) < rows ? p.a_scale[r0 + 16 * i + (lane & 15)] : 0.0f;
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
            pin(acc[2 * i], acc[2 * i + 1]);
            stage_block<CT, NB>(reg, lane, [&](auto hh, auto jj) {
                constexpr int r = 2 * i + decltype(hh)::value, j = decltype(jj)::value;
                const int c = 16 * j + 4 * (lane >> 4);
                const float4 s = *reinterpret_cast<const float4 *>(cs + c), b = *reinterpret_cast<const float4 *>(cb + c);
                const f32x4 x = acc[r][j];
                return make_float4((float)__float_as_int(x[0]) * rs[r] * s.x + b.x, (float)__float_as_int(x[1]) * rs[r] * s.y + b.y,
                                   (float)__float_as_int(x[2]) * rs[r] * s.z + b.z, (float)__float_as_int(x[3]) * rs[r] * s.w + b.w);
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
    if (i >= p.m * n4) return;
    const int64_t r = i / n4, c = i % n4 * 4;
    // (scales and bias on their way before the sums, which take longest)
    const float rs = p.a_scale[r], *const cs = p.b_scale + c;
    const float s0 = cs[0], s1 = cs[1], s2 = cs[2], s3 = cs[3];
    float b0 = 0, b1 = 0, b2 = 0, b3 = 0;
    if (p.bias) {
        b0 = load_float(p.bias, c, p.bias_dtype);
        b1 = load_float(p.bias, c + 1, p.bias_dtype);
        b2 = load_float(p.bias, c + 2, p.bias_dtype);
        b3 = load_float(p.bias, c + 3, p.bias_dtype);
    }
    const float4 s = join4<IN_I8>((const float *)p.workspace + 4 * i, p.m * p.n, splits);
    store4<CT>(p.c, 4 * i, make_float4(s.x * rs * s0 + b0, s.y * rs * s1 + b1, s.z * rs * s2 + b2, s.w * rs * s3 + b3));
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
    // this thread's outputs, (token, channel) number threadIdx.x + 512 e; their
    // scales come while the weights do
    constexpr int N = (16 * 16 * MB + kFewThreads - 1) / kFewThreads;
    float rs[N], cs[N], bias[N];
    const int ch = threadIdx.x % 16;
    const int64_t c = c0 + ch;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int tk = (threadIdx.x + kFewThreads * e) / 16;
        const bool in = tk < p.m && c < p.n;
        rs[e] = in ? p.a_scale[tk] : 0.0f;
        cs[e] = in ? p.b_scale[c] : 0.0f;
        bias[e] = in && p.bias ? load_float(p.bias, c, p.bias_dtype) : 0.0f;
    }
    few_sums<IN_I8, MB, U>(red, wrow, xrow, (int)p.k);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int tk = (threadIdx.x + kFewThreads * e) / 16;
        if (tk < p.m && c < p.n) store_one<CT>(p.c, tk * p.n + c, few_join<IN_I8, MB>(red, tk, ch) * rs[e] * cs[e] + bias[e]);
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
    const Form f = form_gemm_i8(a.m, a.n, a.k);
    if (f.few == 16) return go_few<CT, 1, 2>(a, s);
    if (f.few == 32) return go_few<CT, 2, 2>(a, s);
    if (f.few == 64) return go_few<CT, 4, 1>(a, s);
    const Plan &p = f.tiles;
    with_shape(p, [&](auto shape, auto split) {
        k_i8<CT, decltype(shape), decltype(split)::value><<<p.grid(), 256, 0, s>>>(a, p.mt, p.nt, p.splits);
    });
    if (p.splits > 1) k_i8_join<CT><<<(unsigned)((a.m * a.n / 4 + 255) / 256), 256, 0, s>>>(a, p.splits);
}

}  // namespace

int64_t workspace_gemm_i8(int64_t m, int64_t n, int64_t k)
{
    const Form f = form_gemm_i8(m, n, k);
    return !f.few && f.tiles.splits > 1 ? 4 * m * n * f.tiles.splits : 0;
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
