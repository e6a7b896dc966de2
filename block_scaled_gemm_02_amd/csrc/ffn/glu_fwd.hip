// gemm_glu, gemm_glu_i8: H = act(X Wg^T) * (X Wu^T).
//
// G and U stay in fp32 (int32 sums times their scales) up to H, which is
// rounded once; where they are kept they are rounded by themselves.  bf16 8192
// x 8192 x 4096 with both kept: 748-765 us, 1440-1470 TFLOP/s, 76% MFMA busy at
// the power limit (on zeros 535 us); int8 4001 x 8192 x 4096 with gelu: 200-210
// us, of which a quarter are prologues and epilogues of four rounds of tiles;
// fp16 509 x 2048 x 7168: 39-41 us, waiting for the loads into LDS (Small tiles,
// 709 MB, 18 TB/s over the card), and 54.8 us from operands that no cache holds.
#include "few.hpp"

namespace bsg {
namespace ffn {
namespace {

// A tile holds TN / 2 columns of H: of the B panel's rows for each wave's
// quadrant half are gate rows and half the up rows of the same columns, so
// that a lane's gate and up sums belong to the same elements of H.  DT: the
// type of H (and of G and U, stored if SAVE).
template <int IN, int DT, int ACT, bool SAVE, class S, bool SPLIT>
__global__ __launch_bounds__(256, S::kWaves) void k_glu(GluArgs p, int mt, int nt, int splits)
{
    typedef typename S::template Of<IN, true, true> T;
    constexpr int MI = S::MI, NB = S::NB, ES = in_bytes(IN);
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    const int lane = threadIdx.x & 63, w = wave_id();
    const int64_t ld = p.k * ES;
    const auto [at, part] = tile_of_block<SPLIT>(blockIdx.x, mt, nt, splits);
    const Split sp = split_of(part, SPLIT ? splits : 1, pairs_of(ld));
    const int64_t m0 = (int64_t)S::TM * at.m, h0 = (int64_t)(S::TN / 2) * at.n;
    typename T::LA la;
    typename T::LB lb;
    {
        const int64_t r = m0 + S::TM / 4 * w, c = h0 + S::TN / 4 * (w >> 1);
        la.init_k((const uint8_t *)p.x + r * ld, (p.m - r) * ld, ld, ld, w, lane);
        lb.init_k((const uint8_t *)(w & 1 ? p.w_up : p.w_gate) + c * ld, (p.n - c) * ld, ld, ld, w, lane);
    }
    auto seek = [&](int pair) {
        la.seek(sp.at(pair));
        lb.seek(sp.at(pair));
    };
    f32x4 acc[2 * MI][2 * NB];
    T t;
    constexpr int HW = NB / 2, HC = 32 * HW;
    const int64_t r0 = m0 + 32 * MI * (w >> 1), c0 = h0 + HC * (w & 1);
    const int rows = (int)min((int64_t)32 * MI, p.m - r0), cols = (int)min((int64_t)HC, p.n - c0);
    // scales, in registers over the K loop: a row's for each 16-row block, and of the
    // wave's HC <= 64 columns lane l holds gate (l) and up scale
    float rs[2 * MI], gs = 0.0f, us = 0.0f;
    if constexpr (IN == IN_I8 && !SPLIT) {
#pragma unroll
        for (int i = 0; i < 2 * MI; ++i) rs[i] = 16 * i + (lane & 15) < rows ? p.x_scale[r0 + 16 * i + (lane & 15)] : 0.0f;
        if (lane < cols) {
            gs = p.gate_scale[c0 + lane];
            us = p.up_scale[c0 + lane];
        }
    }
    t.run(acc, ring, la, lb, sp.count, seek);
    uint8_t *const reg = ring + w * T::kStage;
    if constexpr (SPLIT) {
        // sums of the gate columns [0, n) and the up columns [n, 2n)
        float *const dst = (float *)p.workspace + (sp.index * p.m + r0) * 2 * p.n + c0;
        put_sums<HW, 0>(acc, reg, dst, 2 * p.n, rows, cols, lane);
        put_sums<HW, HW>(acc, reg, dst + p.n, 2 * p.n, rows, cols, lane);
    } else {
        constexpr int kReg = 32 * StageGeom<2, HW>::RBP;
        static_assert(3 * kReg <= T::kStage && kReg + 512 <= T::kStage, "the staging fits the wave's part of the ring");
        float *const cs = reinterpret_cast<float *>(reg + kReg);   // gate, then up scales of the columns (integers)
        if constexpr (IN == IN_I8) {
            if (lane < HC) {
                cs[lane] = gs;
                cs[HC + lane] = us;
            }
        }
        const uint32_t row_bytes = (uint32_t)(2 * p.n);
        static_for<MI>([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            __builtin_amdgcn_sched_barrier(0);
            pin(acc[2 * i], acc[2 * i + 1]);
            // four gate or up values (block column j) of row 16 hh + l%16
            auto quad = [&](auto hh, auto jj) {
                constexpr int r = 2 * i + decltype(hh)::value, j = decltype(jj)::value;
                const f32x4 v = acc[r][j];
                float4 x = make_float4(v[0], v[1], v[2], v[3]);
                if constexpr (IN == IN_I8) {
                    const float4 s = *reinterpret_cast<const float4 *>(cs + 16 * j + 4 * (lane >> 4));
                    x.x = (float)__float_as_int(x.x) * rs[r] * s.x;
                    x.y = (float)__float_as_int(x.y) * rs[r] * s.y;
                    x.z = (float)__float_as_int(x.z) * rs[r] * s.z;
                    x.w = (float)__float_as_int(x.w) * rs[r] * s.w;
                }
                return x;
            };
            auto up = [&](auto hh, auto jj) { return quad(hh, std::integral_constant<int, decltype(jj)::value + 2 * HW>{}); };
            auto h = [&](auto hh, auto jj) {
                const float4 g = quad(hh, jj), u = up(hh, jj);
                return make_float4(act_value<ACT>(g.x) * u.x, act_value<ACT>(g.y) * u.y, act_value<ACT>(g.z) * u.z,
                                   act_value<ACT>(g.w) * u.w);
            };
            const int64_t o = 2 * ((r0 + 32 * i) * p.n + c0);
            stage_block<DT, HW>(reg, lane, h);
            if constexpr (SAVE) {
                stage_block<DT, HW>(reg + kReg, lane, quad);
                stage_block<DT, HW>(reg + 2 * kReg, lane, up);
            }
            flush_block<2, HW>(reg, (char *)p.h + o, row_bytes, rows - 32 * i, 2 * cols, lane);
            if constexpr (SAVE) {
                flush_block<2, HW>(reg + kReg, (char *)p.g + o, row_bytes, rows - 32 * i, 2 * cols, lane);
                flush_block<2, HW>(reg + 2 * kReg, (char *)p.u + o, row_bytes, rows - 32 * i, 2 * cols, lane);
            }
        });
    }
}

// Joins the splits' sums: four columns a thread.
template <int IN, int DT, int ACT, bool SAVE>
__global__ __launch_bounds__(256) void k_glu_join(GluArgs p, int splits)
{
    const int64_t i = 256ll * blockIdx.x + threadIdx.x, n4 = p.n / 4;
    if (i >= p.m * n4) return;
    const int64_t r = i / n4, c = i % n4 * 4;
    const float *const src = (const float *)p.workspace + r * 2 * p.n + c;
    float gs[4], us[4], rs = 0;
    if constexpr (IN == IN_I8) {
        rs = p.x_scale[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            gs[e] = p.gate_scale[c + e];
            us[e] = p.up_scale[c + e];
        }
    }
    float4 g = join4<IN>(src, 2 * p.m * p.n, splits), u = join4<IN>(src + p.n, 2 * p.m * p.n, splits);
    if constexpr (IN == IN_I8) {
        g = make_float4(g.x * rs * gs[0], g.y * rs * gs[1], g.z * rs * gs[2], g.w * rs * gs[3]);
        u = make_float4(u.x * rs * us[0], u.y * rs * us[1], u.z * rs * us[2], u.w * rs * us[3]);
    }
    store4<DT>(p.h, 4 * i, make_float4(act_value<ACT>(g.x) * u.x, act_value<ACT>(g.y) * u.y, act_value<ACT>(g.z) * u.z,
                                       act_value<ACT>(g.w) * u.w));
    if constexpr (SAVE) {
        store4<DT>(p.g, 4 * i, g);
        store4<DT>(p.u, 4 * i, u);
    }
}

// A few tokens: of a workgroup's 16 weight rows 8 are gate rows and 8 the up
// rows of the same channels.
template <int IN, int DT, int ACT, bool SAVE, int MB, int U>
__global__ __launch_bounds__(kFewThreads) void k_glu_few(GluArgs p)
{
    __shared__ __attribute__((aligned(16))) float red[kFewWaves * 16 * MB * 16];
    const int lane = threadIdx.x & 63;
    const int64_t c0 = 8ll * blockIdx.x, ld = p.k * in_bytes(IN);
    const uint8_t *const wrow = (const uint8_t *)(lane & 8 ? p.w_up : p.w_gate) + (c0 + (lane & 7)) * ld, *xrow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) xrow[b] = (const uint8_t *)p.x + min((int64_t)16 * b + (lane & 15), p.m - 1) * ld;
    // this thread's output; its scales come while the weights do
    static_assert(8 * 16 * MB <= kFewThreads, "one output a thread");
    const int ch = threadIdx.x % 8, tk = threadIdx.x / 8;
    const int64_t c = c0 + ch, o = tk * p.n + c;
    const bool in = tk < p.m;
    float rs = 0, gs = 0, us = 0;
    if (IN == IN_I8 && in) {
        rs = p.x_scale[tk];
        gs = p.gate_scale[c];
        us = p.up_scale[c];
    }
    few_sums<IN, MB, U>(red, wrow, xrow, (int)ld);
    if (!in) return;
    float g = few_join<IN, MB>(red, tk, ch), u = few_join<IN, MB>(red, tk, 8 + ch);
    if constexpr (IN == IN_I8) {
        g = g * rs * gs;
        u = u * rs * us;
    }
    store_one<DT>(p.h, o, act_value<ACT>(g) * u);
    if constexpr (SAVE) {
        store_one<DT>(p.g, o, g);
        store_one<DT>(p.u, o, u);
    }
}

template <int IN, int DT, int ACT, bool SAVE, int MB, int U>
void go_few(const GluArgs &a, hipStream_t s)
{
    k_glu_few<IN, DT, ACT, SAVE, MB, U><<<(unsigned)(a.n / 8), kFewThreads, 0, s>>>(a);
}

template <int IN, int DT, bool SAVE>
void launch(const GluArgs &a, hipStream_t s)
{
    with_act(a.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        const Form f = form_gemm_glu(a.m, a.n, a.k, IN == IN_I8);
        if (f.few == 16) return go_few<IN, DT, A, SAVE, 1, 2>(a, s);
        if (f.few == 32) return go_few<IN, DT, A, SAVE, 2, 2>(a, s);
        if (f.few == 64) return go_few<IN, DT, A, SAVE, 4, 1>(a, s);
        const Plan &p = f.tiles;
        with_shape(p, [&](auto shape, auto split) {
            k_glu<IN, DT, A, SAVE, decltype(shape), decltype(split)::value><<<p.grid(), 256, 0, s>>>(a, p.mt, p.nt, p.splits);
        });
        if (p.splits > 1) k_glu_join<IN, DT, A, SAVE><<<(unsigned)((a.m * a.n / 4 + 255) / 256), 256, 0, s>>>(a, p.splits);
    });
}

}  // namespace

int64_t workspace_gemm_glu(int64_t m, int64_t n, int64_t k, bool in_i8)
{
    const Form f = form_gemm_glu(m, n, k, in_i8);
    return !f.few && f.tiles.splits > 1 ? 8 * m * n * f.tiles.splits : 0;
}

hipError_t launch_gemm_glu(const GluArgs &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    if (a.in_i8) {
        if (a.dtype == DT_F16) launch<IN_I8, DT_F16, false>(a, s);
        else launch<IN_I8, DT_BF16, false>(a, s);
    } else if (a.dtype == DT_F16) {
        if (a.g) launch<IN_F16, DT_F16, true>(a, s);
        else launch<IN_F16, DT_F16, false>(a, s);
    } else {
        if (a.g) launch<IN_BF16, DT_BF16, true>(a, s);
        else launch<IN_BF16, DT_BF16, false>(a, s);
    }
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
