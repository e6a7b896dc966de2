// gemm_glu, gemm_glu_i8: H = act(X Wg^T) * (X Wu^T).
#include "few.hpp"

namespace bsg {
namespace ffn {
namespace {

// A tile holds (32 NB) columns of H: the B panel of a wave's quadrant is half
// gate rows, half up rows, so that a lane's gate and up accumulators belong
// to the same elements of H.
// DT: the type of H (and of G and U, stored if SAVE).
template <int IN, int DT, int ACT, bool SAVE, int MI, int NB, int NS, bool PF>
__global__ __launch_bounds__(256, MI *NB == 16 ? 1 : 2) void k_glu(GluArgs p, int mt, int nt)
{
    typedef Tile<IN, true, true, MI, NB, NS, PF> T;
    constexpr int HW = NB / 2, ES = in_bytes(IN);
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    const int lane = threadIdx.x & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
    const TileAt at = tile_at(blockIdx.x, mt, nt);
    const int64_t ld = p.k * ES, m0 = (int64_t)T::TM * at.m, h0 = (int64_t)(T::TN / 2) * at.n;
    typename T::LA la;
    typename T::LB lb;
    {
        const int64_t r = m0 + T::TM / 4 * w, c = h0 + 16 * NB * (w >> 1);
        la.init_k((const uint8_t *)p.x + r * ld, (p.m - r) * ld, ld, ld, w, lane);
        lb.init_k((const uint8_t *)(w & 1 ? p.w_up : p.w_gate) + c * ld, (p.n - c) * ld, ld, ld, w, lane);
    }
    const int64_t r0 = m0 + 32 * MI * wm, c0 = h0 + 16 * NB * wn;
    const int rows = (int)min((int64_t)32 * MI, p.m - r0), cols = (int)min((int64_t)32 * HW, p.n - c0);
    // scales, in registers over the K loop: a row's for each block, and of
    // the wave's 32 HW columns lane l holds gate (l) and up scale
    float rs[MI], gs = 0.0f, us = 0.0f;
    if constexpr (IN == IN_I8) {
#pragma unroll
        for (int i = 0; i < MI; ++i) rs[i] = 32 * i + (lane & 31) < rows ? p.x_scale[r0 + 32 * i + (lane & 31)] : 0.0f;
        if (lane < min(cols, 32 * HW)) {
            gs = p.gate_scale[c0 + lane];
            us = p.up_scale[c0 + lane];
        }
    }
    f32x16 acc[MI][NB];
    T t;
    t.run(acc, ring, la, lb, pairs_of(ld), [&](int pair) {
        la.seek(pair);
        lb.seek(pair);
    });

    uint8_t *const reg = ring + w * T::kStage;
    constexpr int kReg = 32 * StageGeom<2, HW>::RBP;
    float *const cs = reinterpret_cast<float *>(reg + kReg);   // gate, then up scales of the columns
    if constexpr (IN == IN_I8) {
        cs[lane < 32 * HW ? lane : 64 * HW] = gs;
        cs[lane < 32 * HW ? 32 * HW + lane : 64 * HW] = us;
    }
    const uint32_t row_bytes = (uint32_t)(2 * p.n);
    static_for<MI>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        __builtin_amdgcn_sched_barrier(0);
        pin(acc[i]);
        // the unscaled pre-activations of one quad
        auto quad = [&](auto blk, auto qq) {
            constexpr int b = decltype(blk)::value, q = decltype(qq)::value;
            float4 x = make_float4(acc[i][b][4 * q], acc[i][b][4 * q + 1], acc[i][b][4 * q + 2], acc[i][b][4 * q + 3]);
            if constexpr (IN == IN_I8) {
                const float4 s = *reinterpret_cast<const float4 *>(cs + 32 * b + 8 * q + 4 * (lane >> 5));
                x.x = (float)__float_as_int(x.x) * rs[i] * s.x;
                x.y = (float)__float_as_int(x.y) * rs[i] * s.y;
                x.z = (float)__float_as_int(x.z) * rs[i] * s.z;
                x.w = (float)__float_as_int(x.w) * rs[i] * s.w;
            }
            return x;
        };
        auto up = [&](auto j, auto q) { return quad(std::integral_constant<int, decltype(j)::value + HW>{}, q); };
        auto h = [&](auto j, auto q) {
            const float4 g = quad(j, q), u = up(j, q);
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
    static_assert(3 * kReg + 512 <= T::kStage, "the staging fits the wave's part of the ring");
}

// A few tokens: of a workgroup's 16 RB weight rows the first half are gate
// rows and the second the up rows of the same channels.
template <int IN, int DT, int ACT, bool SAVE, int RB, int MB, int U>
__global__ __launch_bounds__(kFewThreads) void k_glu_few(GluArgs p)
{
    __shared__ __attribute__((aligned(16))) float red[kFewWaves * 16 * MB * 16 * RB];
    constexpr int H = 8 * RB;
    const int lane = threadIdx.x & 63;
    const int64_t c0 = (int64_t)H * blockIdx.x, ld = p.k * in_bytes(IN);
    const uint8_t *wrow[RB], *xrow[MB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int r = 16 * b + (lane & 15);
        wrow[b] = (const uint8_t *)(r < H ? p.w_gate : p.w_up) + min(c0 + r % H, p.n - 1) * ld;
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) xrow[b] = (const uint8_t *)p.x + min((int64_t)16 * b + (lane & 15), p.m - 1) * ld;
    few_sums<IN, RB, MB, U>(red, wrow, xrow, (int)ld);
    for (int i = threadIdx.x; i < H * (int)p.m; i += kFewThreads) {
        const int ch = i % H, tk = i / H;
        const int64_t c = c0 + ch, o = tk * p.n + c;
        if (c >= p.n) continue;
        float g = few_join<IN, RB, MB>(red, tk, ch), u = few_join<IN, RB, MB>(red, tk, H + ch);
        if constexpr (IN == IN_I8) {
            g = g * p.x_scale[tk] * p.gate_scale[c];
            u = u * p.x_scale[tk] * p.up_scale[c];
        }
        store_one<DT>(p.h, o, act_value<ACT>(g) * u);
        if constexpr (SAVE) {
            store_one<DT>(p.g, o, g);
            store_one<DT>(p.u, o, u);
        }
    }
}

template <int IN, int DT, int ACT, bool SAVE, int RB, int MB, int U>
void go_few(const GluArgs &a, hipStream_t s)
{
    k_glu_few<IN, DT, ACT, SAVE, RB, MB, U><<<(unsigned)((a.n + 8 * RB - 1) / (8 * RB)), kFewThreads, 0, s>>>(a);
}

template <int IN, int DT, int ACT, bool SAVE, int MI, int NB, int NS, bool PF>
void go(const GluArgs &a, hipStream_t s)
{
    const int mt = (int)((a.m + 64 * MI - 1) / (64 * MI)), nt = (int)((a.n + 32 * NB - 1) / (32 * NB));
    k_glu<IN, DT, ACT, SAVE, MI, NB, NS, PF><<<(unsigned)mt * (unsigned)nt, 256, 0, s>>>(a, mt, nt);
}

template <int IN, int DT, bool SAVE>
void launch(const GluArgs &a, hipStream_t s)
{
    with_act(a.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        if (a.m <= 16) go_few<IN, DT, A, SAVE, 1, 1, 4>(a, s);
        else if (a.m <= 32) go_few<IN, DT, A, SAVE, 1, 2, 2>(a, s);
        else if (a.m <= 64) go_few<IN, DT, A, SAVE, 2, 4, 2>(a, s);
        else if ((a.m + 255) / 256 * ((a.n + 127) / 128) >= 128) go<IN, DT, A, SAVE, 4, 4, 2, true>(a, s);
        else go<IN, DT, A, SAVE, 2, 2, 4, false>(a, s);
    });
}

}  // namespace

int64_t workspace_gemm_glu(int64_t, int64_t, int64_t, bool) { return 0; }

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
