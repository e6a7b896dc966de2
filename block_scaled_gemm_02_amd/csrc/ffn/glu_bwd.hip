// gemm_glu_bwd: dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X, with
// dG = dH * U * act'(G) and dU = dH * act(G).
//
// The element-wise pass writes [dG | dU] as one (m, 2n) matrix.  dX contracts
// it with the weights as they lie (their K rows are n); both weight gradients
// are one product of 2n rows contracted over the tokens.  The two products do
// not depend on each other and go out as one launch where that is cheaper.
// One of them alone keeps its part of that choice, so that its bits do not
// depend on the other; chosen for itself it would be faster (bf16, us, dX alone
// / dWg and dWu alone, in brackets chosen for themselves): 1003 x 1408 x 2048
// 29.9 (24.5) / 24.2 (24.0), 200 x 4528 x 2904 56.5 (30.2, K in parts) / 40.0
// (33.5), 4096 x 1408 x 2048 64.5 (53.2) / 84.1 (62.9).
//
// bf16 8192 x 8192 x 4096: the pass 105 us, 6.3 TB/s (writing dG and dU, and
// reading them back, is what keeps the products plain: formed inside dX they
// would be computed again for every tile of columns); the products 1.47-1.51
// ms, 1450-1500 TFLOP/s, 76% MFMA busy at the power limit.  fp16 1003 x 1408 x
// 2048: 32 us, 4 of them the pass, and the products (Shared tiles) waiting for
// their loads into LDS; 39 us from operands that no cache holds.
#include "tile.hpp"

namespace bsg {
namespace ffn {
namespace {

// dG and dU are rounded to 16 bits here, the type that the matrix cores read;
// G, U and dH are of that type themselves.  It adds one rounding to the
// output's: the gradients are off by 1.41 times what rounding the exact ones
// gives (bf16 0.0023 of their norm for 0.0017, fp16 0.00029 for 0.00021).
// Keeping fp32 would take two 16-bit parts each and twice the MFMAs.  In fp16
// it also bounds their range (65504, 2^-25), which scaling dH moves.
template <int DT, int ACT>
__global__ __launch_bounds__(256) void k_dact(const uint4 *dh, const uint4 *g, const uint4 *u, uint4 *d, int64_t count,
                                              uint32_t n8)
{
    const int64_t i = 256ll * blockIdx.x + threadIdx.x;     // 8 elements each
    if (i >= count) return;
    const uint4 hv = dh[i], gv = g[i], uv = u[i];
    uint4 a, b;
    auto one = [&](uint32_t h, uint32_t gg, uint32_t uu, uint32_t &x, uint32_t &y) {
        const ActGrad p = act_grad<ACT>(lo16<DT>(gg)), q = act_grad<ACT>(hi16<DT>(gg));
        x = pack2<DT>(lo16<DT>(h) * lo16<DT>(uu) * p.d, hi16<DT>(h) * hi16<DT>(uu) * q.d);
        y = pack2<DT>(lo16<DT>(h) * p.v, hi16<DT>(h) * q.v);
    };
    one(hv.x, gv.x, uv.x, a.x, b.x);
    one(hv.y, gv.y, uv.y, a.y, b.y);
    one(hv.z, gv.z, uv.z, a.z, b.z);
    one(hv.w, gv.w, uv.w, a.w, b.w);
    const int64_t r = i / n8, c = i % n8;
    d[r * 2 * n8 + c] = a;
    d[r * 2 * n8 + n8 + c] = b;
}

template <int DT, int M2, int N2, class Flush>
__device__ __forceinline__ void store16(f32x4 (&acc)[M2][N2], uint8_t *reg, int lane, Flush &&flush)
{
    static_for<M2 / 2>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        __builtin_amdgcn_sched_barrier(0);
        pin(acc[2 * i], acc[2 * i + 1]);
        stage_block<DT, N2 / 2>(reg, lane, [&](auto hh, auto jj) {
            const f32x4 x = acc[2 * i + decltype(hh)::value][decltype(jj)::value];
            return make_float4(x[0], x[1], x[2], x[3]);
        });
        flush(i);
    });
}

// dX: K runs over the n columns of dG against Wg, then of dU against Wu; each
// part is padded to whole pairs with zeros.  d: [dG | dU]; sums: the splits'.
template <int IN, class S, bool SPLIT>
__device__ __forceinline__ void dx_tile(const GluBwdArgs &p, const uint8_t *d, float *sums, int mt, int nt, int splits,
                                        uint32_t block, uint8_t *ring)
{
    typedef typename S::template Of<IN, true, false> T;
    constexpr int MI = S::MI, NB = S::NB;
    const int lane = threadIdx.x & 63, w = wave_id();
    const int np = pairs_of(2 * p.n);
    const auto [at, part] = tile_of_block<SPLIT>(block, mt, nt, splits);
    const Split sp = split_of(part, SPLIT ? splits : 1, 2 * np);
    const int64_t m0 = (int64_t)S::TM * at.m, n0 = (int64_t)S::TN * at.n, ld = 4 * p.n, lw = 2 * p.k;
    typename T::LA la;
    typename T::LB lb;
    const int64_t r = m0 + S::TM / 4 * w;
    const uint8_t *const da = d + r * ld, *const wg = (const uint8_t *)p.w_gate + 2 * n0, *const wu = (const uint8_t *)p.w_up + 2 * n0;
    la.init_k(da, (p.m - r) * ld, ld, 2 * p.n, w, lane);
    lb.init_mn(wg, p.n * lw - 2 * n0, lw, p.k - n0, w, lane);
    auto seek = [&](int pair) {
        const int q = sp.at(pair);
        const bool up = q >= np;
        la.base = up ? da + 2 * p.n : da;
        // the last row's dU ends with the matrix
        la.r = make_rsrc_words(la.base, clamp_bytes((p.m - r) * ld - (up ? 2 * p.n : 0)));
        lb.base = up ? wu : wg;
        la.seek(up ? q - np : q);
        lb.seek(up ? q - np : q);
    };
    f32x4 acc[2 * MI][2 * NB];
    T t;
    t.run(acc, ring, la, lb, sp.count, seek);
    const int64_t r0 = m0 + 32 * MI * (w >> 1), c0 = n0 + 32 * NB * (w & 1);
    const int rows = (int)min((int64_t)32 * MI, p.m - r0), cols = (int)min((int64_t)32 * NB, p.k - c0);
    uint8_t *const reg = ring + w * T::kStage;
    static_assert(32 * StageGeom<SPLIT ? 4 : 2, NB>::RBP <= T::kStage, "the staging fits the wave's part of the ring");
    if constexpr (SPLIT) {
        put_sums<NB, 0>(acc, reg, sums + (sp.index * p.m + r0) * p.k + c0, p.k, rows, cols, lane);
    } else {
        store16<dt_of(IN)>(acc, reg, lane, [&](int i) {
            flush_block<2, NB>(reg, (char *)p.dx + 2 * ((r0 + 32 * i) * p.k + c0), (uint32_t)lw, rows - 32 * i, 2 * cols, lane);
        });
    }
}

// dWg (rows 0 .. n) and dWu (rows n .. 2n)
template <int IN, class S, bool SPLIT>
__device__ __forceinline__ void dw_tile(const GluBwdArgs &p, const uint8_t *d, float *sums, int mt, int nt, int splits,
                                        uint32_t block, uint8_t *ring)
{
    typedef typename S::template Of<IN, false, false> T;
    constexpr int MI = S::MI, NB = S::NB;
    const int lane = threadIdx.x & 63, w = wave_id();
    const auto [at, part] = tile_of_block<SPLIT>(block, mt, nt, splits);
    const Split sp = split_of(part, SPLIT ? splits : 1, pairs_of(2 * p.m));
    const int64_t m0 = (int64_t)S::TM * at.m, n0 = (int64_t)S::TN * at.n, ld = 4 * p.n, lx = 2 * p.k;
    typename T::LA la;
    typename T::LB lb;
    la.init_mn(d + 2 * m0, p.m * ld - 2 * m0, ld, 2 * p.n - m0, w, lane);
    lb.init_mn((const uint8_t *)p.x + 2 * n0, p.m * lx - 2 * n0, lx, p.k - n0, w, lane);
    auto seek = [&](int pair) {
        la.seek(sp.at(pair));
        lb.seek(sp.at(pair));
    };
    f32x4 acc[2 * MI][2 * NB];
    T t;
    t.run(acc, ring, la, lb, sp.count, seek);
    const int64_t r0 = m0 + 32 * MI * (w >> 1), c0 = n0 + 32 * NB * (w & 1);
    const int rows = (int)min((int64_t)32 * MI, 2 * p.n - r0), cols = (int)min((int64_t)32 * NB, p.k - c0);
    uint8_t *const reg = ring + w * T::kStage;
    // (a block's second flush may start at any of its rows)
    static_assert(64 * StageGeom<2, NB>::RBP <= T::kStage && 32 * StageGeom<SPLIT ? 4 : 2, NB>::RBP <= T::kStage,
                  "the staging fits the wave's part of the ring");
    if constexpr (SPLIT) {
        put_sums<NB, 0>(acc, reg, sums + (sp.index * 2 * p.n + r0) * p.k + c0, p.k, rows, cols, lane);
    } else {
        store16<dt_of(IN)>(acc, reg, lane, [&](int i) {
            // a 32-row block may straddle the two gradients: its first `gate` rows are dWg's
            const int64_t row = r0 + 32 * i;
            const int rv = min(32, rows - 32 * i), gate = (int)min((int64_t)32, max((int64_t)0, p.n - row));
            flush_block<2, NB>(reg, (char *)p.dw_gate + 2 * (row * p.k + c0), (uint32_t)lx, min(gate, rv), 2 * cols, lane);
            flush_block<2, NB>(reg + gate * StageGeom<2, NB>::RBP, (char *)p.dw_up + 2 * ((row + gate - p.n) * p.k + c0),
                               (uint32_t)lx, rv - gate, 2 * cols, lane);
        });
    }
}

template <int IN, class S, bool SPLIT>
__global__ __launch_bounds__(256, S::kWaves) void k_dx(GluBwdArgs p, const uint8_t *d, float *sums, int mt, int nt, int splits)
{
    __shared__ __attribute__((aligned(16))) uint8_t ring[S::template Of<IN, true, false>::kLds];
    dx_tile<IN, S, SPLIT>(p, d, sums, mt, nt, splits, blockIdx.x, ring);
}
template <int IN, class S, bool SPLIT>
__global__ __launch_bounds__(256, S::kWaves) void k_dw(GluBwdArgs p, const uint8_t *d, float *sums, int mt, int nt, int splits)
{
    __shared__ __attribute__((aligned(16))) uint8_t ring[S::template Of<IN, false, false>::kLds];
    dw_tile<IN, S, SPLIT>(p, d, sums, mt, nt, splits, blockIdx.x, ring);
}
// Both: the tiles with the longer K first (x_first), so that short ones end the launch.
template <int IN, class S>
__global__ __launch_bounds__(256, S::kWaves) void k_dxw(GluBwdArgs p, const uint8_t *d, int xm, int xn, int wm, int wn, int x_first)
{
    static_assert(S::template Of<IN, true, false>::kLds == S::template Of<IN, false, false>::kLds, "one ring for both");
    __shared__ __attribute__((aligned(16))) uint8_t ring[S::template Of<IN, true, false>::kLds];
    const uint32_t first = x_first ? xm * xn : wm * wn, b = blockIdx.x;
    if ((b < first) == (x_first != 0)) dx_tile<IN, S, false>(p, d, nullptr, xm, xn, 1, b < first ? b : b - first, ring);
    else dw_tile<IN, S, false>(p, d, nullptr, wm, wn, 1, b < first ? b : b - first, ring);
}

// Joins the splits' sums of `count4` times four outputs; the first `first4`
// go to out0, the others to out1.
template <int DT>
__global__ __launch_bounds__(256) void k_join(const float *sums, void *out0, void *out1, int64_t first4, int64_t count4, int splits)
{
    const int64_t i = 256ll * blockIdx.x + threadIdx.x;
    if (i >= count4) return;
    const float4 s = join4<IN_BF16>(sums + 4 * i, 4 * count4, splits);
    if (i < first4) store4<DT>(out0, 4 * i, s);
    else store4<DT>(out1, 4 * (i - first4), s);
}

int64_t d_bytes(int64_t m, int64_t n) { return (4 * m * n + 255) / 256 * 256; }

}  // namespace

int64_t workspace_gemm_glu_bwd(int64_t m, int64_t n, int64_t k)
{
    // dX and the weight gradients follow each other: their splits share the space
    const auto [x, w, together] = pair_glu_bwd(m, n, k);
    const int64_t sx = x.splits > 1 ? 4 * m * k * x.splits : 0, sw = w.splits > 1 ? 8 * n * k * w.splits : 0;
    return d_bytes(m, n) + (sx > sw ? sx : sw);
}

hipError_t launch_gemm_glu_bwd(const GluBwdArgs &a, hipStream_t s)
{
    uint8_t *d = (uint8_t *)a.workspace;
    float *sums = (float *)(d + d_bytes(a.m, a.n));
    auto blocks = [](int64_t items) { return (unsigned)((items + 255) / 256); };
    auto by_type = [&](auto in) {
        constexpr int I = decltype(in)::value;
        if (const int64_t count = a.m * a.n / 8) {
            with_act(a.act, [&](auto act) {
                k_dact<dt_of(I), decltype(act)::value><<<blocks(count), 256, 0, s>>>(
                    (const uint4 *)a.dh, (const uint4 *)a.g, (const uint4 *)a.u, (uint4 *)d, count, (uint32_t)(a.n / 8));
            });
        }
        const auto [px, pw, together] = pair_glu_bwd(a.m, a.n, a.k);
        const bool x = a.dx && a.m && a.k, w = a.dw_gate && a.n && a.k;
        if (x && w && together) {
            with_shape(px, [&, &px = px, &pw = pw](auto shape, auto) {
                k_dxw<I, decltype(shape)><<<px.grid() + pw.grid(), 256, 0, s>>>(a, d, px.mt, px.nt, pw.mt, pw.nt, 2 * a.n >= a.m);
            });
            return;
        }
        if (x) {
            with_shape(px, [&, &px = px](auto shape, auto split) {
                k_dx<I, decltype(shape), decltype(split)::value><<<px.grid(), 256, 0, s>>>(a, d, sums, px.mt, px.nt, px.splits);
            });
            const int64_t c = a.m * a.k / 4;
            if (px.splits > 1) k_join<dt_of(I)><<<blocks(c), 256, 0, s>>>(sums, a.dx, nullptr, c, c, px.splits);
        }
        if (w) {
            with_shape(pw, [&, &pw = pw](auto shape, auto split) {
                k_dw<I, decltype(shape), decltype(split)::value><<<pw.grid(), 256, 0, s>>>(a, d, sums, pw.mt, pw.nt, pw.splits);
            });
            const int64_t c = a.n * a.k / 4;
            if (pw.splits > 1) k_join<dt_of(I)><<<blocks(2 * c), 256, 0, s>>>(sums, a.dw_gate, a.dw_up, c, 2 * c, pw.splits);
        }
    };
    if (a.dtype == DT_F16) by_type(std::integral_constant<int, IN_F16>{});
    else by_type(std::integral_constant<int, IN_BF16>{});
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
