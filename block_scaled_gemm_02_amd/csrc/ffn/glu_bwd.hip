// gemm_glu_bwd: dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X, with
// dG = dH * U * act'(G) and dU = dH * act(G).
//
// Three launches: the element-wise pass writes [dG | dU] as one (m, 2n)
// matrix; dX contracts it with the weights as they lie (their K rows are n);
// both weight gradients are one product of 2n rows contracted over the tokens.
#include "tile.hpp"

namespace bsg {
namespace ffn {
namespace {

// dG and dU are rounded to 16 bits here, the type that the matrix cores read;
// G, U and dH are of that type themselves.
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

template <int DT, int MI, int NB, int kStage, class Ptr>
__device__ __forceinline__ void store16(f32x16 (&acc)[MI][NB], uint8_t *reg, int rows, int cols, uint32_t row_bytes,
                                        int lane, Ptr &&dst)
{
    static_assert(32 * StageGeom<2, NB>::RBP <= kStage, "the staging fits the wave's part of the ring");
    static_for<MI>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        __builtin_amdgcn_sched_barrier(0);
        pin(acc[i]);
        stage_block<DT, NB>(reg, lane, [&](auto jj, auto qq) {
            constexpr int j = decltype(jj)::value, q = decltype(qq)::value;
            return make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        });
        dst(i, rows - 32 * i, 2 * cols);
    });
}

// dX: K runs over the n columns of dG against Wg, then of dU against Wu; each
// part is padded to whole pairs with zeros.
template <int IN, int MI, int NB, int NS, bool PF>
__global__ __launch_bounds__(256, MI *NB == 16 ? 1 : 2) void k_dx(GluBwdArgs p, const uint8_t *d, int mt, int nt)
{
    typedef Tile<IN, true, false, MI, NB, NS, PF> T;
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    const int lane = threadIdx.x & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
    const TileAt at = tile_at(blockIdx.x, mt, nt);
    const int64_t m0 = (int64_t)T::TM * at.m, n0 = (int64_t)T::TN * at.n, ld = 4 * p.n, lw = 2 * p.k;
    const int np = pairs_of(2 * p.n);
    typename T::LA la;
    typename T::LB lb;
    const int64_t r = m0 + T::TM / 4 * w;
    const uint8_t *const da = d + r * ld, *const wg = (const uint8_t *)p.w_gate + 2 * n0, *const wu = (const uint8_t *)p.w_up + 2 * n0;
    la.init_k(da, (p.m - r) * ld, ld, 2 * p.n, w, lane);
    lb.init_mn(wg, p.n * lw - 2 * n0, lw, p.k - n0, w, lane);
    f32x16 acc[MI][NB];
    T t;
    t.run(acc, ring, la, lb, 2 * np, [&](int pair) {
        const bool up = pair >= np;
        la.base = up ? da + 2 * p.n : da;
        // the last row's dU ends with the matrix
        la.r = make_rsrc_words(la.base, clamp_bytes((p.m - r) * ld - (up ? 2 * p.n : 0)));
        lb.base = up ? wu : wg;
        la.seek(up ? pair - np : pair);
        lb.seek(up ? pair - np : pair);
    });
    const int64_t r0 = m0 + 32 * MI * wm, c0 = n0 + 32 * NB * wn;
    const int rows = (int)min((int64_t)32 * MI, p.m - r0), cols = (int)min((int64_t)32 * NB, p.k - c0);
    uint8_t *const reg = ring + w * T::kStage;
    store16<dt_of(IN), MI, NB, T::kStage>(acc, reg, rows, cols, (uint32_t)lw, lane, [&](int i, int rv, int cb) {
        flush_block<2, NB>(reg, (char *)p.dx + 2 * ((r0 + 32 * i) * p.k + c0), (uint32_t)lw, rv, cb, lane);
    });
}

// dWg (rows 0 .. n) and dWu (rows n .. 2n)
template <int IN, int MI, int NB, int NS, bool PF>
__global__ __launch_bounds__(256, MI *NB == 16 ? 1 : 2) void k_dw(GluBwdArgs p, const uint8_t *d, int mt, int nt)
{
    typedef Tile<IN, false, false, MI, NB, NS, PF> T;
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    const int lane = threadIdx.x & 63, w = wave_id(), wm = w >> 1, wn = w & 1;
    const TileAt at = tile_at(blockIdx.x, mt, nt);
    const int64_t m0 = (int64_t)T::TM * at.m, n0 = (int64_t)T::TN * at.n, ld = 4 * p.n, lx = 2 * p.k;
    typename T::LA la;
    typename T::LB lb;
    la.init_mn(d + 2 * m0, p.m * ld - 2 * m0, ld, 2 * p.n - m0, w, lane);
    lb.init_mn((const uint8_t *)p.x + 2 * n0, p.m * lx - 2 * n0, lx, p.k - n0, w, lane);
    f32x16 acc[MI][NB];
    T t;
    t.run(acc, ring, la, lb, pairs_of(2 * p.m), [&](int pair) {
        la.seek(pair);
        lb.seek(pair);
    });
    const int64_t r0 = m0 + 32 * MI * wm, c0 = n0 + 32 * NB * wn;
    const int rows = (int)min((int64_t)32 * MI, 2 * p.n - r0), cols = (int)min((int64_t)32 * NB, p.k - c0);
    uint8_t *const reg = ring + w * T::kStage;
    store16<dt_of(IN), MI, NB, T::kStage>(acc, reg, rows, cols, (uint32_t)lx, lane, [&](int i, int rv, int cb) {
        // a 32-row block may straddle the two gradients
        const int64_t row = r0 + 32 * i;
        const int gate = (int)min((int64_t)32, max((int64_t)0, p.n - row));
        flush_block<2, NB>(reg, (char *)p.dw_gate + 2 * (row * p.k + c0), (uint32_t)lx, min(gate, rv), cb, lane);
        // (its rows of dWu start at staged row `gate`)
        flush_block<2, NB>(reg + gate * StageGeom<2, NB>::RBP, (char *)p.dw_up + 2 * ((row + gate - p.n) * p.k + c0),
                           (uint32_t)lx, min(32, rv) - gate, cb, lane);
    });
}

}  // namespace

int64_t workspace_gemm_glu_bwd(int64_t m, int64_t n, int64_t) { return (4 * m * n + 255) / 256 * 256; }

hipError_t launch_gemm_glu_bwd(const GluBwdArgs &a, hipStream_t s)
{
    uint8_t *d = (uint8_t *)a.workspace;
    const int64_t count = a.m * a.n / 8;
    auto by_type = [&](auto in) {
        constexpr int I = decltype(in)::value;
        if (count) {
            with_act(a.act, [&](auto act) {
                k_dact<dt_of(I), decltype(act)::value><<<(unsigned)((count + 255) / 256), 256, 0, s>>>(
                    (const uint4 *)a.dh, (const uint4 *)a.g, (const uint4 *)a.u, (uint4 *)d, count, (uint32_t)(a.n / 8));
            });
        }
        auto go = [&](auto big, int64_t m, int64_t n, auto &&launch) {
            constexpr int E = decltype(big)::value ? 256 : 128;
            const int mt = (int)((m + E - 1) / E), nt = (int)((n + E - 1) / E);
            launch((unsigned)mt * (unsigned)nt, mt, nt);
        };
        auto big = [](int64_t m, int64_t n) { return (m + 255) / 256 * ((n + 255) / 256) >= 128; };
        if (a.dx && a.m && a.k) {
            if (big(a.m, a.k))
                go(std::true_type{}, a.m, a.k, [&](unsigned g, int mt, int nt) { k_dx<I, 4, 4, 2, true><<<g, 256, 0, s>>>(a, d, mt, nt); });
            else
                go(std::false_type{}, a.m, a.k, [&](unsigned g, int mt, int nt) { k_dx<I, 2, 2, 4, false><<<g, 256, 0, s>>>(a, d, mt, nt); });
        }
        if (a.dw_gate && a.n && a.k) {
            if (big(2 * a.n, a.k))
                go(std::true_type{}, 2 * a.n, a.k, [&](unsigned g, int mt, int nt) { k_dw<I, 4, 4, 2, true><<<g, 256, 0, s>>>(a, d, mt, nt); });
            else
                go(std::false_type{}, 2 * a.n, a.k, [&](unsigned g, int mt, int nt) { k_dw<I, 2, 2, 4, false><<<g, 256, 0, s>>>(a, d, mt, nt); });
        }
    };
    if (a.dtype == DT_F16) by_type(std::integral_constant<int, IN_F16>{});
    else by_type(std::integral_constant<int, IN_BF16>{});
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
