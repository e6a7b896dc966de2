// Rows of tokens into expert order and back (moe_gather, moe_combine and
// their gradients).  A map, row_of (tokens, top_k), says which row holds a
// token's choice j, or -1; every row belongs to one pair at most, so all sums
// run over a token's own choices, in their order, and nothing is added
// atomically.
//
// A token's workgroups read it once and write each of its rows (or read each and
// write it once): memory bounds them.  4001 tokens of 7168 bf16 to E4M3 rows, 8
// each (270 MB) 57 us with the sort, 46 us without it; 8192 of 4096 bf16 to 8 rows
// each, padding zeroed (640 MB) 113 us; their gradients back (604 MB) 116 us, 5.2
// TB/s; moe_combine's gradients (1.21 GB) 232 us, 5.2 TB/s (a plain copy reaches
// 5.4, reads alone 6.9, stores alone 5.8).  Few tokens are bound by the launch: 33 of
// 7168 fp16 4.7 us.
#include "rows.hpp"

namespace bsg {
namespace moe {
namespace {

// The row of a token's choice, or -1 for none: what is not in [0, m) is none.
__device__ __forceinline__ int row_at(const int32_t *row_of, int64_t pair, int64_t m)
{
    const int r = row_of[pair];
    return (uint64_t)(uint32_t)r < (uint64_t)m ? r : -1;
}

// Rows of an expert that hold no pair, up to 255 behind moe_sort: four workgroups
// are added for them, which take 64 rows each in turn.
struct Pad {
    int64_t first, last;
    __device__ __forceinline__ int64_t row(int64_t i) const { return first + 256 * (i >> 6) + (i & 63); }
};
__device__ __forceinline__ Pad pad_of(int b, const int32_t *padded_offsets, const int32_t *expert_rows, int64_t m)
{
    const int e = b / 4, q = b % 4;
    const int64_t begin = e ? padded_offsets[e - 1] : 0, end = min((int64_t)padded_offsets[e], m);
    return {max((int64_t)0, begin + expert_rows[e] + 64 * q), end};
}

// Copies 16-byte pieces of rows.
__global__ __launch_bounds__(256) void k_gather(GatherArgs p, int lg, unsigned rows_grid, int64_t pieces)
{
    const int per = 256 >> lg, sub = threadIdx.x >> lg;
    const int64_t col = ((int64_t)blockIdx.y << lg) + (threadIdx.x & ((1 << lg) - 1));
    u32x4 *const y = (u32x4 *)p.y;
    if (blockIdx.x >= rows_grid) {
        const Pad d = pad_of(blockIdx.x - rows_grid, p.padded_offsets, p.expert_rows, p.m);
        for (int64_t i = sub, r; (r = d.row(i)) < d.last; i += per) {
            if (col < pieces) y[r * pieces + col] = u32x4{0, 0, 0, 0};
            if (col == 0 && p.prob) p.prob[r] = 0.0f;
        }
        return;
    }
    const int64_t t = (int64_t)blockIdx.x * per + sub;
    if (t >= p.tokens || col >= pieces) return;
    const u32x4 x = ((const u32x4 *)p.x)[t * pieces + col];
    for (int j = 0; j < p.top_k; ++j) {
        const int r = row_at(p.row_of, t * p.top_k + j, p.m);
        if (r < 0) continue;
        store_past(y + r * pieces + col, x);
        if (col == 0 && p.prob) p.prob[r] = p.weight[t * p.top_k + j];
    }
}

// Quantises pieces of 8 elements on their way; 16 lanes hold a group of 128.
template <int DT>
__global__ __launch_bounds__(256) void k_gather_fp8(GatherArgs p, int lg, unsigned rows_grid, int64_t pieces)
{
    const int per = 256 >> lg, sub = threadIdx.x >> lg;
    const int64_t col = ((int64_t)blockIdx.y << lg) + (threadIdx.x & ((1 << lg) - 1));
    u32x2 *const y = (u32x2 *)p.y;
    const bool first = (col & 15) == 0 && col < pieces;         // of a group
    float *const sc = p.scale + (col >> 4) * p.m;
    if (blockIdx.x >= rows_grid) {
        const Pad d = pad_of(blockIdx.x - rows_grid, p.padded_offsets, p.expert_rows, p.m);
        const float least = scale_of<false>(0).scale;
        for (int64_t i = sub, r; (r = d.row(i)) < d.last; i += per) {
            if (col < pieces) y[r * pieces + col] = u32x2{0, 0};
            if (first) sc[r] = least;
            if (col == 0 && p.prob) p.prob[r] = 0.0f;
        }
        return;
    }
    const int64_t t = (int64_t)blockIdx.x * per + sub;
    const bool in = t < p.tokens && col < pieces;
    Piece<DT, 8> x;
    x.zero();
    if (in) x.load((const char *)p.x + (t * pieces + col) * 8 * es_dt(DT));
    uint32_t top = x.top(0);
#pragma unroll
    for (int d = 8; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if (!in) return;
    const Scale s = scale_of<false>(top);
    const u32x2 q = {codes4<false>(x.at(0), x.at(1), x.at(2), x.at(3), s.inv, s.keep),
                     codes4<false>(x.at(4), x.at(5), x.at(6), x.at(7), s.inv, s.keep)};
    for (int j = 0; j < p.top_k; ++j) {
        const int r = row_at(p.row_of, t * p.top_k + j, p.m);
        if (r < 0) continue;
        store_past(y + r * pieces + col, q);
        if (first) sc[r] = s.scale;
        if (col == 0 && p.prob) p.prob[r] = p.weight[t * p.top_k + j];
    }
}

// out[t] = sum_j weight[t, j] y[row_of[t, j]], in fp32, rounded once.
template <int DT, bool WEIGHT>
__global__ __launch_bounds__(256) void k_combine(CombineArgs p, int lg, int64_t pieces)
{
    constexpr int N = 16 / es_dt(DT);
    const int64_t col = ((int64_t)blockIdx.y << lg) + (threadIdx.x & ((1 << lg) - 1));
    const int64_t t = (int64_t)blockIdx.x * (256 >> lg) + (threadIdx.x >> lg);
    if (t >= p.tokens) return;
    if constexpr (!WEIGHT) {
        if (p.dweight && blockIdx.y == 0)
            for (int j = threadIdx.x & ((1 << lg) - 1); j < p.top_k; j += 1 << lg) {
                const int r = row_at(p.row_of, t * p.top_k + j, p.m);
                p.dweight[t * p.top_k + j] = r < 0 ? 0.0f : p.dprob[r];
            }
    }
    if (col >= pieces || !p.out) return;
    float acc[N] = {};
    // four choices at a time, their rows under way together
    for (int j0 = 0; j0 < p.top_k; j0 += 4) {
        int r[4];
        float w[4];
        Piece<DT, N> y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t pair = t * p.top_k + j0 + j;
            r[j] = j0 + j < p.top_k ? row_at(p.row_of, pair, p.m) : -1;
            w[j] = WEIGHT && j0 + j < p.top_k ? p.weight[pair] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r[j] >= 0) y[j].load((const u32x4 *)p.y + r[j] * pieces + col);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (r[j] < 0) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = WEIGHT ? fmaf(w[j], y[j].at(i), acc[i]) : acc[i] + y[j].at(i);
        }
    }
    ((u32x4 *)p.out)[t * pieces + col] = pack16<DT>(acc);
}

// dy[row] = weight dout[t] and dweight = <dout[t], y[row]>, J choices at a
// time, so that a piece of dout is read once for them and their rows are under
// way together.
template <int DT, int J>
__global__ __launch_bounds__(256) void k_combine_bwd(CombineBwdArgs p, int lg, unsigned rows_grid, int64_t pieces)
{
    constexpr int N = 16 / es_dt(DT);
    const int tpr = 1 << lg, per = 256 >> lg, sub = threadIdx.x >> lg, c0 = threadIdx.x & (tpr - 1);
    u32x4 *const dy = (u32x4 *)p.dy;
    if (blockIdx.x >= rows_grid) {
        const Pad d = pad_of(blockIdx.x - rows_grid, p.padded_offsets, p.expert_rows, p.m);
        for (int64_t i = sub, r; (r = d.row(i)) < d.last; i += per)
            for (int64_t c = c0; c < pieces; c += tpr) dy[r * pieces + c] = u32x4{0, 0, 0, 0};
        return;
    }
    __shared__ float part[J][4];
    const int64_t t = (int64_t)blockIdx.x * per + sub;
    const bool in = t < p.tokens;
    for (int j0 = 0; j0 < p.top_k; j0 += J) {
        int r[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t pair = t * p.top_k + j0 + j;
            r[j] = in && j0 + j < p.top_k ? row_at(p.row_of, pair, p.m) : -1;
            w[j] = r[j] >= 0 && p.weight ? p.weight[pair] : 1.0f;
            dot[j] = 0.0f;
        }
        if (in)
            for (int64_t c = c0; c < pieces; c += tpr) {
                Piece<DT, N> d, y[J];
                d.load((const u32x4 *)p.dout + t * pieces + c);
                if (p.dweight) {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        y[j].zero();
                        if (r[j] >= 0) y[j].load((const u32x4 *)p.y + r[j] * pieces + c);
                    }
                    // (what is not a row of a pair counts as nothing, also where dout is not finite)
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < N; ++i) dot[j] = r[j] >= 0 ? fmaf(d.at(i), y[j].at(i), dot[j]) : 0.0f;
                }
                if (dy) {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        if (r[j] < 0) continue;
                        float o[N];
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = w[j] * d.at(i);
                        store_past(dy + r[j] * pieces + c, pack16<DT>(o));
                    }
                }
            }
        if (!p.dweight) continue;
#pragma unroll
        for (int j = 0; j < J; ++j)
            for (int d = min(tpr, 64) / 2; d; d >>= 1) dot[j] += __shfl_xor(dot[j], d);
        if (tpr > 64) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < J; ++j)
                if ((threadIdx.x & 63) == 0) part[j][threadIdx.x >> 6] = dot[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float *const q = part[j];
                dot[j] = tpr == 128 ? q[2 * sub] + q[2 * sub + 1] : (q[0] + q[1]) + (q[2] + q[3]);
            }
        }
        if (in && c0 == 0)
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j0 + j < p.top_k) p.dweight[t * p.top_k + j0 + j] = dot[j];
    }
}

}  // namespace

hipError_t launch_moe_gather(const GatherArgs &a, hipStream_t s)
{
    const unsigned pads = a.zero_pad ? 4u * (unsigned)a.num_experts : 0u;
    if (a.y_dtype == DT_E4M3) {
        const int64_t pieces = a.hidden / 8;
        const Lay l = lay_of(a.tokens, pieces, 4);
        if (l.rows + pads == 0) return hipSuccess;
        with_float(a.x_dtype, [&](auto dt) {
            k_gather_fp8<decltype(dt)::value><<<dim3(l.rows + pads, l.cols), 256, 0, s>>>(a, l.lg, l.rows, pieces);
        });
    } else {
        const int64_t pieces = a.hidden * es_dt(a.x_dtype) / 16;
        const Lay l = lay_of(a.tokens, pieces, 4);
        if (l.rows + pads == 0) return hipSuccess;
        k_gather<<<dim3(l.rows + pads, l.cols), 256, 0, s>>>(a, l.lg, l.rows, pieces);
    }
    return hipGetLastError();
}

hipError_t launch_moe_combine(const CombineArgs &a, hipStream_t s)
{
    if (a.tokens == 0) return hipSuccess;
    const int64_t pieces = a.hidden * es_dt(a.dtype) / 16;
    const Lay l = lay_of(a.tokens, pieces, 4);
    with_float(a.dtype, [&](auto dt) {
        if (a.weight) k_combine<decltype(dt)::value, true><<<dim3(l.rows, l.cols), 256, 0, s>>>(a, l.lg, pieces);
        else k_combine<decltype(dt)::value, false><<<dim3(l.rows, l.cols), 256, 0, s>>>(a, l.lg, pieces);
    });
    return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const CombineBwdArgs &a, hipStream_t s)
{
    const unsigned pads = a.zero_pad && a.dy ? 4u * (unsigned)a.num_experts : 0u;
    const int64_t pieces = a.hidden * es_dt(a.dtype) / 16;
    const Lay l = lay_of(a.tokens, pieces, 4);
    if (l.rows + pads == 0) return hipSuccess;
    with_float(a.dtype, [&](auto dt) {
        // (as many at a time as a token has, up to 8)
        if (a.top_k <= 2) k_combine_bwd<decltype(dt)::value, 2><<<l.rows + pads, 256, 0, s>>>(a, l.lg, l.rows, pieces);
        else if (a.top_k <= 4) k_combine_bwd<decltype(dt)::value, 4><<<l.rows + pads, 256, 0, s>>>(a, l.lg, l.rows, pieces);
        else k_combine_bwd<decltype(dt)::value, 8><<<l.rows + pads, 256, 0, s>>>(a, l.lg, l.rows, pieces);
    });
    return hipGetLastError();
}

}  // namespace moe
}  // namespace bsg
