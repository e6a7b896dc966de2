// quant_fp8: 8-bit floats with one fp32 scale for each group of 128 values
// along a row, along a column (written transposed), or for each 128 x 128.
//
// A workgroup takes a 128 x 128 piece: thread (r, c) = (t / 16, t % 16) of 256
// holds rows 8r .. 8r + 7 and columns 8c .. 8c + 7 in registers, so a row's
// maximum is one over 16 lanes, a column's one over 8 registers, 4 lanes and
// 4 waves, and the transposed codes are formed 8 rows at a time and turned
// round in the LDS.
// Bound by memory: 16384 x 4096 bf16 both ways (272 MB) takes 58 us, 4.7 TB/s (a
// plain copy reaches 5.4), 47 us with the input in the memory-side cache; 32
// matrices of 2048 x 4096 fp32 in tiles, both ways (1.61 GB), 293 us, 5.5 TB/s.
#include "rows.hpp"

namespace bsg {
namespace moe {
namespace {

template <int DT, bool E5, bool TILE>
__global__ __launch_bounds__(256) void k_quant(QuantFp8Args p)
{
    constexpr int LD = 128 + 16;                // bytes of a staged row
    __shared__ __attribute__((aligned(16))) uint8_t turned[128 * LD];
    __shared__ uint32_t tops[4][128];
    const int t = threadIdx.x, c = t & 15, r = t >> 4, w = t >> 6;
    const int64_t kb = blockIdx.x, mb = blockIdx.y, l = blockIdx.z;
    const int64_t m0 = 128 * mb + 8 * r, k0 = 128 * kb + 8 * c;
    const int64_t kbs = gridDim.x, mbs = gridDim.y;
    Piece<DT, 8> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i].zero();
        if (m0 + i < p.m && k0 < p.k) x[i].load((const char *)p.x + ((l * p.m + m0 + i) * p.k + k0) * es_dt(DT));
    }
    Scale tile{};
    if constexpr (TILE) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = x[i].top(top);
#pragma unroll
        for (int d = 32; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        if ((t & 63) == 0) tops[w][0] = top;
        __syncthreads();
        tile = scale_of<E5>(max(max(tops[0][0], tops[1][0]), max(tops[2][0], tops[3][0])));
        if (t == 0) {
            if (p.q) p.scale[(l * mbs + mb) * kbs + kb] = tile.scale;
            if (p.q_t) p.scale_t[(l * kbs + kb) * mbs + mb] = tile.scale;
        }
    }
    if (p.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            Scale s = tile;
            if constexpr (!TILE) {
                uint32_t top = x[i].top(0);
#pragma unroll
                for (int d = 8; d; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
                s = scale_of<E5>(top);
            }
            if (m0 + i >= p.m) continue;
            if (k0 < p.k)
                store_past((u32x2 *)(p.q + (l * p.m + m0 + i) * p.k + k0),
                           u32x2{codes4<E5>(x[i].at(0), x[i].at(1), x[i].at(2), x[i].at(3), s.inv, s.keep),
                                 codes4<E5>(x[i].at(4), x[i].at(5), x[i].at(6), x[i].at(7), s.inv, s.keep)});
            if (!TILE && c == 0) p.scale[(l * kbs + kb) * p.m + m0 + i] = s.scale;
        }
    }
    if (!p.q_t) return;
    if constexpr (!TILE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i].at(j)) & 0x7FFFFFFFu);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            if ((t & 63) < 16) tops[w][8 * c + j] = top;
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        Scale s = tile;
        if constexpr (!TILE) {
            const int col = 8 * c + j;
            s = scale_of<E5>(max(max(tops[0][col], tops[1][col]), max(tops[2][col], tops[3][col])));
            if (r == 0 && k0 + j < p.k) p.scale_t[(l * mbs + mb) * p.k + k0 + j] = s.scale;
        }
        *(u32x2 *)(turned + (8 * c + j) * LD + 8 * r) =
            u32x2{codes4<E5>(x[0].at(j), x[1].at(j), x[2].at(j), x[3].at(j), s.inv, s.keep),
                  codes4<E5>(x[4].at(j), x[5].at(j), x[6].at(j), x[7].at(j), s.inv, s.keep)};
    }
    __syncthreads();
    // whole rows of the transposed codes: 8 lanes of 16 bytes each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = 32 * i + (t >> 3), o = 16 * (t & 7);
        const int64_t k = 128 * kb + col, m = 128 * mb + o;
        if (k < p.k && m < p.m) store_past((u32x4 *)(p.q_t + (l * p.k + k) * p.m + m), *(const u32x4 *)(turned + col * LD + o));
    }
}

}  // namespace

hipError_t launch_quant_fp8(const QuantFp8Args &a, hipStream_t s)
{
    if (a.l == 0 || a.m == 0 || a.k == 0) return hipSuccess;
    const dim3 grid((unsigned)((a.k + 127) / 128), (unsigned)((a.m + 127) / 128), (unsigned)a.l);
    with_float(a.x_dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (a.q_dtype == DT_E5M2) {
            if (a.tile) k_quant<DT, true, true><<<grid, 256, 0, s>>>(a);
            else k_quant<DT, true, false><<<grid, 256, 0, s>>>(a);
        } else {
            if (a.tile) k_quant<DT, false, true><<<grid, 256, 0, s>>>(a);
            else k_quant<DT, false, false><<<grid, 256, 0, s>>>(a);
        }
    });
    return hipGetLastError();
}

}  // namespace moe
}  // namespace bsg
