// Products of a few tokens: the weights are read once and bound the time.
//
// A workgroup of 8 waves computes 16 weight rows (output channels) for up to
// 16 MB tokens.  The waves split K: wave w takes the 128-byte pieces w,
// w + 8, ... of every row, straight into registers in the layout of the 16x16
// MFMAs (lane (r = l%16, g = l/16) holds 16 bytes of row r), U pieces ahead,
// and the 8 partial sums are joined in LDS, in a fixed order.  So every
// weight is read by one wave once, no barrier stands in the loop, and a
// narrow output still has a workgroup for every 16 (gated: 8) channels.
// Weights are the MFMA's first operand: register v of lane (t, g) is channel
// 4g + v of token t.
//
// Bound by HBM and, when small, by its launch (about 2.5 us).  Sets of weights
// in turn that no cache holds (640 MB of them) / that the 256 MB memory-side
// cache does: gated bf16 1 x 2048 x 7168 (58.7 MB) 12.5 us, 4.7 TB/s / 10.7; 1 x
// 8192 x 4096 (134 MB) 26.9 us, 5.0 TB/s (a large copy reaches 4.9); gated int8
// 8 x 2048 x 7168 (29.5 MB) 8.4 us / 7.6; int8 1 x 7168 x 2048 (14.7 MB) 5.2 us
// / 4.9.  (The order in which workgroups walk K made no difference.)
#pragma once
#include "tile.hpp"

namespace bsg {
namespace ffn {

template <int IN>
__device__ __forceinline__ f32x4 mfma16(const i32x4 &w, const i32x4 &x, const f32x4 &acc)
{
    if constexpr (IN == IN_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
    else if constexpr (IN == IN_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), acc, 0, 0, 0);
    else
        return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, __builtin_bit_cast(i32x4, acc), 0, 0, 0));
}

constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;

// Sums over K of 16 weight rows against 16 MB tokens.  wrow: this lane's
// weight row; xrow: its token of block b (a row or token past the last one
// repeats it: it is not stored).  The result is left in red: partial w of
// (token, channel) at red[(w * 16 MB + token) * 16 + channel].
template <int IN, int MB, int U>
__device__ __forceinline__ void few_sums(float *red, const uint8_t *wrow, const uint8_t *const (&xrow)[MB],
                                         int kbytes)
{
    const int lane = threadIdx.x & 63, w = wave_id(), g = lane >> 4;
    struct Piece {
        i32x4 w[2], x[MB][2];
    };
    f32x4 acc[MB] = {};
    auto load = [&](Piece &p, int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            p.w[h] = *reinterpret_cast<const i32x4 *>(wrow + k + 64 * h + 16 * g);
#pragma unroll
            for (int b = 0; b < MB; ++b) p.x[b][h] = *reinterpret_cast<const i32x4 *>(xrow[b] + k + 64 * h + 16 * g);
        }
    };
    auto mma = [&](const Piece &p) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < MB; ++t) acc[t] = mfma16<IN>(p.w[h], p.x[t][h], acc[t]);
    };
    // whole pieces of this wave, U at a time, the next ones on their way
    const int full = kbytes / 128, mine = full > w ? (full - w + kFewWaves - 1) / kFewWaves : 0;
    const int rounds = mine / U;
    auto at = [&](int i) { return 128 * (w + kFewWaves * i); };
    if (rounds) {
        Piece cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) load(cur[u], at(u));
        for (int r = 1; r < rounds; ++r) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Piece p = cur[u];
                load(cur[u], at(r * U + u));
                mma(p);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) mma(cur[u]);
    }
    for (int i = rounds * U; i < mine; ++i) {
        Piece p;
        load(p, at(i));
        mma(p);
    }
    // the last, partial piece: chunks past K are zeros on both sides
    if (kbytes % 128 && w == full % kFewWaves) {
        Piece p;
        const int k = 128 * full;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = k + 64 * h + 16 * g < kbytes;
            p.w[h] = i32x4{0, 0, 0, 0};
            if (in) p.w[h] = *reinterpret_cast<const i32x4 *>(wrow + k + 64 * h + 16 * g);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                p.x[b][h] = i32x4{0, 0, 0, 0};
                if (in) p.x[b][h] = *reinterpret_cast<const i32x4 *>(xrow[b] + k + 64 * h + 16 * g);
            }
        }
        mma(p);
    }
#pragma unroll
    for (int t = 0; t < MB; ++t) *reinterpret_cast<f32x4 *>(red + (w * 16 * MB + 16 * t + (lane & 15)) * 16 + 4 * g) = acc[t];
    __syncthreads();
}

// The joined sum of (token, channel), as the accumulator's type gives it.
template <int IN, int MB>
__device__ __forceinline__ float few_join(const float *red, int token, int channel)
{
    const float *p = red + token * 16 + channel;
    constexpr int S = 16 * MB * 16;
    if constexpr (IN == IN_I8) {
        int s = 0;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) s += __float_as_int(p[w * S]);
        return (float)s;
    } else {
        float s = p[0];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) s += p[w * S];
        return s;
    }
}

template <int DT>
__device__ __forceinline__ void store_one(void *p, int64_t i, float v)
{
    if constexpr (DT == DT_F32) ((float *)p)[i] = v;
    else if constexpr (DT == DT_F16) ((_Float16 *)p)[i] = (_Float16)v;
    else ((__bf16 *)p)[i] = (__bf16)v;
}

}  // namespace ffn
}  // namespace bsg
