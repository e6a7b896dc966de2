// The matrix-product tile of the 8-bit float operators with a scale for each
// block of 128 of K.
//
//   C[m, n] = sum_kb  f[kb, m]  sum_{k in kb} a[m, k] b[n, k],
//   f[kb, m] = a_scale[kb, m] b_scale[n / 128, kb]
//
// A workgroup of GM x GN waves computes a (16 WM GM) x (16 WN GN) tile, a wave
// 16 WM rows and 16 WN columns of it, all within one 128 of N.  A K block is
// one 16x16x128 MFMA for each 16 x 16, whose accumulator starts at zero: its
// result cannot stay in the matrix core, because each row's factor changes from
// block to block, so it comes out and is added with a multiply-add for each
// value.  Those take half the vector unit's time at the matrix cores' full rate
// and run beside the MFMAs, but they need the sums in plain registers, which
// bounds a wave to 128 x 64: twelve instructions' registers move between
// AGPRs and VGPRs otherwise.  B is the MFMA's first operand, so that a lane
// holds four columns of one row and needs one factor for 16 rows.
//
// The LDS holds a ring of slots, a K block of A, of B and of A's scales each,
// filled by direct-to-LDS loads; reads past a row, a tensor or the K range
// return zeros (buffer range check).  128 bytes of K are one line of a row; its
// 16-byte chunk c lies at c ^ s(r), so that a fragment read meets every bank
// once (ffn/tile.hpp).  A lane's scales, rows r, r + 16, ... of the wave's, lie
// beside each other.
// One barrier a block, two rows of MFMAs before its end: by then every wave has
// the block's last fragments in registers, and the next block has landed.
// Behind it the slot is filled again, and the next block's first fragments are
// read between the MFMAs of the last ones.
#pragma once
#include "../ffn/tile.hpp"
#include "rows.hpp"

namespace bsg {
namespace moe {

using ffn::f32x4;

// b a^T over 128 of K: register v of lane (r = l%16, g = l/16) is row r of A
// and row 4g + v of B.  Any order of K serves that both operands share.
template <bool AE5>
__device__ __forceinline__ f32x4 mfma128(const i32x8 &b, const i32x8 &a)
{
    const f32x4 zero = {0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, zero, 0, AE5 ? 1 : 0, 0, 0, 0, 0);
}

// One tile's operands: row 0, column 0, K block 0.
struct Part {
    const uint8_t *a, *b;
    const float *sa, *sb;
    int64_t lda, ldb, sa_ld, sb_ld;
    int64_t k;
    int rows, held, cols;       // of C; rows of A that count
    char *c;
};

template <int WM_, int WN_, int GM_, int GN_, int S_>
struct Fp8Tile {
    static constexpr int WM = WM_, WN = WN_, GM = GM_, GN = GN_, S = S_;
    static constexpr int TM = 16 * WM * GM, TN = 16 * WN * GN, W = GM * GN, kThreads = 64 * W;
    static constexpr int kA = TM * 128, kB = TN * 128, kSlot = kA + kB + 256 * W, kLds = S * kSlot;
    static constexpr int LA = TM / 8 / W, LB = TN / 8 / W, L = LA + LB + 1;      // loads of a wave and block
    static constexpr int RW = TM / W;                                            // rows whose scales a wave loads
    static constexpr int kWaves = W * (160 * 1024 / kLds) / 4 > 0 ? W * (160 * 1024 / kLds) / 4 : 1;
    static constexpr int kStage = kLds / W & ~15;
    static_assert(128 % (16 * WN) == 0, "a wave's columns lie in one 128");
    static_assert(LA * 8 * W == TM && LB * 8 * W == TN && RW <= 64 && RW % WM == 0 && WM >= 2, "whole loads");
    static constexpr int kRing = WM % 4 == 0 ? 4 : 2, kAhead = kRing / 2;        // A fragments in registers

    const Part &p;
    uint8_t *const lds;
    int lane, w, wm, wn;
    uint32_t voff_a, voff_b, voff_s, chunk, klimit;
    i32x4 ra, rb;
    uint32_t rd_a[2], rd_b[2], rd_s;

    __device__ __forceinline__ Fp8Tile(const Part &part, uint8_t *ring) : p(part), lds(ring)
    {
        lane = threadIdx.x & 63;
        w = ffn::wave_id();
        wm = w / GN;
        wn = w % GN;
        // loads: 8 rows of 128 bytes each
        const uint32_t row = (uint32_t)lane >> 3;
        chunk = 16 * (((uint32_t)lane & 7) ^ ffn::k_swizzle(row));
        voff_a = row * (uint32_t)p.lda + chunk;
        voff_b = row * (uint32_t)p.ldb + chunk;
        klimit = (uint32_t)p.k;
        ra = make_rsrc_words(p.a, ffn::clamp_bytes(p.held * p.lda));
        rb = make_rsrc_words(p.b, ffn::clamp_bytes(p.cols * p.ldb));
        const int q = w * RW + lane, at = q % (16 * WM);
        voff_s = lane < RW ? 4u * (uint32_t)(q - at + 16 * (at % WM) + at / WM) : kOOB;
        // fragment reads
        const uint32_t r = (uint32_t)lane & 15, g = (uint32_t)lane >> 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t c = 16u * ((4u * h + g) ^ ffn::k_swizzle(r));
            rd_a[h] = (16u * WM * wm + r) * 128u + c;
            rd_b[h] = kA + (16u * WN * wn + r) * 128u + c;
        }
        const uint32_t qr = 16u * WM * wm + r * WM;
        rd_s = kA + kB + qr / RW * 256 + qr % RW * 4;
    }

    // Load Q of this wave's for K block kb, into the slot at lds + at.
    template <int Q>
    __device__ __forceinline__ void load(int at, int kb) const
    {
        const uint32_t k = 128u * (uint32_t)kb;
        if constexpr (Q < LA + LB) {
            const uint32_t add = k + chunk < klimit ? k : kOOB;
            if constexpr (Q < LA)
                lds_load16(ra, lds + at + 1024 * (LA * w + Q), voff_a + add + 8u * (LA * w + Q) * (uint32_t)p.lda);
            else
                lds_load16(rb, lds + at + kA + 1024 * (LB * w + Q - LA), voff_b + add + 8u * (LB * w + Q - LA) * (uint32_t)p.ldb);
        } else {
            const i32x4 rs = make_rsrc_words(p.sa + kb * p.sa_ld, k < klimit ? 4u * (uint32_t)p.held : 0u);
            lds_load4(rs, lds + at + kA + kB + 256 * w, voff_s);
        }
    }
    __device__ __forceinline__ i32x8 frag(int at, const uint32_t (&rd)[2], int off) const
    {
        const i32x4 x = *(const i32x4 *)(lds + at + rd[0] + off), y = *(const i32x4 *)(lds + at + rd[1] + off);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }

    // acc = sum over the K blocks [kb0, kb0 + count), count >= 1.
    template <bool AE5>
    __device__ __forceinline__ void run(f32x4 (&acc)[WM][WN], int kb0, int count)
    {
        const float *const sb = p.sb + (16 * WN * wn) / 128 * p.sb_ld;
        const int sbn = (int)((p.k + 127) / 128);
        // B's scales of 64 blocks, one a lane
        float sbv = kb0 + lane < sbn ? sb[kb0 + lane] : 0.0f;
        auto scale_b = [&](int i) { return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(sbv), i & 63)); };
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        s_wait_vm<0>();
        // past the range a block reads nothing
        auto block = [&](int i) { return i < count ? kb0 + i : 0x00800000; };
#pragma unroll
        for (int s = 0; s < S; ++s) static_for<L>([&](auto q) { load<decltype(q)::value>(s * kSlot, block(s)); });
        s_wait_vm<(S - 1) * L>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        i32x8 a[kRing], b[WN];
        float f[WM];
        f32x4 t[4];
        auto scales = [&](int at, float (&o)[WM]) {
#pragma unroll
            for (int i = 0; i < WM; ++i) o[i] = *(const float *)(lds + at + rd_s + 4 * i);
        };
        float raw[WM];
        scales(0, raw);
#pragma unroll
        for (int j = 0; j < WN; ++j) b[j] = frag(0, rd_b, 2048 * j);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) a[i] = frag(0, rd_a, 2048 * i);
        const float s0 = scale_b(0);
#pragma unroll
        for (int i = 0; i < WM; ++i) f[i] = raw[i] * s0;
        int at = 0;
        for (int n = 0; n < count; ++n) {
            const int next = at == (S - 1) * kSlot ? 0 : at + kSlot;
            if ((n & 63) == 63) {
                sbv = kb0 + n + 1 + lane < sbn ? sb[kb0 + n + 1 + lane] : 0.0f;
                s_wait_vm<0>();
            }
            const int fill = block(n + S);
            static_for<WM * WN>([&](auto mm) {
                constexpr int m = decltype(mm)::value, i = m / WN, j = m % WN;
                if constexpr (i == WM - kAhead && j == 0) {
                    s_wait_lgkm0();
                    s_wait_vm<(S - 2) * L>();
                    __builtin_amdgcn_s_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                }
                t[m % 4] = mfma128<AE5>(b[j], a[i % kRing]);
                if constexpr (m >= 3) add<m - 3>(acc, f, t);
                // the fragment kAhead rows on, this block's or the next one's
                if constexpr (j == 0) {
                    constexpr int o = i + kAhead;
                    if constexpr (o < WM) a[o % kRing] = frag(at, rd_a, 2048 * o);
                    else a[o % kRing] = frag(next, rd_a, 2048 * (o - WM));
                }
                if constexpr (i == WM - kAhead && j == 1 % WN) scales(next, raw);
                if constexpr (i == WM - 1) b[j] = frag(next, rd_b, 2048 * j);
                // refill the slot
                constexpr int c = m - (WM - kAhead) * WN, slots = kAhead * WN;
                if constexpr (c >= 0) {
                    static_for<(L * (c + 1)) / slots - (L * c) / slots>([&](auto q) { load<(L * c) / slots + decltype(q)::value>(at, fill); });
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            add<WM * WN - 3>(acc, f, t);
            add<WM * WN - 2>(acc, f, t);
            add<WM * WN - 1>(acc, f, t);
            const float sc = scale_b(n + 1);
#pragma unroll
            for (int i = 0; i < WM; ++i) f[i] = raw[i] * sc;
            at = next;
        }
        s_wait_vm<0>();
        s_wait_lgkm0();
        __builtin_amdgcn_s_barrier();       // the ring is free: the epilogue stages in it
        __builtin_amdgcn_sched_barrier(0);
    }

private:
    template <int M>
    static __device__ __forceinline__ void add(f32x4 (&acc)[WM][WN], const float (&f)[WM], const f32x4 (&t)[4])
    {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[M / WN][M % WN][v] = fmaf(f[M / WN], t[M % 4][v], acc[M / WN][M % WN][v]);
    }
};

}  // namespace moe
}  // namespace bsg
