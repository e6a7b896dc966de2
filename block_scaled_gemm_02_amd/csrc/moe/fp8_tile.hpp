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
// and run beside the MFMAs, but they need the sums in vector registers: from
// AGPRs each value would take two moves more, past the MFMA's own time.  That
// bounds a wave to 128 x 64.  B is the MFMA's first operand, so that a lane holds
// four columns of one row and needs one factor for them.
//
// The LDS holds a ring of slots, a K block of A, of B and of A's scales each,
// filled by direct-to-LDS loads; reads past a row, a tensor or the K range
// return zeros (buffer range check).  128 bytes of K are one line of a row; its
// 16-byte chunk c lies at c ^ s(r), so that a fragment read meets every bank
// once (ffn/tile.hpp), and a lane's scales, rows r, r + 16, ... of the wave's, lie
// four together on banks that 16 lanes share out (two rows of lanes on the same
// banks took 27 cycles a block and wave).
//
// The largest tile (256 x 256, EARLY) has two slots.  A wave holds one block's
// columns and four of its eight rows of fragments (240 of 256 registers), and
// a block has two barriers.  At its second row of MFMAs every wave has the
// columns in registers, and B's part of the slot is filled again; three rows before
// its end every wave has the last row, the next block has landed, and A's part
// follows, while the next block's fragments are read between the last MFMAs.  So
// B's loads have 1.75 blocks to land and A's one.  With B filled again beside A,
// weights from HBM came too late: 32 experts of 4096 x 7168, 32768 rows 873 us for
// 813, 64 experts of that with 4 rows each 372 us for 318 (5.9 TB/s).  Half of A
// early too (the barrier then has to wait for its reads), loads all in one row of
// MFMAs, or lines prefetched into the L2 cost 2 to 7%.  The last three results of
// a block are added in the next one, so that no wave waits for them.
// The smallest (64 x 128, WHOLE) holds two blocks' fragments and has one barrier
// a block, at its beginning (25.6 us for 23.5 at 56 blocks).
//
// A workgroup's tiles follow each other in the ring.  What bounds the largest
// one: with all compute units at work the power limit; 8192^3 takes 424-449 us by
// card, 2450-2590 TFLOP/s, the matrix cores 67% busy at the clock that is left (on
// zeros 320 us; without the multiply-adds 9% less).  Each tile's way out costs 5
// us, 128 KB of C a compute unit.
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

// lds_load16 and lds_load4 of a descriptor that a vector instruction may just have
// written: the compiler brings scalar registers back from vector ones where it
// ran out of them, and does not look into assembly for the 5 wait states that a
// memory instruction then needs.  The largest tile takes the loads without them:
// between its MFMAs they cost 1.5 to 2.5% (8192^3 427 -> 437 us, 8192 tokens
// through 32 experts 886 -> 906), and the compiler restores its descriptors long
// before.  That is no promise, so the build checks every load (wait_states.py).
__device__ __forceinline__ void lds_load16_late(const i32x4 &rsrc, uint8_t *dst, uint32_t voff)
{
    const uint32_t m0 = (uint32_t)(uintptr_t)(lds_void *)dst;
    asm volatile("s_nop 2\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(m0), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
__device__ __forceinline__ void lds_load4_late(const i32x4 &rsrc, uint8_t *dst, uint32_t voff)
{
    const uint32_t m0 = (uint32_t)(uintptr_t)(lds_void *)dst;
    asm volatile("s_nop 2\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(m0), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

// What the loads of a tile take: its rows of A and of B, A's scales, and the
// bytes of its K range.  (row 0, K block 0)
struct Source {
    i32x4 ra, rb;
    const float *sa;
    uint32_t klimit, rows;
};
// And what its way out takes.
struct Place {
    char *c;                    // row 0, column 0
    const float *sb;            // of the first 128 columns
    int rows, cols;
};
struct Part {
    Source src;
    Place to;
};

// SUMS: leaves fp32 sums (a part of K) instead of C.
template <int WM_, int WN_, int GM_, int GN_, int S_, bool SUMS_ = false>
struct Fp8Tile {
    static constexpr int WM = WM_, WN = WN_, GM = GM_, GN = GN_, S = S_;
    static constexpr bool SUMS = SUMS_;
    typedef Fp8Tile<WM, WN, GM, GN, S, true> Sums;
    static constexpr int TM = 16 * WM * GM, TN = 16 * WN * GN, W = GM * GN, kThreads = 64 * W;
    static constexpr int kA = TM * 128, kB = TN * 128, kSlot = kA + kB + 256 * W;
    static constexpr int RB = 32 * WN, kRow = RB + 16, kStage = 16 * kRow;      // 16 rows of C on their way out
    static constexpr int kLds = S * kSlot + (SUMS ? 0 : W * kStage);
    static constexpr int LA = TM / 8 / W, LB = TN / 8 / W, L = LA + LB + 1;     // loads of a wave and block
    static constexpr int RW = TM / W;                                           // rows whose scales a wave loads
    static constexpr int kGroups = 160 * 1024 / kLds;                           // workgroups a compute unit
    static constexpr int kWaves = W * kGroups / 4 > 0 ? W * kGroups / 4 : 1;
    static constexpr int C = WM < 4 ? WM : 4;                                   // scales a read
    // Fragments in registers: two whole blocks', or (kAhead rows ahead) those of
    // one block's columns and kRing of its rows, where two do not fit.
    static constexpr bool WHOLE = WM < 4;
    static constexpr int kRing = WHOLE ? WM : 4, kAhead = WHOLE ? WM : 3;
    // B's share of a slot is free, and filled again, when its columns are in registers
    static constexpr bool EARLY = WM >= 8;
    static constexpr int kStores = WM * WN / 2;                                 // of a wave, at the end of a tile
    static constexpr int kMin = WHOLE ? (S + 1) / 2 * 2 : S;                    // least blocks of a tile
    static constexpr int N = WM * WN;
    static_assert(128 % (16 * WN) == 0, "a wave's columns lie in one 128");
    static_assert(LA * 8 * W == TM && LB * 8 * W == TN && RW <= 64 && RW % C == 0 && WM >= 2, "whole loads");
    static_assert(64 % (2 * WN) == 0 && 16 % (32 / WN) == 0, "whole rows a store");

    uint8_t *const lds;
    int lane, w, wm, wn;
    uint32_t ld, chunk, voff, voff_s;
    int64_t sa_ld;
    uint32_t rd_a[2], rd_b[2], rd_s[WM / C];
    int at;                     // the slot of the block at work

    // ld: bytes of a row of A and of B; sa_ld: between A's scales of two blocks
    __device__ __forceinline__ Fp8Tile(uint8_t *ring, int64_t ld, int64_t sa_ld) : lds(ring), ld((uint32_t)ld), sa_ld(sa_ld), at(0)
    {
        lane = threadIdx.x & 63;
        w = ffn::wave_id();
        wm = w / GN;
        wn = w % GN;
        // loads: 8 rows of 128 bytes each
        const uint32_t row = (uint32_t)lane >> 3;
        chunk = 16 * (((uint32_t)lane & 7) ^ ffn::k_swizzle(row));
        voff = row * (uint32_t)ld + chunk;
        // scales: the wave's RW of the tile's TM go to the banks that its neighbours'
        // leave, in the order (i / C, r, i % C) of rows 16 i + r, so that a read of C
        // for each r meets every bank once
        const int sub = w % (64 / RW), q = w * RW + lane - sub * RW, o = q % (16 * WM);
        const int i = o / (16 * C) * C + o % C;
        voff_s = lane / RW == sub ? 4u * (uint32_t)(q - o + 16 * i + o / C % 16) : kOOB;
        // fragment reads
        const uint32_t r = (uint32_t)lane & 15, g = (uint32_t)lane >> 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t c = 16u * ((4u * h + g) ^ ffn::k_swizzle(r));
            rd_a[h] = (16u * WM * wm + r) * 128u + c;
            rd_b[h] = kA + (16u * WN * wn + r) * 128u + c;
        }
#pragma unroll
        for (int h = 0; h < WM / C; ++h) {
            const uint32_t o = 16u * WM * wm + 16 * C * h + C * r, lw = o / RW;
            rd_s[h] = kA + kB + lw * 256 + (lw % (64 / RW) * RW + o % RW) * 4;
        }
    }

    // Load Q of this wave's for K block kb of a tile, into the slot at lds + to.
    // Past the K range it reads nothing.
    template <int Q>
    __device__ __forceinline__ void load(const Source &s, int to, int kb) const
    {
        const uint32_t k = 128u * (uint32_t)kb;
        auto load16 = [&](const i32x4 &r, uint8_t *dst, uint32_t off) {
            if constexpr (EARLY) lds_load16(r, dst, off);
            else lds_load16_late(r, dst, off);
        };
        if constexpr (Q < LA + LB) {
            const uint32_t v = k + chunk < s.klimit ? voff : kOOB;
            if constexpr (Q < LA) load16(s.ra, lds + to + 1024 * (LA * w + Q), v + (8u * (LA * w + Q) * ld + k));
            else load16(s.rb, lds + to + kA + 1024 * (LB * w + Q - LA), v + (8u * (LB * w + Q - LA) * ld + k));
        } else {
            const i32x4 rs = make_rsrc_words(s.sa + kb * sa_ld, k < s.klimit ? 4u * s.rows : 0u);
            if constexpr (EARLY) lds_load4(rs, lds + to + kA + kB + 256 * w, voff_s);
            else lds_load4_late(rs, lds + to + kA + kB + 256 * w, voff_s);
        }
    }
    __device__ __forceinline__ i32x8 frag(int from, const uint32_t (&rd)[2], int off) const
    {
        const i32x4 x = *(const i32x4 *)(lds + from + rd[0] + off), y = *(const i32x4 *)(lds + from + rd[1] + off);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ __forceinline__ void scales(int from, float (&o)[WM]) const
    {
        typedef float V __attribute__((ext_vector_type(C)));
#pragma unroll
        for (int h = 0; h < WM / C; ++h) {
            const V x = *(const V *)(lds + from + rd_s[h]);
#pragma unroll
            for (int c = 0; c < C; ++c) o[C * h + c] = x[c];
        }
    }

    // A wave's fragments and scales at the border of two blocks.
    struct Front {
        i32x8 a[kRing], b[WN];
        float raw[WM];
    };

    // The first S blocks of the first tile.
    __device__ __forceinline__ void start(const Source &s) const
    {
        static_for<S>([&](auto n) {
            static_for<L>([&](auto q) { load<decltype(q)::value>(s, decltype(n)::value * kSlot, decltype(n)::value); });
        });
        s_wait_vm<EARLY ? 0 : (S - 1) * L>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }

    // Blocks that run() is called for: whole steps, and as many as the ring has
    // slots.  What is past the K range counts as zeros.
    static __device__ __forceinline__ int count_of(int blocks)
    {
        return max(WHOLE ? (blocks + 1) & ~1 : blocks, kMin);
    }

    // acc = sum over the `count` blocks of a tile, the first of which has landed,
    // as has that of the next tile, whose loads come from `next`, in the end.  sb:
    // B's scales of the wave's columns, nsb of them; sbv: the first 64, one a lane.
    template <bool AE5>
    __device__ __forceinline__ void run(f32x4 (&acc)[WM][WN], Source src, const Source &next, int count,
                                        const float *sb, int nsb, float sbv)
    {
        auto scale_b = [&](int i) { return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(sbv), i & 63)); };
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        // t: results under way; the last three of a block are added in the next
        // one, with the factors old of its last rows
        float f[WM], old[2] = {0, 0};
        f32x4 t[4] = {};
        auto set_factors = [&](const Front &x, int n) {
            const float sc = scale_b(n);
#pragma unroll
            for (int i = 0; i < WM; ++i) f[i] = x.raw[i] * sc;
        };
        auto refill_scales = [&](int n) {
            if ((n & 63) == 0) {
                sbv = n + lane < nsb ? sb[n + lane] : 0.0f;
                s_wait_vm<0>();
            }
        };
        // the m-th MFMA, of b[j] and a[i], and the addition of an earlier one
        auto mfma = [&](auto mm, const i32x8 &b, const i32x8 &a) {
            constexpr int m = decltype(mm)::value;
            t[m % 4] = mfma128<AE5>(b, a);
            asm volatile("" : "+v"(t[m % 4]));      // (stays here, in the order written)
            if constexpr (m >= 3) add<m - 3>(acc, f[(m - 3) / WN], t);
            else add<N - 3 + m>(acc, old[WM - 1 - (N - 3 + m) / WN], t);
        };
        auto barrier = [&](auto first) {
            // this block's fragments are in registers, the next block has landed
            s_wait_lgkm0();
            if constexpr (decltype(first)::value) s_wait_vm<LB + kStores>();
            else s_wait_vm<(S - 2) * L + (EARLY ? LB : 0)>();
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        };
        auto keep_factors = [&] {
            old[0] = f[WM - 1];
            old[1] = f[WM - 2];
        };
        Front fr;
        scales(at, fr.raw);
#pragma unroll
        for (int j = 0; j < WN; ++j) fr.b[j] = frag(at, rd_b, 2048 * j);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fr.a[i] = frag(at, rd_a, 2048 * i);
        if constexpr (WHOLE) {
            Front other;
            auto step = [&](Front &cur, Front &nxt, int n) {
                const int to = at == (S - 1) * kSlot ? 0 : at + kSlot;
                // the slot's next block, this tile's or the next one's
                const int fill = n + S < count ? n + S : n + S - count;
                if (fill == 0) src = next;
                set_factors(cur, n);
                barrier(std::false_type{});
                constexpr int R = 1 + WN + WM, span = N * 3 / 4;
                static_for<N>([&](auto mm) {
                    constexpr int m = decltype(mm)::value, i = m / WN, j = m % WN;
                    mfma(mm, cur.b[j], cur.a[i]);
                    if constexpr (m < span)
                        static_for<R * (m + 1) / span - R * m / span>([&](auto rr) {
                            constexpr int q = R * m / span + decltype(rr)::value;
                            if constexpr (q == 0) scales(to, nxt.raw);
                            else if constexpr (q <= WN) nxt.b[q - 1] = frag(to, rd_b, 2048 * (q - 1));
                            else nxt.a[q - 1 - WN] = frag(to, rd_a, 2048 * (q - 1 - WN));
                        });
                    static_for<L * (m + 1) / N - L * m / N>([&](auto q) { load<L * m / N + decltype(q)::value>(src, at, fill); });
                    __builtin_amdgcn_sched_barrier(0);
                });
                keep_factors();
                at = to;
            };
            for (int n = 0; n < count; n += 2) {
                if (n) refill_scales(n);
                step(fr, other, n);
                step(other, fr, n + 1);
            }
        } else {
            set_factors(fr, 0);
            // first: a tile's first block.  Its successor's loads went out before the
            // wave's stores of the tile before, which memory instructions, returning in
            // order, need not be waited for; or it has landed (start, run_idle).
            // (weight gradient of 32 x 512 rows, 4096 x 2048: 164 us for 167.5)
            auto step = [&](auto first, int n) {
                const int to = at == (S - 1) * kSlot ? 0 : at + kSlot;
                refill_scales(n + 1);
                const int fill = n + S < count ? n + S : n + S - count;
                if (fill == 0) src = next;
                static_for<N>([&](auto mm) {
                    constexpr int m = decltype(mm)::value, i = m / WN, j = m % WN;
                    // every wave has this block's columns in registers
                    if constexpr (EARLY && i == 1 && j == 0) {
                        __builtin_amdgcn_s_barrier();
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if constexpr (i == WM - kAhead && j == 0) barrier(first);
                    mfma(mm, fr.b[j], fr.a[i % kRing]);
                    // the fragment kAhead rows on, this block's or the next one's
                    if constexpr (j == 0) {
                        constexpr int o = i + kAhead;
                        if constexpr (o < WM) fr.a[o % kRing] = frag(at, rd_a, 2048 * o);
                        else fr.a[o % kRing] = frag(to, rd_a, 2048 * (o - WM));
                    }
                    if constexpr (i == WM - kAhead && j == 1 % WN) scales(to, fr.raw);
                    if constexpr (i == WM - 1) fr.b[j] = frag(to, rd_b, 2048 * j);
                    // refill the slot: columns, then rows
                    constexpr int c = m - (WM - kAhead) * WN, slots = kAhead * WN, early = m - WN, room = (WM - kAhead - 1) * WN;
                    if constexpr (EARLY && early >= 0 && early < room)
                        static_for<(LB * (early + 1)) / room - (LB * early) / room>([&](auto q) {
                            load<LA + (LB * early) / room + decltype(q)::value>(src, at, fill);
                        });
                    if constexpr (!EARLY && c >= 0)
                        static_for<(L * (c + 1)) / slots - (L * c) / slots>([&](auto q) {
                            load<(L * c) / slots + decltype(q)::value>(src, at, fill);
                        });
                    if constexpr (EARLY && c >= 0)
                        static_for<((LA + 1) * (c + 1)) / slots - ((LA + 1) * c) / slots>([&](auto q) {
                            constexpr int x = ((LA + 1) * c) / slots + decltype(q)::value;
                            load<(x < LA ? x : LA + LB)>(src, at, fill);
                        });
                    __builtin_amdgcn_sched_barrier(0);
                });
                keep_factors();
                set_factors(fr, n + 1);
                at = to;
            };
            step(std::bool_constant<EARLY>{}, 0);
            for (int n = 1; n < count; ++n) step(std::false_type{}, n);
        }
        static_for<3>([&](auto mm) {
            constexpr int m = N - 3 + decltype(mm)::value;
            add<m>(acc, old[WM - 1 - m / WN], t);
        });
    }

    // run() of a wave that has no row or no column of the tile: its share of the
    // loads, and the barriers.  The waves that have rows then have the matrix
    // cores to themselves.
    __device__ __forceinline__ void run_idle(Source src, const Source &next, int count)
    {
        for (int n = 0; n < count; ++n) {
            const int fill = n + S < count ? n + S : n + S - count;
            if (fill == 0) src = next;
            if constexpr (EARLY) {
                __builtin_amdgcn_s_barrier();
                static_for<LB>([&](auto q) { load<LA + decltype(q)::value>(src, at, fill); });
            }
            s_wait_vm<(S - 2) * L + (EARLY ? LB : 0)>();
            __builtin_amdgcn_s_barrier();
            static_for<LA>([&](auto q) { load<decltype(q)::value>(src, at, fill); });
            if constexpr (!EARLY) static_for<LB>([&](auto q) { load<LA + decltype(q)::value>(src, at, fill); });
            load<LA + LB>(src, at, fill);
            at = at == (S - 1) * kSlot ? 0 : at + kSlot;
        }
        if constexpr (EARLY) s_wait_vm<0>();
    }
    // acc to C, 16 rows at a time through LDS of its own, so that whole lines are
    // stored.
    template <int CT>
    __device__ __forceinline__ void store(const Place &p, int64_t ldc, const f32x4 (&acc)[WM][WN]) const
    {
        uint8_t *const reg = lds + S * kSlot + w * kStage;
        const int r0 = 16 * WM * wm, c0 = 16 * WN * wn;
        constexpr int LPR = RB / 16, RPI = 64 / LPR;            // lanes a row, rows a store
        const int lr = lane / LPR, cb = lane % LPR * 16;
        const uint32_t row_bytes = (uint32_t)(2 * ldc);
        const uint64_t base = (uint64_t)(uintptr_t)(p.c + 2 * (r0 * ldc + c0));
        const int rows = max(0, min(p.rows - r0, 16 * WM));
        void *const dst = (void *)(uintptr_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(base >> 32)) << 32) |
                                              (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)base));
        const uint32_t n = (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)rows * row_bytes));
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(dst, (short)0, (int)n, 0x00020000);
        const uint32_t voff = cb < 2 * (p.cols - c0) ? (uint32_t)lr * row_bytes + (uint32_t)cb : kOOB;
        // whole 128-byte lines go past the L2, which is left to the operands
        constexpr int kNT = RB % 128 == 0 ? 2 : 0;
        static_for<WM>([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            __builtin_amdgcn_sched_barrier(0);
            static_for<WN>([&](auto jj) {
                const f32x4 x = acc[i][decltype(jj)::value];
                *(uint2 *)(reg + (lane & 15) * kRow + 8 * (lane >> 4) + 32 * decltype(jj)::value) = pack_quad<CT>(x[0], x[1], x[2], x[3]);
            });
#pragma unroll
            for (int k = 0; k < 16 / RPI; ++k) {
                static_assert(WM * (16 / RPI) == kStores, "run() counts them");
                const i32x4 v = *(const i32x4 *)(reg + (lr + k * RPI) * kRow + cb);
                __builtin_amdgcn_raw_buffer_store_b128(v, rs, voff + (uint32_t)(16 * i + k * RPI) * row_bytes, 0, kNT);
            }
        });
    }

    // acc to a part's sums (fp32).
    __device__ __forceinline__ void put_sums(const Place &p, int64_t ldc, const f32x4 (&acc)[WM][WN]) const
    {
        static_for<WM>([&](auto ii) {
            const int r = 16 * (WM * wm + decltype(ii)::value) + (lane & 15);
            static_for<WN>([&](auto jj) {
                const int c = 16 * (WN * wn + decltype(jj)::value) + 4 * (lane >> 4);
                if (r < p.rows && c < p.cols) *(f32x4 *)((float *)p.c + r * ldc + c) = acc[decltype(ii)::value][decltype(jj)::value];
            });
        });
    }

private:
    template <int M>
    static __device__ __forceinline__ void add(f32x4 (&acc)[WM][WN], float f, const f32x4 (&t)[4])
    {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[M / WN][M % WN][v] = fmaf(f, t[M % 4][v], acc[M / WN][M % WN][v]);
    }
};

}  // namespace moe
}  // namespace bsg
