// The matrix-product tile of the feed-forward operators: a workgroup of four
// wave64s computes a (64 MI) x (64 NB) tile, each wave a (32 MI) x (32 NB)
// quadrant in 16x16 MFMA blocks whose accumulators stay in registers.
//
// Operands are bf16, fp16 or int8, and any of them is read in 16-byte chunks:
// one MFMA of 16x16x32 (16 bits) or 16x16x64 (8 bits) takes one chunk a lane
// and operand, lane (r = l%16, g = l/16) holding K bytes [16g, 16g + 16) of
// row r.  K advances in pairs of 128 bytes a row (one whole line), in two
// steps of 64 bytes (one MFMA a block).  The 32x32 MFMAs need half the operand
// reads and keep the matrix cores as busy, but their accumulators are read
// and written twice as often, and at these sizes the card runs at its power
// limit: on random operands the 16x16 ones are 9% faster (int8 8192^3 418 ->
// 381 us) and 6% (bf16, gated 8192 x 8192 x 4096, 814 -> 763 us), though on
// zeros they are 1% slower.  (Both now 374-384 and 748-765 us.)
//
// The LDS holds a ring of panels, a pair of A or B each, filled by
// direct-to-LDS loads (buffer_load_dwordx4 ... lds) that no register passes
// through; reads past a row, a tensor or the K range return zeros (buffer
// range check), which is all that ragged sizes need.  Within a pair's second
// step its slots are free (its last fragments are in registers, and a barrier
// says so for all waves), and the loads of a later pair go out between the
// MFMAs.  The fragments of the next step are read between the MFMAs too.
//
// k-major panel (rows of K): row r at 128 r, its 16-byte chunk c at position
// c ^ s(r), s(r) = (r%8) ^ ((r/4)%2).  A 128-bit read of 16 rows and 4 chunks
// is served 16 lanes at a time, of each 32 lanes 0-3, 12-15, 20-23 and 24-27
// and then the others (the bank conflict counter tells: without the second
// term 0.5 conflicts a read, with it none), and s puts those on all 64 banks.
// mn-major panel (16-bit; rows of M or N at each K): K row kk at (2 T) kk, its
// 32-byte block b at b ^ x(kk).  The transposing read (ds_read_b64_tr_b16)
// takes 32 bytes from each of 4 consecutive K rows in a 16-lane group, and
// from the 4 rows 8 further on in the next group; x puts a half wave's 8
// pieces on different banks: kk%4 in 64-byte steps ((kk%4)/2 where a row is
// 128 bytes, T = 64, and its neighbour the other half of the banks) and
// (kk/8)%2 in 32-byte ones.
#pragma once
#include "act.hpp"
#include "plan.hpp"

namespace bsg {
namespace ffn {

enum In : int { IN_BF16 = 0, IN_F16 = 1, IN_I8 = 2 };
constexpr int in_bytes(int in) { return in == IN_I8 ? 1 : 2; }
constexpr int dt_of(int in) { return in == IN_F16 ? DT_F16 : DT_BF16; }

typedef float f32x4 __attribute__((ext_vector_type(4)));

// acc += b a.  Written as assembly with the accumulator tied to AGPRs: of the
// builtin's 64 four-register accumulators the compiler kept copying some
// between the register files, 220 moves a pair of K.
template <int IN>
__device__ __forceinline__ void mfma_into(f32x4 &acc, const i32x4 &b, const i32x4 &a)
{
    if constexpr (IN == IN_BF16) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
    else if constexpr (IN == IN_F16) asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
    else asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}

// mfma_into with a load of 16 bytes a lane into the LDS at dst + OFF + 16 lane.
// One statement, so that nothing of the compiler's comes between M0, which holds
// the LDS address, and the load; the MFMA is the wait state that the two need.
template <int IN, int OFF>
__device__ __forceinline__ void mfma_load(f32x4 &acc, const i32x4 &b, const i32x4 &a, const i32x4 &rsrc, uint8_t *dst, uint32_t voff)
{
    const uint32_t m0 = (uint32_t)(uintptr_t)(lds_void *)dst;
    if constexpr (IN == IN_BF16)
        asm volatile("s_add_u32 m0, %3, %6\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                     : "+a"(acc) : "v"(b), "v"(a), "s"(m0), "v"(voff), "s"(rsrc), "n"(OFF) : "memory", "m0", "scc");
    else if constexpr (IN == IN_F16)
        asm volatile("s_add_u32 m0, %3, %6\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                     : "+a"(acc) : "v"(b), "v"(a), "s"(m0), "v"(voff), "s"(rsrc), "n"(OFF) : "memory", "m0", "scc");
    else
        asm volatile("s_add_u32 m0, %3, %6\n\tv_mfma_i32_16x16x64_i8 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %4, %5, 0 offen lds"
                     : "+a"(acc) : "v"(b), "v"(a), "s"(m0), "v"(voff), "s"(rsrc), "n"(OFF) : "memory", "m0", "scc");
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

// Pairs of a K extent in bytes; an empty sum runs one, of zeros.
__device__ __forceinline__ int pairs_of(int64_t kbytes) { return kbytes > 128 ? (int)((kbytes + 127) / 128) : 1; }

// Readable bytes as a buffer resource takes them.
__device__ __forceinline__ uint32_t clamp_bytes(int64_t b) { return b <= 0 ? 0u : (b < 0x7FFFFFFF ? (uint32_t)b : 0x7FFFFFFFu); }

__device__ __forceinline__ uint32_t k_swizzle(uint32_t row) { return (row & 7) ^ (row >> 2 & 1); }
template <int T>
__device__ __forceinline__ uint32_t mn_swizzle(uint32_t kk)
{
    return (kk >> 3 & 1) + 2 * (T == 64 ? kk >> 1 & 1 : kk & 3);
}

// One wave's share of the loads of a T-row panel: T/32 loads of 1 KB a pair.
// k-major: rows T/4 w ...  of the panel, base at the first of them, `bytes`
// readable from there, K bytes [0, klimit) of each row.  mn-major: base at
// the tile's first column in K row 0, `cols` of its columns exist.
template <bool KM, int T>
struct Loader {
    static constexpr int L = T / 32;
    const uint8_t *base;
    int64_t bytes, step;
    i32x4 r;
    uint32_t v[L], klimit, chunk, add;

    __device__ __forceinline__ void init_k(const uint8_t *b, int64_t n, int64_t ld, int64_t kbytes, int w, int lane)
    {
        base = b;
        bytes = n;
        klimit = (uint32_t)kbytes;
        r = make_rsrc_words(base, clamp_bytes(bytes));
        const uint32_t row = (uint32_t)lane >> 3;
        chunk = 16 * (((uint32_t)lane & 7) ^ k_swizzle(row));
#pragma unroll
        for (int q = 0; q < L; ++q) v[q] = (8 * q + row) * (uint32_t)ld + chunk;
    }
    __device__ __forceinline__ void init_mn(const uint8_t *b, int64_t n, int64_t ld, int64_t cols, int w, int lane)
    {
        base = b;
        bytes = n;
        step = 64 * ld;
        const uint32_t valid = cols < T ? (uint32_t)(2 * cols) : 2u * T;
#pragma unroll
        for (int q = 0; q < L; ++q) {
            const uint32_t p = 1024u * (L * w + q) + 16u * (uint32_t)lane, kk = p / (2 * T), o = p % (2 * T);
            const uint32_t col = o ^ (32u * mn_swizzle<T>(kk));
            v[q] = col < valid ? kk * (uint32_t)ld + col : kOOB;
        }
    }
    // Aims the loads at a pair.
    __device__ __forceinline__ void seek(int pair)
    {
        if constexpr (KM) {
            const uint32_t kb = (uint32_t)pair * 128u;
            add = kb + chunk < klimit ? kb : kOOB;
        } else {
            const int64_t off = (int64_t)pair * step;
            r = make_rsrc_words(base + off, clamp_bytes(bytes - off));
        }
    }
    // Load Q of the wave's share of the panel: its offset in the tensor.  In the
    // LDS it goes to 1024 Q past the wave's part.
    template <int Q>
    __device__ __forceinline__ uint32_t offset() const { return v[Q] + (KM ? add : 0u); }
    static __device__ __forceinline__ uint8_t *part(uint8_t *panel, int w) { return panel + 1024 * L * w; }
};

// Fragment reads of one wave from a panel: C blocks of 16 rows.
template <bool KM, int T, int C>
struct Reader {
    static constexpr int kReads = KM ? C : 2 * C;      // of a step
    uint32_t off[KM ? 2 : C];
    // row0: the wave's first row (column) in the panel
    __device__ __forceinline__ void init(int row0, int lane)
    {
        const uint32_t r = (uint32_t)lane & 15, g = (uint32_t)lane >> 4;
        if constexpr (KM) {
#pragma unroll
            for (int h = 0; h < 2; ++h) off[h] = ((uint32_t)row0 + r) * 128u + 16u * ((4u * h + g) ^ k_swizzle(r));
        } else {
            // (rows 32 H + 4 e on exchange the same way)
            const uint32_t kk = 8u * g + (r >> 2);
#pragma unroll
            for (int c = 0; c < C; ++c)
                off[c] = kk * (2u * T) + 32u * (((uint32_t)row0 / 16u + c) ^ mn_swizzle<T>(kk)) + 8u * (r & 3);
        }
    }
    // Read Q of the step in half H of a pair.
    template <int H, int Q>
    __device__ __forceinline__ void read(i32x4 (&f)[C], const uint8_t *panel) const
    {
        if constexpr (KM) {
            f[Q] = *reinterpret_cast<const i32x4 *>(panel + off[H] + 2048 * Q);
        } else {
            constexpr int c = Q / 2, e = Q % 2;
            const uint8_t *p = panel + off[c] + (32 * H + 4 * e) * 2 * T;
            const auto x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_void *)p);
            const i32x2_t u = __builtin_bit_cast(i32x2_t, x);
            if constexpr (e == 0) {
                f[c].x = u.x;
                f[c].y = u.y;
            } else {
                f[c].z = u.x;
                f[c].w = u.y;
            }
        }
    }
};

template <int MI, int NB>
struct Frag {
    i32x4 a[2 * MI], b[2 * NB];
};

// The ring of a tile and the K loop over it: NA slots for A panels, NB_ for
// B panels.  With one more for B (NB_ = NA + 1 = 3, the largest tile, whose
// ring then fills the 160 KB) the loads of a pair are staggered: B's go out a
// step before A's, half as many a step, and have a step longer to land.
template <int IN, bool AK, bool BK, int MI, int NB, int NA, int NB_>
struct Tile {
    static constexpr int TM = 64 * MI, TN = 64 * NB;
    static constexpr bool STAG = NB_ > NA;
    static_assert(NB_ == NA || (STAG && NA == 2 && NB_ == 3), "the ring's slots");
    static constexpr int kA = TM * 128, kB = TN * 128, kRing = NA * kA + NB_ * kB, kLds = kRing;
    static constexpr int kStage = kRing / 4 & ~15;          // epilogue staging bytes of a wave
    typedef Loader<AK, TM> LA;
    typedef Loader<BK, TN> LB;
    static constexpr int kM = 4 * MI * NB;                  // MFMAs of a step
    Reader<AK, TM, 2 * MI> ra;
    Reader<BK, TN, 2 * NB> rb;
    static constexpr int kR = Reader<AK, TM, 2 * MI>::kReads + Reader<BK, TN, 2 * NB>::kReads;
    static constexpr int kRSpan = kM * 3 / 4 > 0 ? kM * 3 / 4 : 1;

    template <int H, int Q>
    __device__ __forceinline__ void read1(Frag<MI, NB> &f, const uint8_t *pa, const uint8_t *pb) const
    {
        constexpr int RA = Reader<AK, TM, 2 * MI>::kReads;
        if constexpr (Q < RA) ra.template read<H, Q>(f.a, pa);
        else rb.template read<H, Q - RA>(f.b, pb);
    }
    // Load Q of a step that loads A (WA) and / or B panels: its offset, and the
    // load behind an MFMA, or by itself.
    template <bool WA, int Q>
    __device__ __forceinline__ uint32_t offset1(const LA &la, const LB &lb) const
    {
        if constexpr (WA && Q < LA::L) return la.template offset<Q>();
        else return lb.template offset<Q - (WA ? LA::L : 0)>();
    }
    template <bool WA, int Q>
    __device__ __forceinline__ void mfma_load1(f32x4 &acc, const i32x4 &b, const i32x4 &a, const LA &la, const LB &lb, uint8_t *pa,
                                               uint8_t *pb, int w, uint32_t voff) const
    {
        if constexpr (WA && Q < LA::L) mfma_load<IN, 1024 * Q>(acc, b, a, la.r, LA::part(pa, w), voff);
        else mfma_load<IN, 1024 * (Q - (WA ? LA::L : 0))>(acc, b, a, lb.r, LB::part(pb, w), voff);
    }
    template <int Q>
    __device__ __forceinline__ void load1(const LA &la, const LB &lb, uint8_t *pa, uint8_t *pb, int w) const
    {
        if constexpr (Q < LA::L) lds_load16(la.r, LA::part(pa, w) + 1024 * Q, la.template offset<Q>());
        else lds_load16(lb.r, LB::part(pb, w) + 1024 * (Q - LA::L), lb.template offset<Q - LA::L>());
    }
    // The load, of L in a step, that MFMA m carries (-1: none): spread evenly,
    // with the first MFMA left free where there are two or more for each.
    static constexpr int load_of(int m, int l)
    {
        if (l == 0) return -1;
        if (kM >= 2 * l) return m % (kM / l) == 1 && m / (kM / l) < l ? m / (kM / l) : -1;
        return l * (m + 1) / kM > l * m / kM ? l * m / kM : -1;
    }

    // One step: MFMAs on cur, fragments of the next step (of panels ra_, rb_)
    // into nxt, and loads into the panels pa and pb.  An MFMA of 16 cycles
    // covers about three other instructions, so reads and loads are dealt out
    // one by one, and a load's offset is formed one MFMA ahead of it.
    template <bool ODD, class Seek>
    __device__ __forceinline__ void step(f32x4 (&acc)[2 * MI][2 * NB], Frag<MI, NB> &cur, Frag<MI, NB> &nxt, LA &la, LB &lb,
                                         const uint8_t *ra_, const uint8_t *rb_, uint8_t *pa, uint8_t *pb, int w, Seek &&seek)
    {
        constexpr bool WA = ODD, WB = ODD != STAG;
        constexpr int L = (WA ? LA::L : 0) + (WB ? LB::L : 0);
        if constexpr (ODD) {
            // the next pair has landed; what may be in flight are the pairs
            // after it, or (staggered) the B panel after it
            s_wait_vm<STAG ? LB::L : (NA - 2) * (LA::L + LB::L)>();
            s_wait_lgkm0();
            __builtin_amdgcn_s_barrier();
        } else {
            s_wait_lgkm0();
            seek();                  // aim at the pair that this step and the next one load
        }
        __builtin_amdgcn_sched_barrier(0);
        static_assert(L <= kM, "at most one load an MFMA");
        uint32_t voff = 0;
        if constexpr (load_of(0, L) == 0) voff = offset1<WA, 0>(la, lb);
        static_for<kM>([&](auto mm) {
            // columns back and forth, so that neighbours share an operand (0.5%)
            constexpr int m = decltype(mm)::value, i = m / (2 * NB), c = m % (2 * NB), j = i % 2 ? 2 * NB - 1 - c : c;
            constexpr int q = load_of(m, L), next = m + 1 < kM ? load_of(m + 1, L) : -1;
            if constexpr (q >= 0) mfma_load1<WA, q>(acc[i][j], cur.b[j], cur.a[i], la, lb, pa, pb, w, voff);
            else mfma_into<IN>(acc[i][j], cur.b[j], cur.a[i]);
            if constexpr (next >= 0) voff = offset1<WA, next>(la, lb);
            if constexpr (m < kRSpan) {
                static_for<(kR * (m + 1)) / kRSpan - (kR * m) / kRSpan>([&](auto rr) {
                    read1<ODD ? 0 : 1, (kR * m) / kRSpan + decltype(rr)::value>(nxt, ra_, rb_);
                });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    }

    // acc = sum over np >= 1 pairs.  seek(p) aims la and lb at the p-th pair,
    // which past the last one has to read nothing.  The loop body is one block
    // without branches and runs at least once.
    template <class Seek>
    __device__ __forceinline__ void run(f32x4 (&acc)[2 * MI][2 * NB], uint8_t *ring, LA &la, LB &lb, int np, Seek &&seek)
    {
        const int lane = threadIdx.x & 63, w = wave_id();
#pragma unroll
        for (int i = 0; i < 2 * MI; ++i)
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        ra.init(32 * MI * (w >> 1), lane);
        rb.init(32 * NB * (w & 1), lane);
        uint8_t *const ringb = ring + NA * kA;
#pragma unroll
        for (int s = 0; s < NA; ++s) {
            seek(s);
            static_for<LA::L + LB::L>([&](auto q) { load1<decltype(q)::value>(la, lb, ring + s * kA, ringb + s * kB, w); });
        }
        s_wait_vm<(NA - 1) * (LA::L + LB::L)>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        Frag<MI, NB> fx, fy;
        static_for<kR>([&](auto q) { read1<0, decltype(q)::value>(fx, ring, ringb); });
        auto next_a = [&](uint8_t *p) { return p == ring + (NA - 1) * kA ? ring : p + kA; };
        auto next_b = [&](uint8_t *p) { return p == ringb + (NB_ - 1) * kB ? ringb : p + kB; };
        uint8_t *a = ring, *b = ringb;                      // panels of the current pair
        int pair = 0;
        do {
            uint8_t *const a1 = next_a(a), *const b1 = next_b(b);
            // staggered: the B panel two pairs on has a slot of its own already
            step<false>(acc, fx, fy, la, lb, a, b, a, STAG ? next_b(b1) : b, w, [&] { seek(pair + NA); });
            step<true>(acc, fy, fx, la, lb, a1, b1, a, b, w, [] {});
            a = a1;
            b = b1;
        } while (++pair < np);
        asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
        s_wait_vm<0>();
        s_wait_lgkm0();
        __builtin_amdgcn_s_barrier();       // the ring is free: the epilogue stages in it
        __builtin_amdgcn_sched_barrier(0);
    }
};

// The sum of `parts` partial sums of four columns, `stride` floats apart, the
// first at p; integers are added as integers.
// Four at a time, so that their latencies overlap.
template <int IN>
__device__ __forceinline__ float4 join4(const float *p, int64_t stride, int parts)
{
    typedef std::conditional_t<IN == IN_I8, i32x4, f32x4> V;
    auto at = [&](int i) { return *reinterpret_cast<const V *>(p + i * stride); };
    V s = at(0);
    int i = 1;
    for (; i + 4 <= parts; i += 4) {
        const V a = at(i), b = at(i + 1), c = at(i + 2), d = at(i + 3);
        s = s + a + b + c + d;
    }
    for (; i < parts; ++i) s = s + at(i);
    return make_float4((float)s[0], (float)s[1], (float)s[2], (float)s[3]);
}
template <int DT>
__device__ __forceinline__ void store4(void *p, int64_t i, float4 v)
{
    *reinterpret_cast<typename Quad<es_of<DT>()>::T *>((char *)p + i * es_of<DT>()) = pack_quad<DT>(v.x, v.y, v.z, v.w);
}

// The tile shapes: Big for products with enough 256 x 256 tiles, the others
// with more and smaller ones.  Mid's ring holds four pairs, for a compute unit
// that has one tile; Shared is the same tile on half the LDS, for products of
// more than 256 of them: two workgroups share a compute unit and one's first
// loads and epilogue hide behind the other (us, Mid / Shared: int8 2048 x 4096,
// K 2048 24.3 / 20.5; gated bf16 2000 x 2048, K 4096 64.2 / 57.5; the gradients
// of 1003 x 1408 x 2048 36.2 / 30.7; but int8 67 x 4096, K 7168 in 4 parts, one
// workgroup a compute unit, 13.3 / 14.1).  Below Big the loads into the LDS set
// the time, not the matrix cores: 32 KB (Mid) or 24 KB (Small) a pair for 512 or
// 256 cycles of MFMA.  With all compute units at work that is 18-20 TB/s over
// the card, 30-40 bytes a cycle for each; with half of them a Mid tile's pair
// takes 0.36 us for 0.47.  So it is something that the units share, and what
// has not been found: with K longer by one or two 128-byte lines, which spreads
// a pair's rows otherwise over the L2s, a product takes the same time a pair.
// Cold operands come on top of it: gated fp16 509 x 2048 x 7168 (68 MB) 38.9 us
// from the memory-side cache, 54.8 from HBM.  (Letting the four waves divide a
// pair's K instead of the tile, so that no fragment is read from LDS twice,
// gained nothing for that reason and its joining of the four sums cost 2 us.)
template <int MI_, int NB_, int SA, int SB>
struct Shape {
    static constexpr int MI = MI_, NB = NB_, TM = 64 * MI, TN = 64 * NB;
    static constexpr int kWaves = 128 * (SA * TM + SB * TN) <= 80 * 1024 ? 2 : 1;    // waves a SIMD, by the LDS
    template <int IN, bool AK, bool BK>
    using Of = Tile<IN, AK, BK, MI, NB, SA, SB>;
};
typedef Shape<4, 4, 2, 3> Big;
typedef Shape<2, 2, 4, 4> Mid;
typedef Shape<1, 2, 3, 3> Small;
typedef Shape<2, 2, 2, 3> Shared;

// K divided over workgroups, where a product has fewer tiles than the card
// has compute units: split s of `splits` sums the pairs [first, first + count)
// of all `pairs` and leaves the raw sums in the workspace, for a second kernel
// to join in the order of the splits.
struct Split {
    int index, first, count, pairs;
    // the p-th pair of the split, or one past all of K, which reads nothing
    __device__ __forceinline__ int at(int p) const { return p < count ? first + p : pairs; }
};
__device__ __forceinline__ Split split_of(int index, int splits, int pairs)
{
    const int a = (int)((int64_t)pairs * index / splits), b = (int)((int64_t)pairs * (index + 1) / splits);
    return {index, a, b - a, pairs};
}

// f(shape, std::bool_constant<split>)
template <class F>
void with_shape(const Plan &p, F &&f)
{
    if (p.shape == 0) f(Big{}, std::false_type{});
    else if (p.shape == 2) f(Small{}, std::false_type{});
    else if (p.shape == 3) f(Shared{}, std::false_type{});
    else if (p.splits == 1) f(Mid{}, std::false_type{});
    else f(Mid{}, std::true_type{});
}

// Order of workgroups: b runs on XCD b % 8, and each XCD has an L2 of its own.
// The sequence is cut into rounds of 256 (a workgroup a CU), and each round
// into one run an XCD, so that neighbours in the sequence share an L2.
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t total)
{
    const uint32_t first = b / 256 * 256, round = min(256u, total - first), x = b % 8;
    return first + x * (round / 8) + min(x, round % 8) + (b - first) / 8;
}

struct TileAt {
    int m, n;
};
// Tiles in squares of 16 x 16, a square in strips of 4 rows: an XCD's run is 4
// x 8 tiles, whose 12 panels its L2 streams once, and a round is a square,
// whose 32 panels come from memory once.
__device__ __forceinline__ TileAt tile_at(uint32_t b, uint32_t mt, uint32_t nt)
{
    constexpr uint32_t Q = 16, G = 4;
    const uint32_t s = xcd_run(b, mt * nt);
    const uint32_t sq = s / (Q * nt), r = s % (Q * nt), rows = min(Q, mt - sq * Q);
    const uint32_t c = r / (rows * Q), r2 = r % (rows * Q), cols = min(Q, nt - c * Q);
    const uint32_t st = r2 / (G * cols), r3 = r2 % (G * cols), g = min(G, rows - st * G);
    return {(int)(sq * Q + st * G + r3 % g), (int)(c * Q + r3 / g)};
}

// A split product: rows fastest, then splits, so that the workgroups that
// read the same piece of the columns' weights share an L2.
struct SplitTile {
    TileAt at;
    int split;
};
__device__ __forceinline__ SplitTile split_tile(uint32_t b, uint32_t mt, uint32_t nt, uint32_t splits)
{
    const uint32_t s = xcd_run(b, mt * nt * splits);
    return {{(int)(s % mt), (int)(s / (mt * splits))}, (int)(s / mt % splits)};
}
template <bool SPLIT>
__device__ __forceinline__ SplitTile tile_of_block(uint32_t b, uint32_t mt, uint32_t nt, uint32_t splits)
{
    if constexpr (SPLIT) return split_tile(b, mt, nt, splits);
    else return {tile_at(b, mt, nt), 0};
}

// Holds two rows of accumulator blocks in their AGPRs up to here: the compiler
// otherwise reads all 256 at the end of the K loop and spills the fragments.
template <int N>
__device__ __forceinline__ void pin(f32x4 (&r0)[N], f32x4 (&r1)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+a"(r0[j]), "+a"(r1[j]));
}

// Epilogue: a 32-row block of a wave's quadrant goes through LDS, so that
// whole row segments are stored.  stage_block writes value(h, j), the four
// columns 16j + 4g .. + 3 of row 16h + l%16 (lane l, g = l/16), W times 32 columns;
// flush_block stores the staged rows at dst (row r at dst + r row_bytes),
// `rows` of which exist, `col_bytes` of each.
template <int DT, int W, class F>
__device__ __forceinline__ void stage_block(uint8_t *reg, int lane, F &&value)
{
    constexpr int ES = es_of<DT>(), RBP = StageGeom<ES, W>::RBP;
    uint8_t *row = reg + (lane & 15) * RBP + 4 * (lane >> 4) * ES;
    static_for<2>([&](auto hh) {
        static_for<2 * W>([&](auto jj) {
            const float4 x = value(hh, jj);
            *reinterpret_cast<typename Quad<ES>::T *>(row + 16 * decltype(hh)::value * RBP + 16 * decltype(jj)::value * ES) =
                pack_quad<DT>(x.x, x.y, x.z, x.w);
        });
    });
}
template <int ES, int W, bool STREAM = true>
__device__ __forceinline__ void flush_block(const uint8_t *reg, void *dst, uint32_t row_bytes, int rows, int col_bytes,
                                            int lane)
{
    typedef StageGeom<ES, W> G;
    static_assert(64 % G::LPR == 0 && 32 % G::RPI == 0, "whole rows a store");
    const int lr = lane / G::LPR, cb = lane % G::LPR * 16;
    const uint64_t base = (uint64_t)(uintptr_t)dst;
    void *const udst = (void *)(uintptr_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(base >> 32)) << 32) |
                                           (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)base));
    const uint32_t n = (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)max(0, min(rows, 32)) * row_bytes));
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(udst, (short)0, (int)n, 0x00020000);
    const uint32_t voff = cb < col_bytes ? (uint32_t)lr * row_bytes + (uint32_t)cb : kOOB;
    // outputs are streamed past the L2 (nt), which is left to the operand
    // panels, where a wave writes whole 128-byte lines
    constexpr int kNT = STREAM && G::RB % 128 == 0 ? 2 : 0;
#pragma unroll
    for (int k = 0; k < G::NK; ++k) {
        const i32x4 v = *reinterpret_cast<const i32x4 *>(reg + (lr + k * G::RPI) * G::RBP + cb);
        __builtin_amdgcn_raw_buffer_store_b128(v, rs, voff + (uint32_t)(k * G::RPI) * row_bytes, 0, kNT);
    }
}

// The raw sums of W accumulator blocks from block column J0 on, to dst (row
// stride ld floats): a split's part of the workspace.
template <int W, int J0, int M2, int N2>
__device__ __forceinline__ void put_sums(f32x4 (&acc)[M2][N2], uint8_t *reg, float *dst, int64_t ld, int rows, int cols, int lane)
{
    static_for<M2 / 2>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        __builtin_amdgcn_sched_barrier(0);
        pin(acc[2 * i], acc[2 * i + 1]);
        stage_block<DT_F32, W>(reg, lane, [&](auto hh, auto jj) {
            const f32x4 x = acc[2 * i + decltype(hh)::value][2 * J0 + decltype(jj)::value];
            return make_float4(x[0], x[1], x[2], x[3]);
        });
        flush_block<4, W, false>(reg, dst + 32 * i * ld, (uint32_t)(4 * ld), rows - 32 * i, 4 * cols, lane);
    });
}

}  // namespace ffn
}  // namespace bsg
