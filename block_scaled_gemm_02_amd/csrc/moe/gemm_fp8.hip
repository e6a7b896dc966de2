// gemm_fp8, grouped_gemm_fp8, grouped_gemm_fp8_wgrad: products of 8-bit
// floats with a scale for each block of 128 of K,
//
//   C[m, n] = sum_kb  a_scale[kb, m] b_scale[n / 128, kb]  sum_{k in kb} a[m, k] b[n, k]
//
// C is fp16 or bf16: the matrix instruction (both of the card's 8-bit ones) drops
// of each 8 products the bits below 2^-13 of the largest, towards zero.  That is
// less than 7 * 2^-13 = 8.5e-4 of the sum of magnitudes, at worst more than an
// fp16 rounding, and 5e-5 of the result on random normal operands: the error of
// C against 64 bits is then 1.6615e-3 in bf16 and 2.082e-4 in fp16, that of the
// exact sum rounded 1.6614e-3 and 2.077e-4.  A block's sum, its factor and the
// sum over blocks are fp32; C is rounded once.
//
// Tiles (fp8_tile.hpp) or a kernel for few rows, by plan.hpp.  Measured, calls in a
// row by card: 8192^3 424-449 us; 32768 unevenly routed rows, 32 experts of 4096 x
// 7168, 865-930 us (12% more rows than pairs by the padding, in 8.9 rounds of tiles);
// their gradient of 32 x 4096 x 2048 from 16382 rows 197 us, 247 from HBM (0.69
// GB); 32 tokens through 64 experts of 4096 x 7168 301 us (1.73 GB, 5.8 TB/s); 1 x
// 7168 x 2048 4.3 us, 5.0 from HBM.
#include "../ffn/few.hpp"
#include "fp8_tile.hpp"
#include "plan.hpp"

namespace bsg {
namespace moe {
namespace {

// The expert that holds a row: the number of experts that end at it or before.
__device__ __forceinline__ int expert_of(const int32_t *ends, int num, int64_t row)
{
    int e = 0;
    for (int i = 0; i < num; i += 64) {
        const int j = i + (threadIdx.x & 63);
        e += __popcll(__ballot(j < num && ends[j] <= row));
    }
    return e;
}

// A value that is the same for the whole wave, as a scalar: what a kernel
// loads after it has stored comes in a vector register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The operands of rows [m0, m0 + tm) and columns [n0, n0 + tn) of C, or of
// expert z's C.
__device__ __forceinline__ Part part_of(const Fp8Args &p, int64_t m0, int tm, int64_t n0, int tn, int z)
{
    const int64_t nb = (p.n + 127) / 128, kb = (p.k + 127) / 128;
    const int cols = (int)min((int64_t)tn, p.n - n0);
    int rows = (int)min((int64_t)tm, p.m - m0);
    int64_t k = p.k;
    const uint8_t *a = p.a + m0 * p.k, *b = p.b + n0 * p.k;
    const float *sa = p.a_scale + m0, *sb = p.b_scale + n0 / 128 * kb;
    char *c = (char *)p.c + 2 * (m0 * p.n + n0);
    if (p.group == GROUP_K) {
        const int64_t first = z ? uniform(p.padded_offsets[z - 1]) : 0, last = min((int64_t)uniform(p.padded_offsets[z]), p.k);
        a += first;
        b += first;
        sa += first / 128 * p.m;
        sb += first / 128;
        k = max((int64_t)0, last - first);
        c += 2 * z * p.m * p.n;
    } else if (p.group == GROUP_ROWS) {
        const int e = uniform(expert_of(p.padded_offsets, p.num_experts, m0));
        b += e * p.n * p.k;
        sb += e * nb * kb;
        if (p.expert_rows) {
            const int64_t begin = e ? uniform(p.padded_offsets[e - 1]) : 0;
            rows = (int)max((int64_t)0, min((int64_t)rows, begin + uniform(p.expert_rows[e]) - m0));
        }
    }
    return {{make_rsrc_words(a, ffn::clamp_bytes(rows * p.k)), make_rsrc_words(b, ffn::clamp_bytes(cols * p.k)), sa, (uint32_t)k,
             (uint32_t)rows},
            {c, sb, rows, cols}};
}

// The tiles of one workgroup, in turn.
//
// Big tiles that a last round of at most half the compute units would take go
// out in halves of 128 rows, to twice as many workgroups: a half, whose other
// waves are idle, takes 0.6 of a whole one's time.
template <class T>
struct Stride {
    const Fp8Args &p;
    unsigned mt, nt, total, whole, units, next;
    __device__ __forceinline__ Stride(const Fp8Args &p, unsigned mt, unsigned nt, unsigned splits) : p(p), mt(mt), nt(nt), next(blockIdx.x)
    {
        total = mt * nt * splits;
        whole = total / gridDim.x * gridDim.x;
        const unsigned rest = total - whole;
        if (T::TM < 256 || 2 * rest > gridDim.x) whole = total;
        units = whole + 2 * (total - whole);
    }
    // the next tile that has rows; false behind the last one
    __device__ __forceinline__ bool take(Part &t)
    {
        for (; next < units; next += gridDim.x) {
            unsigned i = next;
            int half = 0;
            if (i >= whole) {
                const unsigned j = i - whole, rest = total - whole;
                half = j >= rest;
                i = whole + (half ? j - rest : j);
            }
            const ffn::TileAt at = ffn::tile_at(i, mt, nt);
            t = part_of(p, (int64_t)T::TM * at.m + T::TM / 2 * half, next < whole ? T::TM : T::TM / 2, (int64_t)T::TN * at.n, T::TN, 0);
            if (t.to.rows > 0) break;
        }
        const bool some = next < units;
        next += gridDim.x;
        return some;
    }
};

// A part of K of a tile each (gemm_fp8).
template <class T>
struct Parts {
    const Fp8Args &p;
    unsigned mt, nt, splits, next;
    __device__ __forceinline__ Parts(const Fp8Args &p, unsigned mt, unsigned nt, unsigned splits)
        : p(p), mt(mt), nt(nt), splits(splits), next(blockIdx.x)
    {
    }
    __device__ __forceinline__ bool take(Part &t)
    {
        if (next >= mt * nt * splits) return false;
        const auto [at, split] = ffn::split_tile(next, mt, nt, splits);
        const ffn::Split s = ffn::split_of(split, (int)splits, (int)((p.k + 127) / 128));
        const int64_t first = 128ll * s.first, m0 = (int64_t)T::TM * at.m, n0 = (int64_t)T::TN * at.n;
        t = part_of(p, m0, T::TM, n0, T::TN, 0);
        // (the bytes of the rows shrink by what their beginning moves)
        t.src.ra = make_rsrc_words(p.a + m0 * p.k + first, ffn::clamp_bytes(t.to.rows * p.k - first));
        t.src.rb = make_rsrc_words(p.b + n0 * p.k + first, ffn::clamp_bytes(t.to.cols * p.k - first));
        t.src.sa += s.first * p.m;
        t.src.klimit = (uint32_t)min(p.k - first, 128ll * s.count);
        t.to.sb += s.first;
        t.to.c = (char *)((float *)p.workspace + (s.index * p.m + m0) * p.n + n0);
        next += gridDim.x;
        return true;
    }
};

// GROUP_K: experts differ in how long their sums are, so the tiles of all of
// them, expert by expert, are cut into a run of equal work for each XCD (a
// tile's way out counts as kOut blocks), and the XCD's workgroups take its run's
// tiles in turn: at any time they share an expert's operands in their L2, and
// each has as many tiles of every expert as the others.
template <class T>
struct Runs {
    static constexpr int kOut = 4;
    const Fp8Args &p;
    unsigned mt, nt, per, step;
    int e, w;                       // the next tile's expert, and the work of each of its tiles
    unsigned index;                 // the next tile of the expert's `per`
    uint64_t begins, end;           // where the expert begins in all the work, and the run ends
    __device__ __forceinline__ int work(int i) const
    {
        if (i >= p.num_experts) return 0;
        const int64_t first = i ? p.padded_offsets[i - 1] : 0, last = min((int64_t)p.padded_offsets[i], p.k);
        return (int)(max((int64_t)0, last - first) / 128) + kOut;
    }
    __device__ __forceinline__ Runs(const Fp8Args &p, unsigned mt, unsigned nt, unsigned) : p(p), mt(mt), nt(nt), per(mt * nt)
    {
        const int lane = threadIdx.x & 63;
        auto scan = [&](int x) {        // sums up to and with this lane
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int o = __shfl_up(x, d);
                x += lane >= d ? o : 0;
            }
            return x;
        };
        uint64_t all = 0;
        for (int i = 0; i < p.num_experts; i += 64) all += (uint32_t)__builtin_amdgcn_readlane(scan(work(i + lane)), 63);
        all *= per;
        const unsigned runs = gridDim.x % 8 ? 1 : 8, run = blockIdx.x % runs;
        step = gridDim.x / runs;
        const uint64_t at = all * run / runs;
        end = all * (run + 1) / runs;
        // the first tile that begins at or behind the run's beginning
        e = p.num_experts;
        w = 1;
        index = 0;
        begins = 0;
        uint64_t before = 0;
        for (int i = 0; i < p.num_experts; i += 64) {
            const int x = work(i + lane), s = scan(x);
            const uint64_t ends = before + (uint64_t)s * per;
            const uint64_t found = __ballot(i + lane < p.num_experts && ends > at);
            if (found) {
                const int l = __builtin_ctzll(found);
                e = i + l;
                w = __builtin_amdgcn_readlane(x, l);
                begins = before + (uint64_t)(uint32_t)(__builtin_amdgcn_readlane(s, l) - w) * per;
                index = at > begins ? (unsigned)((at - begins + w - 1) / w) : 0;
                break;
            }
            before += (uint64_t)(uint32_t)__builtin_amdgcn_readlane(s, 63) * per;
        }
        index += blockIdx.x / runs;
    }
    __device__ __forceinline__ bool take(Part &t)
    {
        while (index >= per && e < p.num_experts) {
            index -= per;
            begins += (uint64_t)(uint32_t)w * per;
            w = uniform(work(++e));
        }
        if (e >= p.num_experts || begins + (uint64_t)(uint32_t)w * index >= end) return false;
        // strips of four rows of tiles, column by column
        const unsigned strip = index / (4 * nt), r = index % (4 * nt), rows = min(4u, mt - 4 * strip);
        t = part_of(p, (int64_t)T::TM * (4 * strip + r % rows), T::TM, (int64_t)T::TN * (r / rows), T::TN, e);
        index += step;
        return true;
    }
};

// A workgroup goes from tile to tile; the loads of a tile's first blocks go out
// in the last blocks of the one before it, so that only the way out of a tile
// keeps the matrix cores waiting.
template <class T, template <class> class Walk, bool AE5, int CT>
__global__ __launch_bounds__(T::kThreads, T::kWaves) void k_fp8(Fp8Args p, unsigned mt, unsigned nt, unsigned splits)
{
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    // rows behind the last expert are no tiles
    if (p.group == GROUP_ROWS)
        mt = (unsigned)((min((int64_t)max(p.padded_offsets[p.num_experts - 1], 0), p.m) + T::TM - 1) / T::TM);
    Walk<T> walk(p, mt, nt, splits);
    Part cur;
    if (!walk.take(cur)) return;
    T tile(ring, p.k, p.m);
    // B's scales of the wave's columns, and the first 64 of them, one a lane: loaded
    // before the stores of the tile before, which nothing then waits for
    auto scales = [&](const Part &t) { return t.to.sb + 16 * T::WN * tile.wn / 128 * ((p.k + 127) / 128); };
    auto first_scales = [&](const Part &t) {
        return 16 * T::WN * tile.wn < t.to.cols && tile.lane < (int)((t.src.klimit + 127) / 128) ? scales(t)[tile.lane] : 0.0f;
    };
    float sbv = first_scales(cur);
    tile.start(cur.src);
    bool more = true;
    while (more) {
        Part then = cur;
        more = walk.take(then);
        if (!more) then.src.klimit = 0;         // nothing after the last tile
        const int blocks = (int)((cur.src.klimit + 127) / 128), count = T::count_of(blocks);
        // (a wave past the last column would also read scales past B's last ones)
        if (cur.to.rows <= 16 * T::WM * tile.wm || cur.to.cols <= 16 * T::WN * tile.wn) {
            tile.run_idle(cur.src, then.src, count);
            if (!more) s_wait_vm<0>();
            sbv = first_scales(then);
        } else {
            f32x4 acc[T::WM][T::WN];
            tile.template run<AE5>(acc, cur.src, then.src, count, scales(cur), blocks, sbv);
            if (!more) s_wait_vm<0>();          // no load is under way to the LDS when the workgroup ends
            sbv = first_scales(then);
            if constexpr (T::SUMS) tile.put_sums(cur.to, p.n, acc);
            else tile.template store<CT>(cur.to, p.n, acc);
        }
        cur = then;
    }
}

// Joins the parts' sums: four columns a thread.
template <int CT>
__global__ __launch_bounds__(256) void k_join(Fp8Args p, int splits)
{
    const int64_t i = 256ll * blockIdx.x + threadIdx.x;
    if (4 * i < p.m * p.n)
        ffn::store4<CT>(p.c, 4 * i, ffn::join4<ffn::IN_BF16>((const float *)p.workspace + 4 * i, p.m * p.n, splits));
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
// A workgroup of 8 waves computes 16 columns (weight rows) for up to 16 MB rows
// of A at a time.  The waves divide K: wave w takes the blocks w, w + 8, ... of
// every weight row, straight into registers in the MFMA's layout, two ahead, and
// the 8 partial sums are joined in the LDS, in a fixed order.  So every weight
// is read once (again for each further 16 MB rows) and no barrier stands in the
// loop.  The weights' bytes bound it: 1 x 7168 x 2048 4.3 us, 16 rows 5.8, 16 x 4096
// x 7168 8.7 us; 8 experts of 4096 x 7168 with a row each 38 us, 6.2 TB/s.
constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;

template <bool AE5, int CT, int MB>
__device__ __forceinline__ void few_rows(const Fp8Args &p, float *red, int64_t row0, int rows, int64_t c0, const uint8_t *b,
                                         const float *sb)
{
    const int lane = threadIdx.x & 63, w = ffn::wave_id(), r = lane & 15, g = lane >> 4;
    const int64_t k = p.k;
    const int blocks = (int)((k + 127) / 128);
    // a column or row past the last one repeats it: it is not stored
    const uint8_t *const wrow = b + min(c0 + r, p.n - 1) * k + 16 * g;
    const uint8_t *xrow[MB];
    const float *srow[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int64_t at = row0 + min(16 * i + r, rows - 1);
        xrow[i] = p.a + at * k + 16 * g;
        srow[i] = p.a_scale + at;
    }
    struct Piece {
        i32x4 w[2], x[MB][2];
        float sb, sa[MB];
    };
    f32x4 acc[MB] = {};
    auto load = [&](Piece &q, int kb) {
        const int64_t o = 128ll * kb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = o + 64 * h + 16 * g < k;        // chunks past K are zeros on both sides
            q.w[h] = i32x4{0, 0, 0, 0};
            if (in) q.w[h] = *(const i32x4 *)(wrow + o + 64 * h);
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                q.x[i][h] = i32x4{0, 0, 0, 0};
                if (in) q.x[i][h] = *(const i32x4 *)(xrow[i] + o + 64 * h);
            }
        }
        q.sb = sb[kb];
#pragma unroll
        for (int i = 0; i < MB; ++i) q.sa[i] = srow[i][kb * p.m];
    };
    auto mma = [&](const Piece &q) {
        const i32x8 x = __builtin_shufflevector(q.w[0], q.w[1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const f32x4 t = mfma128<AE5>(x, __builtin_shufflevector(q.x[i][0], q.x[i][1], 0, 1, 2, 3, 4, 5, 6, 7));
            const float f = q.sa[i] * q.sb;
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][v] = fmaf(f, t[v], acc[i][v]);
        }
    };
    if (w < blocks) {
        Piece q[2];
        load(q[0], w);
        int kb = w;
        for (; kb + 2 * kFewWaves < blocks; kb += 2 * kFewWaves) {
            load(q[1], kb + kFewWaves);
            mma(q[0]);
            load(q[0], kb + 2 * kFewWaves);
            mma(q[1]);
        }
        if (kb + kFewWaves < blocks) {
            load(q[1], kb + kFewWaves);
            mma(q[0]);
            mma(q[1]);
        } else {
            mma(q[0]);
        }
    }
    // partial w of (row, column) at red[(w * 16 MB + row) * 16 + column]
#pragma unroll
    for (int i = 0; i < MB; ++i) *(f32x4 *)(red + (w * 16 * MB + 16 * i + r) * 16 + 4 * g) = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < 256 * MB; o += kFewThreads) {
        const int row = o / 16, col = o % 16;
        float s = red[o];
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v) s += red[v * 256 * MB + o];
        if (row < rows && c0 + col < p.n) ffn::store_one<CT>(p.c, (row0 + row) * p.n + c0 + col, s);
    }
}

// GROUP_ROWS: 256 rows of one expert for each blockIdx.y.
template <bool AE5, int CT, int MB>
__global__ __launch_bounds__(kFewThreads) void k_fp8_few(Fp8Args p)
{
    __shared__ __attribute__((aligned(16))) float red[kFewWaves * 16 * MB * 16];
    const int64_t c0 = 16ll * blockIdx.x, row0 = 256ll * blockIdx.y;
    const int64_t nb = (p.n + 127) / 128, kb = (p.k + 127) / 128;
    const uint8_t *b = p.b;
    const float *sb = p.b_scale + c0 / 128 * kb;
    int rows = (int)min((int64_t)256, p.m - row0);
    if (p.group == GROUP_ROWS) {
        const int e = uniform(expert_of(p.padded_offsets, p.num_experts, row0));
        if (e >= p.num_experts) return;
        const int64_t begin = e ? uniform(p.padded_offsets[e - 1]) : 0;
        rows = (int)min((int64_t)rows, begin + uniform(p.expert_rows[e]) - row0);
        b += e * p.n * p.k;
        sb += e * nb * kb;
    }
    for (int at = 0; at < rows; at += 16 * MB) {
        if (at) __syncthreads();            // the partial sums of the last rows have been read
        few_rows<AE5, CT, MB>(p, red, row0 + at, min(rows - at, 16 * MB), c0, b, sb);
    }
}

template <bool AE5, int CT, int MB>
void go_few(const Fp8Args &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.n + 15) / 16), (unsigned)((a.m + 255) / 256));
    k_fp8_few<AE5, CT, MB><<<grid, kFewThreads, 0, s>>>(a);
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
typedef Fp8Tile<8, 4, 2, 4, 2> Big;         // 256 x 256, 8 waves
typedef Fp8Tile<4, 4, 2, 2, 2> Mid;         // 128 x 128, 4 waves, two workgroups a compute unit
typedef Fp8Tile<2, 2, 2, 4, 3> Small;       // 64 x 128, 8 waves, with K in parts two workgroups a compute unit

template <class T, template <class> class Walk, bool AE5, int CT>
void go_tiles(const Fp8Args &a, int splits, hipStream_t s)
{
    const int64_t mt = (a.m + T::TM - 1) / T::TM, nt = (a.n + T::TN - 1) / T::TN;
    // (Big ones may go out in halves)
    const int64_t tiles = mt * nt * (a.group == GROUP_K ? a.num_experts : 1) * splits * (T::TM / 128 > 1 ? 2 : 1);
    k_fp8<T, Walk, AE5, CT><<<(unsigned)std::min(tiles, (int64_t)256 * T::kGroups), T::kThreads, 0, s>>>(a, (unsigned)mt, (unsigned)nt,
                                                                                                      (unsigned)splits);
}

template <class T, bool AE5, int CT>
void go_whole(const Fp8Args &a, hipStream_t s)
{
    if (a.group == GROUP_K) go_tiles<T, Runs, AE5, CT>(a, 1, s);
    else go_tiles<T, Stride, AE5, CT>(a, 1, s);
}

template <bool AE5, int CT>
void launch(const Fp8Args &a, const Plan &p, hipStream_t s)
{
    if (p.few == 16) return go_few<AE5, CT, 1>(a, s);
    if (p.few == 32) return go_few<AE5, CT, 2>(a, s);
    if (p.few == 64) return go_few<AE5, CT, 4>(a, s);
    if (p.splits > 1) {
        go_tiles<Small::Sums, Parts, AE5, CT>(a, p.splits, s);
        k_join<CT><<<(unsigned)((a.m * a.n / 4 + 255) / 256), 256, 0, s>>>(a, p.splits);
    } else if (p.shape == BIG) {
        go_whole<Big, AE5, CT>(a, s);
    } else if (p.shape == MID) {
        go_whole<Mid, AE5, CT>(a, s);
    } else {
        go_tiles<Small, Stride, AE5, CT>(a, 1, s);
    }
}

}  // namespace

int64_t workspace_gemm_fp8(int64_t m, int64_t n, int64_t k)
{
    if (m == 0 || n == 0) return 0;
    const Plan p = plan_gemm_fp8(m, n, k);
    return !p.few && p.splits > 1 ? 4 * m * n * p.splits : 0;
}

hipError_t launch_fp8(const Fp8Args &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    const Plan p = a.group == GROUP_NONE   ? plan_gemm_fp8(a.m, a.n, a.k)
                   : a.group == GROUP_ROWS ? plan_grouped_fp8(a.m, a.n, a.k, a.num_experts, a.max_rows, a.expert_rows != nullptr)
                                           : plan_wgrad_fp8(a.k, a.m, a.n, a.num_experts);
    if (a.a_dtype == DT_E5M2) {
        if (a.c_dtype == DT_F16) launch<true, DT_F16>(a, p, s);
        else launch<true, DT_BF16>(a, p, s);
    } else {
        if (a.c_dtype == DT_F16) launch<false, DT_F16>(a, p, s);
        else launch<false, DT_BF16>(a, p, s);
    }
    return hipGetLastError();
}

}  // namespace moe
}  // namespace bsg
