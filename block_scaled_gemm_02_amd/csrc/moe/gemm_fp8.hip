// gemm_fp8, grouped_gemm_fp8, grouped_gemm_fp8_wgrad: products of 8-bit
// floats with a scale for each block of 128 of K,
//
//   C[m, n] = sum_kb  a_scale[kb, m] b_scale[n / 128, kb]  sum_{k in kb} a[m, k] b[n, k]
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

// Workgroup b takes the tiles b, b + gridDim.x, ... in the order of tile_at;
// the loads of a tile's first blocks go out in the last blocks of the one
// before it, so that only the way out of a tile keeps the matrix cores waiting.
// With K in parts (gemm_fp8) a tile is a part of one, whose sums go to the
// workspace.
template <class T, bool AE5, int CT>
__global__ __launch_bounds__(T::kThreads, T::kWaves) void k_fp8(Fp8Args p, unsigned mt, unsigned nt, int splits)
{
    constexpr bool SPLIT = T::SUMS;
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    // rows behind the last expert are no tiles
    if (p.group == GROUP_ROWS)
        mt = (unsigned)((min((int64_t)max(p.padded_offsets[p.num_experts - 1], 0), p.m) + T::TM - 1) / T::TM);
    const unsigned rows = p.group == GROUP_K ? mt * p.num_experts : mt, total = rows * nt * (SPLIT ? splits : 1);
    auto part = [&](unsigned i) {
        const auto [at, split] = ffn::tile_of_block<SPLIT>(i, rows, nt, splits);
        const int z = p.group == GROUP_K ? at.m / (int)mt : 0;
        Part t = part_of(p, (int64_t)T::TM * (at.m - z * (int)mt), T::TM, (int64_t)T::TN * at.n, T::TN, z);
        if constexpr (SPLIT) {
            const ffn::Split s = ffn::split_of(split, splits, (int)((p.k + 127) / 128));
            const int64_t first = 128ll * s.first;
            // (the bytes of the rows shrink by what their beginning moves)
            t.src.ra = make_rsrc_words(p.a + (int64_t)T::TM * at.m * p.k + first, ffn::clamp_bytes(t.to.rows * p.k - first));
            t.src.rb = make_rsrc_words(p.b + (int64_t)T::TN * at.n * p.k + first, ffn::clamp_bytes(t.to.cols * p.k - first));
            t.src.sa += s.first * p.m;
            t.src.klimit = (uint32_t)min(p.k - first, 128ll * s.count);
            t.to.sb += s.first;
            t.to.c = (char *)((float *)p.workspace + (s.index * p.m + (int64_t)T::TM * at.m) * p.n + (int64_t)T::TN * at.n);
        }
        return t;
    };
    // the next tile with rows from i on, or one past them all
    Part cur;
    auto seek = [&](unsigned i, Part &t) {
        for (; i < total; i += gridDim.x) {
            t = part(i);
            if (t.to.rows > 0) break;
        }
        return i;
    };
    unsigned b = seek(blockIdx.x, cur);
    if (b >= total) return;
    T tile(ring, p.k, p.m);
    typename T::Front front;
    tile.start(cur.src, front);
    for (;;) {
        Part then = cur;
        b = seek(b + gridDim.x, then);
        if (b >= total) then.src.klimit = 0;            // nothing after the last tile
        f32x4 acc[T::WM][T::WN];
        const int blocks = (int)((cur.src.klimit + 127) / 128);
        tile.template run<AE5>(acc, front, cur.src, then.src, T::count_of(blocks),
                               cur.to.sb + 16 * T::WN * tile.wn / 128 * ((p.k + 127) / 128), blocks);
        if (b >= total) s_wait_vm<0>();         // no load is under way to the LDS when the workgroup ends
        if constexpr (SPLIT) tile.put_sums(cur.to, p.n, acc);
        else tile.template store<CT>(cur.to, p.n, acc);
        if (b >= total) break;
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
// loop.  The weights' bytes bound it.
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

template <class T, bool AE5, int CT>
void go_tiles(const Fp8Args &a, int splits, hipStream_t s)
{
    const unsigned mt = (unsigned)((a.m + T::TM - 1) / T::TM), nt = (unsigned)((a.n + T::TN - 1) / T::TN);
    const unsigned tiles = mt * nt * (a.group == GROUP_K ? a.num_experts : 1) * splits;
    k_fp8<T, AE5, CT><<<min(tiles, 256u * T::kGroups), T::kThreads, 0, s>>>(a, mt, nt, splits);
}

template <bool AE5, int CT>
void launch(const Fp8Args &a, const Plan &p, hipStream_t s)
{
    if (p.few == 16) return go_few<AE5, CT, 1>(a, s);
    if (p.few == 32) return go_few<AE5, CT, 2>(a, s);
    if (p.few == 64) return go_few<AE5, CT, 4>(a, s);
    if (p.splits > 1) {
        go_tiles<Small::Sums, AE5, CT>(a, p.splits, s);
        k_join<CT><<<(unsigned)((a.m * a.n / 4 + 255) / 256), 256, 0, s>>>(a, p.splits);
    } else if (p.shape == BIG) {
        go_tiles<Big, AE5, CT>(a, 1, s);
    } else if (p.shape == MID) {
        go_tiles<Mid, AE5, CT>(a, 1, s);
    } else {
        go_tiles<Small, AE5, CT>(a, 1, s);
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
