// gemm_fp8, grouped_gemm_fp8, grouped_gemm_fp8_wgrad: products of 8-bit
// floats with a scale for each block of 128 of K,
//
//   C[m, n] = sum_kb  a_scale[kb, m] b_scale[n / 128, kb]  sum_{k in kb} a[m, k] b[n, k]
//
// One 16x16x128 MFMA sums a block's products; its result meets both scales in
// fp32 and is added to the accumulator.
#include "rows.hpp"

namespace bsg {
namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// a b^T over 128 of K, B first: register v of lane (r = l%16, g = l/16) is row r
// of A and row 4g + v of B.  Any order of K serves that both operands share.
template <bool AE5>
__device__ __forceinline__ f32x4 mfma128(const i32x4 (&b)[2], const i32x4 (&a)[2])
{
    const i32x8 x = {b[0][0], b[0][1], b[0][2], b[0][3], b[1][0], b[1][1], b[1][2], b[1][3]};
    const i32x8 y = {a[0][0], a[0][1], a[0][2], a[0][3], a[1][0], a[1][1], a[1][2], a[1][3]};
    const f32x4 zero = {0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, zero, 0, AE5 ? 1 : 0, 0, 0, 0, 0);
}

// One tile's operands.
struct Part {
    const uint8_t *a, *b;
    const float *sa, *sb;       // of K block 0: of row 0; of the first 128 columns
    int64_t lda, ldb, sa_ld, sb_ld;
    int64_t k;
    int rows, held;             // rows of C, rows of A that count
    char *c;                    // row 0, column 0
};

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

// Rows [m0, m0 + tm) of C, or of expert z's C.
__device__ __forceinline__ bool part_of(const Fp8Args &p, int64_t m0, int tm, int z, Part &t)
{
    const int64_t nb = (p.n + 127) / 128, kb = (p.k + 127) / 128;
    t.rows = (int)min((int64_t)tm, p.m - m0);
    t.held = t.rows;
    t.lda = t.ldb = p.k;
    t.k = p.k;
    t.sa_ld = p.m;
    t.sb_ld = kb;
    if (p.group == GROUP_K) {
        const int64_t first = z ? p.padded_offsets[z - 1] : 0, last = min((int64_t)p.padded_offsets[z], p.k);
        t.a = p.a + m0 * p.k + first;
        t.b = p.b + first;
        t.sa = p.a_scale + first / 128 * p.m + m0;
        t.sb = p.b_scale + first / 128;
        t.k = max((int64_t)0, last - first);
        t.c = (char *)p.c + 2 * (z * p.m + m0) * p.n;
        return true;
    }
    t.a = p.a + m0 * p.k;
    t.sa = p.a_scale + m0;
    t.b = p.b;
    t.sb = p.b_scale;
    t.c = (char *)p.c + 2 * m0 * p.n;
    if (p.group == GROUP_ROWS) {
        const int e = __builtin_amdgcn_readfirstlane(expert_of(p.padded_offsets, p.num_experts, m0));
        if (e >= p.num_experts) return false;       // rows behind the last expert
        t.b += e * p.n * p.k;
        t.sb += e * nb * kb;
        if (p.expert_rows) {
            const int64_t begin = e ? p.padded_offsets[e - 1] : 0;
            t.held = (int)max((int64_t)0, min((int64_t)t.rows, begin + p.expert_rows[e] - m0));
        }
    }
    return true;
}

template <bool AE5, int CT>
__global__ __launch_bounds__(256) void k_simple(Fp8Args p)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t m0 = 64 * (int64_t)blockIdx.x, n0 = 64 * (int64_t)blockIdx.y;
    Part t;
    if (!part_of(p, m0, 64, blockIdx.z, t)) return;
    const int row = 16 * w + r;
    f32x4 acc[4] = {};
    for (int64_t k = 0; k < t.k; k += 128) {
        auto load = [&](i32x4 (&f)[2], const uint8_t *x, int64_t ld, int64_t i, bool in) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = k + 64 * h + 16 * g;
                f[h] = i32x4{0, 0, 0, 0};
                if (in && at < t.k) f[h] = *(const i32x4 *)(x + i * ld + at);
            }
        };
        i32x4 a[2];
        load(a, t.a, t.lda, row, row < t.held);
        const float sa = row < t.held ? t.sa[k / 128 * t.sa_ld + row] : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            i32x4 b[2];
            load(b, t.b, t.ldb, n0 + 16 * j + r, n0 + 16 * j + r < p.n);
            const f32x4 x = mfma128<AE5>(b, a);
            const float f = sa * t.sb[n0 / 128 * t.sb_ld + k / 128];
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[j][v] = fmaf(f, x[v], acc[j][v]);
        }
    }
    if (row >= t.rows) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + 16 * j + 4 * g;
        if (n < p.n)
            *(uint2 *)(t.c + 2 * (row * p.n + n)) = pack_quad<CT>(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    }
}

}  // namespace

int64_t workspace_gemm_fp8(int64_t m, int64_t n, int64_t k) { return 0; }

hipError_t launch_fp8(const Fp8Args &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    const dim3 grid((unsigned)((a.m + 63) / 64), (unsigned)((a.n + 63) / 64), a.group == GROUP_K ? (unsigned)a.num_experts : 1u);
    if (a.a_dtype == DT_E5M2) {
        if (a.c_dtype == DT_F16) k_simple<true, DT_F16><<<grid, 256, 0, s>>>(a);
        else k_simple<true, DT_BF16><<<grid, 256, 0, s>>>(a);
    } else {
        if (a.c_dtype == DT_F16) k_simple<false, DT_F16><<<grid, 256, 0, s>>>(a);
        else k_simple<false, DT_BF16><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace moe
}  // namespace bsg
