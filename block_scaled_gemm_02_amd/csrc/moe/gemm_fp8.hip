// gemm_fp8, grouped_gemm_fp8, grouped_gemm_fp8_wgrad: products of 8-bit
// floats with a scale for each block of 128 of K,
//
//   C[m, n] = sum_kb  a_scale[kb, m] b_scale[n / 128, kb]  sum_{k in kb} a[m, k] b[n, k]
#include "fp8_tile.hpp"

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

// The operands of rows [m0, m0 + tm) and columns [n0, n0 + tn) of C, or of
// expert z's C; false where there is nothing to do.
__device__ __forceinline__ bool part_of(const Fp8Args &p, int64_t m0, int tm, int64_t n0, int tn, int z, Part &t)
{
    const int64_t nb = (p.n + 127) / 128, kb = (p.k + 127) / 128;
    t.rows = (int)min((int64_t)tm, p.m - m0);
    t.cols = (int)min((int64_t)tn, p.n - n0);
    t.held = t.rows;
    t.lda = t.ldb = t.k = p.k;
    t.sa_ld = p.m;
    t.sb_ld = kb;
    t.a = p.a + m0 * p.k;
    t.b = p.b + n0 * p.k;
    t.sa = p.a_scale + m0;
    t.sb = p.b_scale + n0 / 128 * kb;
    t.c = (char *)p.c + 2 * (m0 * p.n + n0);
    if (p.group == GROUP_K) {
        const int64_t first = z ? p.padded_offsets[z - 1] : 0, last = min((int64_t)p.padded_offsets[z], p.k);
        t.a += first;
        t.b += first;
        t.sa += first / 128 * p.m;
        t.sb += first / 128;
        t.k = max((int64_t)0, last - first);
        t.c += 2 * z * p.m * p.n;
    } else if (p.group == GROUP_ROWS) {
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

template <class T, bool AE5, int CT>
__global__ __launch_bounds__(T::kThreads, T::kWaves) void k_fp8(Fp8Args p, unsigned mt, unsigned nt)
{
    __shared__ __attribute__((aligned(16))) uint8_t ring[T::kLds];
    const ffn::TileAt at = ffn::tile_at(blockIdx.x, p.group == GROUP_K ? mt * p.num_experts : mt, nt);
    const int z = p.group == GROUP_K ? at.m / (int)mt : 0, tm = at.m - z * (int)mt;
    Part t;
    if (!part_of(p, (int64_t)T::TM * tm, T::TM, (int64_t)T::TN * at.n, T::TN, z, t)) return;
    T tile(t, ring);
    f32x4 acc[T::WM][T::WN];
    const int blocks = (int)((t.k + 127) / 128);
    tile.template run<AE5>(acc, 0, max(blocks, 1));
    uint8_t *const reg = ring + tile.w * T::kStage;
    const int r0 = 16 * T::WM * tile.wm, c0 = 16 * T::WN * tile.wn;
    static_for<T::WM / 2>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        __builtin_amdgcn_sched_barrier(0);
        ffn::stage_block<CT, T::WN / 2>(reg, tile.lane, [&](auto hh, auto jj) {
            constexpr int r = 2 * i + decltype(hh)::value;
            const f32x4 x = acc[r][decltype(jj)::value];
            // (zeros also where the weight's scale is not finite)
            const bool in = r0 + 16 * r + (tile.lane & 15) < t.held;
            return make_float4(in ? x[0] : 0.0f, in ? x[1] : 0.0f, in ? x[2] : 0.0f, in ? x[3] : 0.0f);
        });
        ffn::flush_block<2, T::WN / 2>(reg, t.c + 2 * ((r0 + 32 * i) * p.n + c0), (uint32_t)(2 * p.n), t.rows - r0 - 32 * i,
                                       2 * (t.cols - c0), tile.lane);
    });
}

typedef Fp8Tile<8, 4, 2, 4, 2> Big;         // 256 x 256, 8 waves
typedef Fp8Tile<4, 4, 2, 2, 2> Mid;         // 128 x 128, 4 waves, two workgroups a compute unit

template <class T, bool AE5, int CT>
void go(const Fp8Args &a, hipStream_t s)
{
    const unsigned mt = (unsigned)((a.m + T::TM - 1) / T::TM), nt = (unsigned)((a.n + T::TN - 1) / T::TN);
    k_fp8<T, AE5, CT><<<mt * nt * (a.group == GROUP_K ? a.num_experts : 1), T::kThreads, 0, s>>>(a, mt, nt);
}

template <bool AE5, int CT>
void launch(const Fp8Args &a, hipStream_t s)
{
    if (((a.m + 255) / 256) * ((a.n + 255) / 256) * (a.group == GROUP_K ? a.num_experts : 1) > 128) go<Big, AE5, CT>(a, s);
    else go<Mid, AE5, CT>(a, s);
}

}  // namespace

int64_t workspace_gemm_fp8(int64_t m, int64_t n, int64_t k) { return 0; }

hipError_t launch_fp8(const Fp8Args &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    if (a.a_dtype == DT_E5M2) {
        if (a.c_dtype == DT_F16) launch<true, DT_F16>(a, s);
        else launch<true, DT_BF16>(a, s);
    } else {
        if (a.c_dtype == DT_F16) launch<false, DT_F16>(a, s);
        else launch<false, DT_BF16>(a, s);
    }
    return hipGetLastError();
}

}  // namespace moe
}  // namespace bsg
