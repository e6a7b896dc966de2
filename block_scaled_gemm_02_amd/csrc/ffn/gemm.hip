// Matrix products of the feed-forward operators, in their simplest form:
// one 64 x 64 tile a workgroup, operands staged in LDS through registers.
#include "act.hpp"

namespace bsg {
namespace ffn {
namespace {

enum In : int { IN_BF16 = 0, IN_F16 = 1, IN_I8 = 2 };

// One operand: `rows` rows along M or N, contraction index K.  k-major:
// element (r, kk) at base + r*ld + kk; else at base + kk*ld + r (ld in bytes,
// rows of whole 16-byte pieces either way).
struct Operand {
    const uint8_t *base;
    int64_t ld, rows;
};

constexpr int kBK = 64, kRow = kBK + 16;      // bytes of K per step; LDS row

template <int IN, bool KM>
__device__ __forceinline__ void stage(uint8_t *lds, const Operand &o, int64_t r0, int64_t kb, int64_t kbytes)
{
    const int t = threadIdx.x;
    if constexpr (KM) {
        const int64_t r = r0 + t / 4, b = kb + 16 * (t % 4);
        uint4 v{0, 0, 0, 0};
        if (r < o.rows && b < kbytes) v = *reinterpret_cast<const uint4 *>(o.base + r * o.ld + b);
        *reinterpret_cast<uint4 *>(lds + (t / 4) * kRow + 16 * (t % 4)) = v;
    } else {
        const int64_t kk = kb / 2 + t / 8, r = r0 + 8 * (t % 8);
        uint4 v{0, 0, 0, 0};
        if (r < o.rows && 2 * kk < kbytes) v = *reinterpret_cast<const uint4 *>(o.base + kk * o.ld + 2 * r);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint16_t *>(lds + (8 * (t % 8) + e) * kRow + 2 * (t / 8)) = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
    }
}

template <int IN>
__device__ __forceinline__ f32x16 mma(const uint8_t *a, const uint8_t *b, f32x16 acc)
{
    const i32x4 av = *reinterpret_cast<const i32x4 *>(a), bv = *reinterpret_cast<const i32x4 *>(b);
    if constexpr (IN == IN_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, bv), __builtin_bit_cast(bf16x8, av), acc, 0, 0, 0);
    else if constexpr (IN == IN_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, bv), __builtin_bit_cast(f16x8, av), acc, 0, 0, 0);
    else
        return __builtin_bit_cast(f32x16, __builtin_amdgcn_mfma_i32_32x32x32_i8(bv, av, __builtin_bit_cast(i32x16, acc), 0, 0, 0));
}

// NB products of one A panel: acc[j] += A B_j over kbytes bytes of K.
template <int IN, bool AK, bool BK, int NB>
__device__ __forceinline__ void product(f32x16 (&acc)[NB], uint8_t *lds, const Operand &A, const Operand (&B)[NB],
                                        int64_t m0, int64_t n0, int64_t kbytes)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const uint8_t *ar = lds + (32 * (w >> 1) + (lane & 31)) * kRow + 16 * (lane >> 5);
    const uint8_t *br = lds + (64 + 32 * (w & 1) + (lane & 31)) * kRow + 16 * (lane >> 5);
    for (int64_t kb = 0; kb < kbytes; kb += kBK) {
        __syncthreads();
        stage<IN, AK>(lds, A, m0, kb, kbytes);
        for (int j = 0; j < NB; ++j) stage<IN, BK>(lds + (64 + 64 * j) * kRow, B[j], n0, kb, kbytes);
        __syncthreads();
        for (int s = 0; s < 2; ++s)
            for (int j = 0; j < NB; ++j) acc[j] = mma<IN>(ar + 32 * s, br + 64 * j * kRow + 32 * s, acc[j]);
    }
}

__device__ __forceinline__ void store1(void *p, int64_t i, int dt, float v)
{
    if (dt == DT_F32) ((float *)p)[i] = v;
    else if (dt == DT_F16) ((_Float16 *)p)[i] = (_Float16)v;
    else ((__bf16 *)p)[i] = (__bf16)v;
}
__device__ __forceinline__ float load1(const void *p, int64_t i, int dt)
{
    return dt == DT_F32 ? ((const float *)p)[i] : dt == DT_F16 ? (float)((const _Float16 *)p)[i] : (float)((const __bf16 *)p)[i];
}

// f(row, column, register) over this lane's 16 outputs that exist
template <class F>
__device__ __forceinline__ void outputs(int64_t m0, int64_t n0, int64_t m, int64_t n, F &&f)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t row = m0 + 32 * (w >> 1) + (lane & 31);
    if (row >= m) return;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int64_t col = n0 + 32 * (w & 1) + 8 * (v / 4) + 4 * (lane >> 5) + v % 4;
        if (col < n) f(row, col, v);
    }
}

__global__ __launch_bounds__(256) void k_gemm_i8(I8Args p)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[128 * kRow];
    const int64_t m0 = 64ll * blockIdx.y, n0 = 64ll * blockIdx.x;
    f32x16 acc[1] = {};
    const Operand A{(const uint8_t *)p.a, p.k, p.m}, B[1] = {{(const uint8_t *)p.b, p.k, p.n}};
    product<IN_I8, true, true, 1>(acc, lds, A, B, m0, n0, p.k);
    outputs(m0, n0, p.m, p.n, [&](int64_t r, int64_t c, int v) {
        float y = (float)__float_as_int(acc[0][v]) * p.a_scale[r] * p.b_scale[c];
        if (p.bias) y += load1(p.bias, c, p.bias_dtype);
        store1(p.c, r * p.n + c, p.c_dtype, y);
    });
}

template <int IN, int ACT>
__global__ __launch_bounds__(256) void k_glu(GluArgs p)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[192 * kRow];
    const int64_t m0 = 64ll * blockIdx.y, n0 = 64ll * blockIdx.x, ld = p.k * (IN == IN_I8 ? 1 : 2);
    f32x16 acc[2] = {};
    const Operand A{(const uint8_t *)p.x, ld, p.m};
    const Operand B[2] = {{(const uint8_t *)p.w_gate, ld, p.n}, {(const uint8_t *)p.w_up, ld, p.n}};
    product<IN, true, true, 2>(acc, lds, A, B, m0, n0, ld);
    outputs(m0, n0, p.m, p.n, [&](int64_t r, int64_t c, int v) {
        float g = acc[0][v], u = acc[1][v];
        if constexpr (IN == IN_I8) {
            g = (float)__float_as_int(g) * p.x_scale[r] * p.gate_scale[c];
            u = (float)__float_as_int(u) * p.x_scale[r] * p.up_scale[c];
        }
        const int64_t i = r * p.n + c;
        store1(p.h, i, p.dtype, act_value<ACT>(g) * u);
        if (p.g) {
            store1(p.g, i, p.dtype, g);
            store1(p.u, i, p.dtype, u);
        }
    });
}

// dG = dH * U * act'(G), dU = dH * act(G): rounded to 16 bits for the matrix
// cores, as G and U themselves are.
template <int ACT>
__global__ __launch_bounds__(256) void k_dact(const void *dh, const void *g, const void *u, void *dg, void *du,
                                              int64_t count, int dt)
{
    const int64_t i = 256ll * blockIdx.x + threadIdx.x;
    if (i >= count) return;
    const float d = load1(dh, i, dt);
    const ActGrad a = act_grad<ACT>(load1(g, i, dt));
    store1(dg, i, dt, d * load1(u, i, dt) * a.d);
    store1(du, i, dt, d * a.v);
}

// dX = dG Wg + dU Wu
template <int IN>
__global__ __launch_bounds__(256) void k_dx(GluBwdArgs p, const uint8_t *dg, const uint8_t *du)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[128 * kRow];
    const int64_t m0 = 64ll * blockIdx.y, n0 = 64ll * blockIdx.x;
    f32x16 acc[1] = {};
    const Operand G[1] = {{(const uint8_t *)p.w_gate, 2 * p.k, p.k}}, U[1] = {{(const uint8_t *)p.w_up, 2 * p.k, p.k}};
    product<IN, true, false, 1>(acc, lds, Operand{dg, 2 * p.n, p.m}, G, m0, n0, 2 * p.n);
    product<IN, true, false, 1>(acc, lds, Operand{du, 2 * p.n, p.m}, U, m0, n0, 2 * p.n);
    outputs(m0, n0, p.m, p.k, [&](int64_t r, int64_t c, int v) { store1(p.dx, r * p.k + c, p.dtype, acc[0][v]); });
}

// dWg = dG^T X (z = 0), dWu = dU^T X (z = 1)
template <int IN>
__global__ __launch_bounds__(256) void k_dw(GluBwdArgs p, const uint8_t *dg, const uint8_t *du)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[128 * kRow];
    const int64_t m0 = 64ll * blockIdx.y, n0 = 64ll * blockIdx.x;
    f32x16 acc[1] = {};
    const Operand X[1] = {{(const uint8_t *)p.x, 2 * p.k, p.k}};
    product<IN, false, false, 1>(acc, lds, Operand{blockIdx.z ? du : dg, 2 * p.n, p.n}, X, m0, n0, 2 * p.m);
    void *out = blockIdx.z ? p.dw_up : p.dw_gate;
    outputs(m0, n0, p.n, p.k, [&](int64_t r, int64_t c, int v) { store1(out, r * p.k + c, p.dtype, acc[0][v]); });
}

dim3 tiles(int64_t m, int64_t n, int z = 1) { return dim3((unsigned)((n + 63) / 64), (unsigned)((m + 63) / 64), z); }
int64_t up256(int64_t b) { return (b + 255) / 256 * 256; }

}  // namespace

int64_t workspace_gemm_i8(int64_t, int64_t, int64_t) { return 0; }
int64_t workspace_gemm_glu(int64_t, int64_t, int64_t, bool) { return 0; }
int64_t workspace_gemm_glu_bwd(int64_t m, int64_t n, int64_t) { return 2 * up256(2 * m * n); }

hipError_t launch_gemm_i8(const I8Args &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    k_gemm_i8<<<tiles(a.m, a.n), 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_gemm_glu(const GluArgs &a, hipStream_t s)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    with_act(a.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        if (a.in_i8) k_glu<IN_I8, A><<<tiles(a.m, a.n), 256, 0, s>>>(a);
        else if (a.dtype == DT_F16) k_glu<IN_F16, A><<<tiles(a.m, a.n), 256, 0, s>>>(a);
        else k_glu<IN_BF16, A><<<tiles(a.m, a.n), 256, 0, s>>>(a);
    });
    return hipGetLastError();
}

hipError_t launch_gemm_glu_bwd(const GluBwdArgs &a, hipStream_t s)
{
    uint8_t *dg = (uint8_t *)a.workspace, *du = dg + up256(2 * a.m * a.n);
    const int64_t count = a.m * a.n;
    if (count) {
        with_act(a.act, [&](auto act) {
            k_dact<decltype(act)::value><<<(unsigned)((count + 255) / 256), 256, 0, s>>>(a.dh, a.g, a.u, dg, du, count, a.dtype);
        });
    }
    if (a.dx && a.m && a.k) {
        if (a.dtype == DT_F16) k_dx<IN_F16><<<tiles(a.m, a.k), 256, 0, s>>>(a, dg, du);
        else k_dx<IN_BF16><<<tiles(a.m, a.k), 256, 0, s>>>(a, dg, du);
    }
    if (a.dw_gate && a.n && a.k) {
        if (a.dtype == DT_F16) k_dw<IN_F16><<<tiles(a.n, a.k, 2), 256, 0, s>>>(a, dg, du);
        else k_dw<IN_BF16><<<tiles(a.n, a.k, 2), 256, 0, s>>>(a, dg, du);
    }
    return hipGetLastError();
}

}  // namespace ffn
}  // namespace bsg
