// Host-side launch interface of the feed-forward operators (quant_i8,
// gemm_i8, gemm_glu, gemm_glu_i8, gemm_glu_bwd): the C ABI validates the
// arguments before these are called.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsg {
namespace ffn {

enum Act : int { ACT_SILU = 0, ACT_GELU_TANH = 1, ACT_RELU = 2 };

struct QuantArgs {
    const void *x;
    int8_t *q;
    float *scale;
    int64_t m, k;
    int x_dtype;            // bsg_dtype: F32, F16 or BF16
};

struct I8Args {
    const int8_t *a, *b;
    const float *a_scale, *b_scale;
    const void *bias;       // null: none
    void *c;
    void *workspace;
    int64_t m, n, k;
    int bias_dtype, c_dtype;
};

// gemm_glu (ab_dtype F16 / BF16) and gemm_glu_i8 (in_i8)
struct GluArgs {
    const void *x, *w_gate, *w_up;
    const float *x_scale, *gate_scale, *up_scale;   // in_i8 only
    void *h, *g, *u;                                // g, u: both or neither
    void *workspace;
    int64_t m, n, k;
    int in_i8, dtype;       // dtype of h (and of x and the weights unless in_i8)
    int act;
};

struct GluBwdArgs {
    const void *dh, *x, *w_gate, *w_up, *g, *u;
    void *dx, *dw_gate, *dw_up;                     // dx, or both dw: may be null
    void *workspace;
    int64_t m, n, k;
    int dtype, act;
};

hipError_t launch_quant_i8(const QuantArgs &a, hipStream_t s);
hipError_t launch_gemm_i8(const I8Args &a, hipStream_t s);
hipError_t launch_gemm_glu(const GluArgs &a, hipStream_t s);
hipError_t launch_gemm_glu_bwd(const GluBwdArgs &a, hipStream_t s);

// Scratch bytes of each operator (0: none).
int64_t workspace_gemm_i8(int64_t m, int64_t n, int64_t k);
int64_t workspace_gemm_glu(int64_t m, int64_t n, int64_t k, bool in_i8);
int64_t workspace_gemm_glu_bwd(int64_t m, int64_t n, int64_t k);

}  // namespace ffn
}  // namespace bsg
