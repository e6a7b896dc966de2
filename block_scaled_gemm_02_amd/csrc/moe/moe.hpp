// Host-side launch interface of the expert operators (moe_sort, moe_gather,
// moe_combine and their gradients, quant_fp8, gemm_fp8 and the grouped forms):
// the C ABI validates the arguments before these are called.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsg {
namespace moe {

struct SortArgs {
    const int32_t *expert;
    int32_t *padded_offsets, *expert_rows, *row_of, *pair_of;   // pair_of may be null
    int32_t *workspace;
    int32_t pairs, num_experts, m;
};

struct GatherArgs {
    const void *x;
    const int32_t *row_of, *padded_offsets, *expert_rows;
    const float *weight;    // with prob
    void *y;
    float *scale, *prob;    // scale: y holds E4M3 codes; prob may be null
    int64_t tokens, hidden, m;
    int top_k, num_experts, zero_pad, x_dtype, y_dtype;
};

// moe_combine (dprob, dweight null) and moe_gather_bwd (weight null)
struct CombineArgs {
    const void *y;
    const int32_t *row_of;
    const float *weight, *dprob;
    void *out;
    float *dweight;
    int64_t tokens, hidden, m;
    int top_k, dtype;
};

struct CombineBwdArgs {
    const void *dout, *y;
    const int32_t *row_of, *padded_offsets, *expert_rows;
    const float *weight;
    void *dy;               // dy or dweight may be null
    float *dweight;
    int64_t tokens, hidden, m;
    int top_k, num_experts, zero_pad, dtype;
};

struct QuantFp8Args {
    const void *x;
    uint8_t *q, *q_t;       // with scale and scale_t; one of the two may be null
    float *scale, *scale_t;
    int64_t l, m, k;
    int tile, x_dtype, q_dtype;
};

// Which rows or K range of A a product takes: all of them, an expert's rows
// (grouped), or an expert's range of K (the weight's gradient).
enum Group : int { GROUP_NONE = 0, GROUP_ROWS = 1, GROUP_K = 2 };

// C (rows, cols) = A (rows, k) B (cols, k)^T.  GROUP_ROWS: B and b_scale one
// an expert; GROUP_K: C one an expert, K over the m sorted rows.
struct Fp8Args {
    const uint8_t *a, *b;
    const float *a_scale, *b_scale;
    const int32_t *padded_offsets, *expert_rows;
    void *c;
    void *workspace;
    int64_t m, n, k;
    int num_experts, max_rows, group, a_dtype, c_dtype;
};

hipError_t launch_moe_sort(const SortArgs &a, hipStream_t s);
hipError_t launch_moe_gather(const GatherArgs &a, hipStream_t s);
hipError_t launch_moe_combine(const CombineArgs &a, hipStream_t s);
hipError_t launch_moe_combine_bwd(const CombineBwdArgs &a, hipStream_t s);
hipError_t launch_quant_fp8(const QuantFp8Args &a, hipStream_t s);
hipError_t launch_fp8(const Fp8Args &a, hipStream_t s);

// Scratch bytes of each operator (0: none).
int64_t workspace_moe_sort(int64_t pairs, int64_t num_experts);
int64_t workspace_gemm_fp8(int64_t m, int64_t n, int64_t k);

}  // namespace moe
}  // namespace bsg
