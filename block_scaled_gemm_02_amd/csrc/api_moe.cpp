// C ABI of the expert operators: argument validation and dispatch, by the
// rules of api.cpp.
#include "api.hpp"
#include "moe/moe.hpp"
#include "moe/plan.hpp"

using namespace bsg::api;

namespace {

constexpr int64_t kMaxTokens = 1ll << 22, kMaxTopK = 64, kMaxExperts = 1024, kMaxRows = 1ll << 30, kMaxHidden = 1ll << 20;

int check_experts(int64_t num_experts)
{
    if (num_experts < 1 || num_experts > kMaxExperts)
        return fail(BSG_ERR_SHAPE, "num_experts=%lld must be in [1, 1024]", (long long)num_experts);
    return BSG_OK;
}

int check_pairs(int64_t tokens, int64_t top_k)
{
    if (tokens < 0 || top_k < 1)
        return fail(BSG_ERR_SHAPE, "tokens=%lld must not be negative, top_k=%lld at least 1", (long long)tokens, (long long)top_k);
    if (tokens > kMaxTokens || top_k > kMaxTopK)
        return fail(BSG_ERR_UNSUPPORTED, "tokens=%lld, top_k=%lld: past 2^22 tokens or 64 choices", (long long)tokens, (long long)top_k);
    return BSG_OK;
}

int check_rows(int64_t m)
{
    if (m < 0 || m % 256) return fail(BSG_ERR_SHAPE, "m=%lld must be a non-negative multiple of 256", (long long)m);
    if (m > kMaxRows) return fail(BSG_ERR_UNSUPPORTED, "m=%lld: past 2^30 rows", (long long)m);
    return BSG_OK;
}

int check_hidden(int64_t hidden, int64_t unit)
{
    if (hidden < 1) return fail(BSG_ERR_SHAPE, "hidden=%lld must be at least 1", (long long)hidden);
    if (hidden > kMaxHidden) return fail(BSG_ERR_UNSUPPORTED, "hidden=%lld: past 2^20 channels", (long long)hidden);
    if (hidden % unit)
        return fail(BSG_ERR_ALIGN, "hidden=%lld must be a multiple of %lld (rows of 16-byte pieces)", (long long)hidden, (long long)unit);
    return BSG_OK;
}

int check_float(int dt, const char *name)
{
    return is_float_out(dt) ? BSG_OK : fail(BSG_ERR_DTYPE, "%s %d is not fp32, fp16 or bf16", name, dt);
}

bool is_fp8(int dt) { return dt == BSG_E4M3 || dt == BSG_E5M2; }

int check_fp8_product(int64_t m, int64_t n, int64_t k, int a_dtype, int c_dtype)
{
    if (int r = check_ffn_sizes(m, n, k)) return r;
    if (!is_fp8(a_dtype)) return fail(BSG_ERR_DTYPE, "a_dtype %d is not E4M3 or E5M2", a_dtype);
    if (c_dtype == BSG_F32)
        return fail(BSG_ERR_UNSUPPORTED, "fp32 C is not built: the 8-bit matrix instructions add less exactly (fp16 and bf16 are)");
    if (!is_16bit(c_dtype)) return fail(BSG_ERR_DTYPE, "c_dtype %d is not fp16 or bf16", c_dtype);
    return BSG_OK;
}

int check_fp8_pointers(const void *a, const void *b, const void *a_scale, const void *b_scale, const void *c, bool sums)
{
    if (!c || (sums && (!a || !b || !a_scale || !b_scale)))
        return fail(BSG_ERR_NULLPTR, "a, b, a_scale, b_scale and c are required");
    if (!aligned16(a) || !aligned16(b) || !aligned16(c)) return fail(BSG_ERR_ALIGN, "a, b and c must be 16-byte aligned");
    if (!aligned4(a_scale) || !aligned4(b_scale)) return fail(BSG_ERR_ALIGN, "scales must be 4-byte aligned");
    return BSG_OK;
}

}  // namespace

extern "C" {

int64_t bsg_moe_rows(int64_t tokens, int64_t top_k, int64_t num_experts)
{
    if (check_pairs(tokens, top_k) || check_experts(num_experts)) return -1;
    const int64_t pairs = tokens * top_k, some = pairs < num_experts ? pairs : num_experts;
    return (pairs + 255 * some) / 256 * 256;
}

int bsg_validate_moe_sort(const int32_t *expert, int32_t *padded_offsets, int32_t *expert_rows, int32_t *row_of,
                          int32_t *pair_of, void *workspace, int64_t workspace_bytes, int64_t tokens, int64_t top_k,
                          int64_t num_experts, int64_t m)
{
    if (int r = check_pairs(tokens, top_k)) return r;
    if (int r = check_experts(num_experts)) return r;
    if (int r = check_rows(m)) return r;
    const int64_t need = bsg_moe_rows(tokens, top_k, num_experts);
    if (m < need) return fail(BSG_ERR_SHAPE, "m=%lld rows; these sizes need up to %lld", (long long)m, (long long)need);
    if (!padded_offsets || !expert_rows || (tokens && (!expert || !row_of)))
        return fail(BSG_ERR_NULLPTR, "expert, padded_offsets, expert_rows and row_of are required");
    if (!aligned4(expert) || !aligned4(padded_offsets) || !aligned4(expert_rows) || !aligned4(row_of) || !aligned4(pair_of))
        return fail(BSG_ERR_ALIGN, "every tensor must be 4-byte aligned");
    return check_workspace(workspace, workspace_bytes, BSG_OP_MOE_SORT, tokens, top_k, num_experts);
}

int moe_sort(const int32_t *expert, int32_t *padded_offsets, int32_t *expert_rows, int32_t *row_of, int32_t *pair_of,
             void *workspace, int64_t workspace_bytes, int64_t tokens, int64_t top_k, int64_t num_experts, int64_t m,
             void *stream)
{
    int st = bsg_validate_moe_sort(expert, padded_offsets, expert_rows, row_of, pair_of, workspace, workspace_bytes, tokens,
                                   top_k, num_experts, m);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::SortArgs args{expert, padded_offsets, expert_rows, row_of, pair_of, static_cast<int32_t *>(workspace),
                                  (int32_t)(tokens * top_k), (int32_t)num_experts, (int32_t)m};
    return launch_status(bsg::moe::launch_moe_sort(args, static_cast<hipStream_t>(stream)), "moe_sort");
}

int bsg_validate_moe_gather(const void *x, const int32_t *row_of, const int32_t *padded_offsets, const int32_t *expert_rows,
                            const float *weight, void *y, float *scale, float *prob, int64_t tokens, int64_t hidden,
                            int64_t top_k, int64_t num_experts, int64_t m, int zero_pad, int x_dtype, int y_dtype)
{
    if (int r = check_pairs(tokens, top_k)) return r;
    if (int r = check_experts(num_experts)) return r;
    if (int r = check_rows(m)) return r;
    if (int r = check_float(x_dtype, "x_dtype")) return r;
    if (y_dtype != x_dtype && y_dtype != BSG_E4M3)
        return fail(BSG_ERR_DTYPE, "y_dtype %d is neither x's nor E4M3", y_dtype);
    if (int r = check_hidden(hidden, y_dtype == BSG_E4M3 ? 16 : 16 / elem_bytes(x_dtype))) return r;
    // (a tensor without elements has no address)
    if ((prob && tokens && !weight) || (weight && m && !prob))
        return fail(BSG_ERR_NULLPTR, "weight and prob are given together or not at all");
    if (y_dtype == BSG_E4M3 ? m && !scale : scale != nullptr) return fail(BSG_ERR_NULLPTR, "scale goes with E4M3 codes");
    if (m && (!y || (tokens && (!x || !row_of)) || (zero_pad && (!padded_offsets || !expert_rows))))
        return fail(BSG_ERR_NULLPTR, "x, row_of and y are required, padded_offsets and expert_rows with zero_pad");
    if (!aligned16(x) || !aligned16(y)) return fail(BSG_ERR_ALIGN, "x and y must be 16-byte aligned");
    if (!aligned4(row_of) || !aligned4(padded_offsets) || !aligned4(expert_rows) || !aligned4(weight) || !aligned4(scale) ||
        !aligned4(prob))
        return fail(BSG_ERR_ALIGN, "maps, weights and scales must be 4-byte aligned");
    return BSG_OK;
}

int moe_gather(const void *x, const int32_t *row_of, const int32_t *padded_offsets, const int32_t *expert_rows,
               const float *weight, void *y, float *scale, float *prob, int64_t tokens, int64_t hidden, int64_t top_k,
               int64_t num_experts, int64_t m, int zero_pad, int x_dtype, int y_dtype, void *stream)
{
    int st = bsg_validate_moe_gather(x, row_of, padded_offsets, expert_rows, weight, y, scale, prob, tokens, hidden, top_k,
                                     num_experts, m, zero_pad, x_dtype, y_dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    if (m == 0) return BSG_OK;
    const bsg::moe::GatherArgs args{x, row_of, padded_offsets, expert_rows, weight, y, scale, prob, tokens, hidden, m,
                                    (int)top_k, (int)num_experts, zero_pad, x_dtype, y_dtype};
    return launch_status(bsg::moe::launch_moe_gather(args, static_cast<hipStream_t>(stream)), "moe_gather");
}

int bsg_validate_moe_gather_bwd(const void *dy, const float *dprob, const int32_t *row_of, void *dx, float *dweight,
                                int64_t tokens, int64_t hidden, int64_t top_k, int64_t m, int dtype)
{
    if (int r = check_pairs(tokens, top_k)) return r;
    if (int r = check_rows(m)) return r;
    if (int r = check_float(dtype, "dtype")) return r;
    if (int r = check_hidden(hidden, 16 / elem_bytes(dtype))) return r;
    if ((dprob && tokens && !dweight) || (dweight && m && !dprob))
        return fail(BSG_ERR_NULLPTR, "dprob and dweight are given together or not at all");
    if (tokens && !dx && !dweight) return fail(BSG_ERR_NULLPTR, "dx or dweight is required");
    if (tokens && (!row_of || (dx && m && !dy))) return fail(BSG_ERR_NULLPTR, "row_of is required, and dy for dx");
    if (!aligned16(dy) || !aligned16(dx)) return fail(BSG_ERR_ALIGN, "dy and dx must be 16-byte aligned");
    if (!aligned4(row_of) || !aligned4(dprob) || !aligned4(dweight))
        return fail(BSG_ERR_ALIGN, "row_of, dprob and dweight must be 4-byte aligned");
    return BSG_OK;
}

int moe_gather_bwd(const void *dy, const float *dprob, const int32_t *row_of, void *dx, float *dweight, int64_t tokens,
                   int64_t hidden, int64_t top_k, int64_t m, int dtype, void *stream)
{
    int st = bsg_validate_moe_gather_bwd(dy, dprob, row_of, dx, dweight, tokens, hidden, top_k, m, dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::CombineArgs args{dy, row_of, nullptr, dprob, dx, dweight, tokens, hidden, m, (int)top_k, dtype};
    return launch_status(bsg::moe::launch_moe_combine(args, static_cast<hipStream_t>(stream)), "moe_gather_bwd");
}

int bsg_validate_moe_combine(const void *y, const int32_t *row_of, const float *weight, void *out, int64_t tokens,
                             int64_t hidden, int64_t top_k, int64_t m, int dtype)
{
    if (int r = check_pairs(tokens, top_k)) return r;
    if (int r = check_rows(m)) return r;
    if (int r = check_float(dtype, "dtype")) return r;
    if (int r = check_hidden(hidden, 16 / elem_bytes(dtype))) return r;
    if (tokens && (!row_of || !out || (m && !y))) return fail(BSG_ERR_NULLPTR, "y, row_of and out are required");
    if (!aligned16(y) || !aligned16(out)) return fail(BSG_ERR_ALIGN, "y and out must be 16-byte aligned");
    if (!aligned4(row_of) || !aligned4(weight)) return fail(BSG_ERR_ALIGN, "row_of and weight must be 4-byte aligned");
    return BSG_OK;
}

int moe_combine(const void *y, const int32_t *row_of, const float *weight, void *out, int64_t tokens, int64_t hidden,
                int64_t top_k, int64_t m, int dtype, void *stream)
{
    int st = bsg_validate_moe_combine(y, row_of, weight, out, tokens, hidden, top_k, m, dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::CombineArgs args{y, row_of, weight, nullptr, out, nullptr, tokens, hidden, m, (int)top_k, dtype};
    return launch_status(bsg::moe::launch_moe_combine(args, static_cast<hipStream_t>(stream)), "moe_combine");
}

int bsg_validate_moe_combine_bwd(const void *dout, const void *y, const int32_t *row_of, const int32_t *padded_offsets,
                                 const int32_t *expert_rows, const float *weight, void *dy, float *dweight, int64_t tokens,
                                 int64_t hidden, int64_t top_k, int64_t num_experts, int64_t m, int zero_pad, int dtype)
{
    if (int r = check_pairs(tokens, top_k)) return r;
    if (int r = check_experts(num_experts)) return r;
    if (int r = check_rows(m)) return r;
    if (int r = check_float(dtype, "dtype")) return r;
    if (int r = check_hidden(hidden, 16 / elem_bytes(dtype))) return r;
    if (tokens && m && !dy && !dweight) return fail(BSG_ERR_NULLPTR, "dy or dweight is required");
    if (tokens && (!dout || !row_of || (dweight && m && !y)))
        return fail(BSG_ERR_NULLPTR, "dout and row_of are required, and y for dweight");
    if (dy && zero_pad && m && (!padded_offsets || !expert_rows))
        return fail(BSG_ERR_NULLPTR, "padded_offsets and expert_rows are required with zero_pad");
    if (!aligned16(dout) || !aligned16(y) || !aligned16(dy)) return fail(BSG_ERR_ALIGN, "dout, y and dy must be 16-byte aligned");
    if (!aligned4(row_of) || !aligned4(padded_offsets) || !aligned4(expert_rows) || !aligned4(weight) || !aligned4(dweight))
        return fail(BSG_ERR_ALIGN, "maps and weights must be 4-byte aligned");
    return BSG_OK;
}

int moe_combine_bwd(const void *dout, const void *y, const int32_t *row_of, const int32_t *padded_offsets,
                    const int32_t *expert_rows, const float *weight, void *dy, float *dweight, int64_t tokens,
                    int64_t hidden, int64_t top_k, int64_t num_experts, int64_t m, int zero_pad, int dtype, void *stream)
{
    int st = bsg_validate_moe_combine_bwd(dout, y, row_of, padded_offsets, expert_rows, weight, dy, dweight, tokens, hidden,
                                          top_k, num_experts, m, zero_pad, dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::CombineBwdArgs args{dout, y, row_of, padded_offsets, expert_rows, weight, dy, dweight, tokens, hidden, m,
                                        (int)top_k, (int)num_experts, zero_pad && m, dtype};
    return launch_status(bsg::moe::launch_moe_combine_bwd(args, static_cast<hipStream_t>(stream)), "moe_combine_bwd");
}

int bsg_validate_quant_fp8(const void *x, uint8_t *q, float *scale, uint8_t *q_t, float *scale_t, int64_t l, int64_t m,
                           int64_t k, int tile, int x_dtype, int q_dtype)
{
    (void)tile;
    if (int r = check_ffn_sizes(m, 0, k)) return r;
    if (l < 0) return fail(BSG_ERR_SHAPE, "negative size");
    if (l > 1024) return fail(BSG_ERR_UNSUPPORTED, "l=%lld: past 1024 matrices", (long long)l);
    if (int r = check_float(x_dtype, "x_dtype")) return r;
    if (!is_fp8(q_dtype)) return fail(BSG_ERR_DTYPE, "q_dtype %d is not E4M3 or E5M2", q_dtype);
    if (k % 16) return fail(BSG_ERR_ALIGN, "K=%lld must be a multiple of 16", (long long)k);
    if (q_t && m % 16) return fail(BSG_ERR_ALIGN, "M=%lld must be a multiple of 16 for q_t", (long long)m);
    if (l == 0 || m == 0 || k == 0) return BSG_OK;
    if (!q != !scale || !q_t != !scale_t) return fail(BSG_ERR_NULLPTR, "codes and their scales are given together or not at all");
    if (!x || (!q && !q_t)) return fail(BSG_ERR_NULLPTR, "x is required, and q or q_t");
    if (!aligned16(x) || !aligned16(q) || !aligned16(q_t)) return fail(BSG_ERR_ALIGN, "x, q and q_t must be 16-byte aligned");
    if (!aligned4(scale) || !aligned4(scale_t)) return fail(BSG_ERR_ALIGN, "scales must be 4-byte aligned");
    return BSG_OK;
}

int quant_fp8(const void *x, uint8_t *q, float *scale, uint8_t *q_t, float *scale_t, int64_t l, int64_t m, int64_t k, int tile,
              int x_dtype, int q_dtype, void *stream)
{
    int st = bsg_validate_quant_fp8(x, q, scale, q_t, scale_t, l, m, k, tile, x_dtype, q_dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::QuantFp8Args args{x, q, q_t, scale, scale_t, l, m, k, tile, x_dtype, q_dtype};
    return launch_status(bsg::moe::launch_quant_fp8(args, static_cast<hipStream_t>(stream)), "quant_fp8");
}

int bsg_validate_gemm_fp8(const uint8_t *a, const uint8_t *b, const float *a_scale, const float *b_scale, void *c,
                          void *workspace, int64_t workspace_bytes, int64_t m, int64_t n, int64_t k, int a_dtype, int c_dtype)
{
    if (int r = check_fp8_product(m, n, k, a_dtype, c_dtype)) return r;
    if (k % 16 || n % 8)
        return fail(BSG_ERR_ALIGN, "K=%lld must be a multiple of 16 and N=%lld of 8", (long long)k, (long long)n);
    if (int r = check_ffn_tiles(m, n)) return r;
    if (m == 0 || n == 0) return BSG_OK;
    if (int r = check_fp8_pointers(a, b, a_scale, b_scale, c, k > 0)) return r;
    return check_workspace(workspace, workspace_bytes, BSG_OP_GEMM_FP8, m, n, k);
}

int gemm_fp8(const uint8_t *a, const uint8_t *b, const float *a_scale, const float *b_scale, void *c, void *workspace,
             int64_t workspace_bytes, int64_t m, int64_t n, int64_t k, int a_dtype, int c_dtype, void *stream)
{
    int st = bsg_validate_gemm_fp8(a, b, a_scale, b_scale, c, workspace, workspace_bytes, m, n, k, a_dtype, c_dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::Fp8Args args{a, b, a_scale, b_scale, nullptr, nullptr, c, workspace, m, n, k, 0, 0,
                                 bsg::moe::GROUP_NONE, a_dtype, c_dtype};
    return launch_status(bsg::moe::launch_fp8(args, static_cast<hipStream_t>(stream)), "gemm_fp8");
}

int bsg_validate_grouped_gemm_fp8(const uint8_t *a, const uint8_t *b, const float *a_scale, const float *b_scale,
                                  const int32_t *padded_offsets, const int32_t *expert_rows, void *c, int64_t m, int64_t n,
                                  int64_t k, int64_t num_experts, int64_t max_rows, int a_dtype, int c_dtype)
{
    if (int r = check_fp8_product(m, n, k, a_dtype, c_dtype)) return r;
    if (int r = check_experts(num_experts)) return r;
    if (int r = check_rows(m)) return r;
    if (max_rows < 0) return fail(BSG_ERR_SHAPE, "max_rows=%lld must not be negative", (long long)max_rows);
    if (k % 16 || n % 8)
        return fail(BSG_ERR_ALIGN, "K=%lld must be a multiple of 16 and N=%lld of 8", (long long)k, (long long)n);
    if (int r = check_ffn_tiles(m, n)) return r;
    if (int r = check_ffn_tiles(num_experts * 64, n)) return r;
    if (m == 0 || n == 0) return BSG_OK;
    if (!padded_offsets) return fail(BSG_ERR_NULLPTR, "padded_offsets is required");
    if (!aligned4(padded_offsets) || !aligned4(expert_rows))
        return fail(BSG_ERR_ALIGN, "padded_offsets and expert_rows must be 4-byte aligned");
    return check_fp8_pointers(a, b, a_scale, b_scale, c, k > 0);
}

int grouped_gemm_fp8(const uint8_t *a, const uint8_t *b, const float *a_scale, const float *b_scale,
                     const int32_t *padded_offsets, const int32_t *expert_rows, void *c, int64_t m, int64_t n, int64_t k,
                     int64_t num_experts, int64_t max_rows, int a_dtype, int c_dtype, void *stream)
{
    int st = bsg_validate_grouped_gemm_fp8(a, b, a_scale, b_scale, padded_offsets, expert_rows, c, m, n, k, num_experts,
                                           max_rows, a_dtype, c_dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::Fp8Args args{a, b, a_scale, b_scale, padded_offsets, expert_rows, c, nullptr, m, n, k, (int)num_experts,
                                 (int)(max_rows < m ? max_rows : m), bsg::moe::GROUP_ROWS, a_dtype, c_dtype};
    return launch_status(bsg::moe::launch_fp8(args, static_cast<hipStream_t>(stream)), "grouped_gemm_fp8");
}

const char *bsg_grouped_plan_string(int wgrad, int64_t m, int64_t n, int64_t k, int64_t num_experts, int64_t max_rows,
                                    int expert_rows)
{
    static thread_local char text[64];
    if (check_ffn_sizes(m, n, k) || check_experts(num_experts) || check_rows(m)) return nullptr;
    if (max_rows < 0) {
        fail(BSG_ERR_SHAPE, "max_rows=%lld must not be negative", (long long)max_rows);
        return nullptr;
    }
    if (!n || (wgrad ? !k : !m)) return "none";
    bsg::moe::text_of(wgrad ? bsg::moe::plan_wgrad_fp8(m, n, k, num_experts)
                            : bsg::moe::plan_grouped_fp8(m, n, k, num_experts, max_rows < m ? max_rows : m, expert_rows != 0),
                      text, sizeof text);
    return text;
}

int bsg_validate_grouped_gemm_fp8_wgrad(const uint8_t *a, const uint8_t *b, const float *a_scale, const float *b_scale,
                                        const int32_t *padded_offsets, void *c, int64_t m, int64_t n, int64_t k,
                                        int64_t num_experts, int a_dtype, int c_dtype)
{
    if (int r = check_fp8_product(m, n, k, a_dtype, c_dtype)) return r;
    if (n > (1ll << 20)) return fail(BSG_ERR_UNSUPPORTED, "N=%lld: past 2^20 channels", (long long)n);
    if (int r = check_experts(num_experts)) return r;
    if (int r = check_rows(m)) return r;
    if (k % 8) return fail(BSG_ERR_ALIGN, "K=%lld must be a multiple of 8", (long long)k);
    const int64_t tiles = ((n + 63) / 64) * ((k + 63) / 64) * num_experts;
    if (tiles >= (1ll << 23)) return fail(BSG_ERR_UNSUPPORTED, "%lld output tiles exceed the launch limit", (long long)tiles);
    if (n == 0 || k == 0) return BSG_OK;
    if (!padded_offsets) return fail(BSG_ERR_NULLPTR, "padded_offsets is required");
    if (!aligned4(padded_offsets)) return fail(BSG_ERR_ALIGN, "padded_offsets must be 4-byte aligned");
    return check_fp8_pointers(a, b, a_scale, b_scale, c, m > 0);
}

int grouped_gemm_fp8_wgrad(const uint8_t *a, const uint8_t *b, const float *a_scale, const float *b_scale,
                           const int32_t *padded_offsets, void *c, int64_t m, int64_t n, int64_t k, int64_t num_experts,
                           int a_dtype, int c_dtype, void *stream)
{
    int st = bsg_validate_grouped_gemm_fp8_wgrad(a, b, a_scale, b_scale, padded_offsets, c, m, n, k, num_experts, a_dtype,
                                                 c_dtype);
    if (st) return st;
    if ((st = check_device())) return st;
    const bsg::moe::Fp8Args args{a, b, a_scale, b_scale, padded_offsets, nullptr, c, nullptr, n, k, m, (int)num_experts, 0,
                                 bsg::moe::GROUP_K, a_dtype, c_dtype};
    return launch_status(bsg::moe::launch_fp8(args, static_cast<hipStream_t>(stream)), "grouped_gemm_fp8_wgrad");
}

}  // extern "C"
