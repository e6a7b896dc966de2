// How a product of 8-bit floats goes out: host code, shared by the launches,
// the workspace size and the plan string.
#pragma once
#include <cstdio>

#include "../ffn/plan.hpp"

namespace bsg {
namespace moe {

enum Shape : int { BIG = 0, MID = 1, SMALL = 2 };       // 256 x 256, 128 x 128, 64 x 128

struct Plan {
    int few;        // rows of the few-row kernel (16, 32, 64), or 0: tiles
    int shape;
    int splits;     // parts of K (Small only; 1: whole)
    double us;      // the estimate
};

// Estimates in microseconds, from times measured on the card (256 compute
// units):
//   * a block of 128 of K takes a Big tile 1.15 us where little more than half the
//     compute units are at work (2048 cycles of MFMA) and 1.5 us with all of them
//     (the clock falls under the power limit); at most 128 tiles go out in halves
//     of 0.85 us; Mid tiles, two a unit, 0.70 and 1.05 us; a Small one 0.35 and 0.41
//     us, and in parts, two a unit, 0.60 us: its loads bound it, not its 256 cycles
//     of MFMA;
//   * launch, first loads and the way out take 7.0, 3.0 and 3.8 us, each further
//     round of tiles 5.2, 2.1 and 1.3 us more;
//   * the operands come from memory at 4.9 TB/s (and 3.5 us of launch);
//   * K in parts costs 1.5 us (a second kernel) and the partial sums' way to
//     memory and back at 2.2 TB/s of them.
// Measured (us, Big / Mid / Small / Small in parts, operands in the memory-side
// cache): 64 x 4096, K 7168 - / 33.3 / 23.0 / 13.2 (4); 256 x 4096, K 7168 - /
// 42.4 / 23.5 / 19.9 (2); 1024 x 2048, K 7168 - / 42.4 / 25.4 / 34.5 (2); 512 x
// 4096, K 4096 - / 24.7 / 16.9 / 24.3 (2); 2048 x 4096, K 2048 19.7 / 20.7 / 31.9 /
// -; 4096 x 2048, K 4096 34.1 / 35.5 / 56.6 / -; 2500 x 4096, K 1040 18.6 / 20.1 / -
// / -; 4200 x 4104, K 2064 57.3 / 59.3 / - / -; 5000 x 4096, K 4096 80.8 (94.2 with
// a whole last round) / 89.3 / - / -; 6000 x 704, K 512 10.7 / 7.8 / 11.5 / -;
// 8192^3 410 / 533 / 694 / -.
struct ShapeCost {
    int tm, tn, per_cu;
    double fixed, round, block, block_all;
};
static constexpr ShapeCost kCost[3] = {
    {256, 256, 1, 7.0, 5.2, 1.15, 1.5}, {128, 128, 2, 3.0, 2.1, 0.70, 1.05}, {64, 128, 1, 3.8, 1.3, 0.35, 0.41}};

static constexpr double kHalf = 0.85;       // a half of a Big tile

// groups: products of these sizes (experts), each with its own sum over k.
inline Plan plan_with(int shape, int splits, int64_t rows, int64_t cols, int64_t k, int64_t groups)
{
    const ShapeCost &c = kCost[shape];
    const int per_cu = splits > 1 ? 2 : c.per_cu;
    const double all = splits > 1 ? 0.60 : c.block_all;
    const int64_t tiles = (rows + c.tm - 1) / c.tm * ((cols + c.tn - 1) / c.tn) * groups * splits, wave = 256 * per_cu;
    const int64_t full = tiles / wave, rest = tiles % wave;
    const double blocks = (double)((ffn::pairs_in(k) + splits - 1) / splits);
    const double part = rest > wave / 2    ? c.block + (all - c.block) * (double)(2 * rest - wave) / (double)wave
                        : shape == BIG && groups == 1 ? kHalf
                                                      : c.block;
    double t = c.fixed + (double)(full + (rest > 0) - 1) * c.round + blocks * ((double)full * all + (rest ? part : 0));
    t = std::max(t, 3.5 + (double)groups * (double)(rows + cols) * (double)k / 4.9e6);
    if (splits > 1) t += 1.5 + (double)rows * (double)cols * splits * 4 / 2.2e6;
    return {0, shape, splits, t};
}

// gemm_fp8
inline Plan plan_gemm_fp8(int64_t m, int64_t n, int64_t k)
{
    Plan best = plan_with(BIG, 1, m, n, k, 1);
    auto offer = [&](const Plan &p) {
        if (p.us < best.us) best = p;
    };
    offer(plan_with(MID, 1, m, n, k, 1));
    offer(plan_with(SMALL, 1, m, n, k, 1));
    // a part keeps at least four blocks, and parts never make more than one round
    const int64_t tiles = (m + 63) / 64 * ((n + 127) / 128), blocks = ffn::pairs_in(k);
    for (int s = 2; s <= 8 && blocks >= 4 * s && tiles * s <= 512; ++s) offer(plan_with(SMALL, s, m, n, k, 1));
    // The few-row kernel, as the products of 8-bit integers estimate theirs.
    // Measured, few / tiles: 16 x 4096, K 7168 8.7 / 11.6, 32 rows 12.0 / 12.3,
    // 64 rows 18.8 / 13.1; 16 x 7168, K 2048 5.8 / 8.3; 64 x 512, K 512 3.6 / 5.2.
    if (m <= 64 && ffn::few_us(m, n, k) <= best.us) best = {m <= 16 ? 16 : m <= 32 ? 32 : 64, SMALL, 1, ffn::few_us(m, n, k)};
    return best;
}

// grouped_gemm_fp8.  The host knows the rows that the buffer has and the most
// that one expert may have, not how many there are.  If m is what bsg_moe_rows
// gives, there are at most m + 255 - 255 num_experts pairs, so that many over
// the experts on average.  Tiles of at most 64 rows each read the experts'
// weights at 5.9 (Big) or 4.6 TB/s (Mid), the few-row kernel at 5.5, and its
// workgroups the rows again (us, few / Big / Mid: 64 experts of 4096 x 7168 with
// 4 rows each 339 / 318 / 497, with 16 rows 509 / 325 / 502; 8 experts with 8
// rows 44.6 / 69 / 51, with one row 38 / 69 / 51).
inline Plan plan_grouped_fp8(int64_t m, int64_t n, int64_t k, int64_t num_experts, int64_t max_rows, bool expert_rows)
{
    const Plan big = plan_with(BIG, 1, m, n, k, 1), mid = plan_with(MID, 1, m, n, k, 1);
    Plan best = mid.us < big.us ? mid : big;
    if (expert_rows && max_rows > 0 && max_rows <= 64) {
        const int64_t blocks = m / 256, experts = std::min(num_experts, blocks), pairs = m + 255 - 255 * num_experts;
        const double each = std::max(1.0, (double)pairs / (double)num_experts), bytes = (double)experts * (double)n * (double)k;
        const int64_t tiles = blocks * ((n + 255) / 256);
        const double tb = std::max((double)((tiles + 255) / 256) * (5.2 + 1.15 * (double)ffn::pairs_in(k)) + 1.8, 3.5 + bytes / 5.9e6);
        const double tm = std::max(plan_with(MID, 1, 128 * blocks, n, k, 1).us, 3.5 + bytes / 4.6e6);
        const double tf = 2.5 + bytes / 5.5e6 + (double)experts * (double)n / 4096 * std::max(0.0, each - 6) * (double)k / 45000;
        best = {0, tm < tb ? MID : BIG, 1, std::min(tm, tb)};
        if (tf < best.us) best = {max_rows <= 16 ? 16 : 32, BIG, 1, tf};
    }
    return best;
}

// grouped_gemm_fp8_wgrad: C (n, k) for each expert, its rows m over the experts.
inline Plan plan_wgrad_fp8(int64_t m, int64_t n, int64_t k, int64_t num_experts)
{
    const Plan big = plan_with(BIG, 1, n, k, m / num_experts, num_experts), mid = plan_with(MID, 1, n, k, m / num_experts, num_experts);
    return mid.us < big.us ? mid : big;
}

inline void text_of(const Plan &p, char *text, size_t size)
{
    static const char *const shape[3] = {"Big", "Mid", "Small"};
    if (p.few) snprintf(text, size, "few %d", p.few);
    else if (p.splits > 1) snprintf(text, size, "%s / %d", shape[p.shape], p.splits);
    else snprintf(text, size, "%s", shape[p.shape]);
}

}  // namespace moe
}  // namespace bsg
