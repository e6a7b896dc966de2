// How a product is cut into workgroups: host code, shared by the launches and
// the workspace sizes.
#pragma once
#include <stdint.h>

#include <algorithm>

namespace bsg {
namespace ffn {

struct Plan {
    int shape;      // 0: Big (256 x 256), 1: Mid (128 x 128), 2: Small (64 x 128), 3: Shared (128 x 128)
    int splits;     // parts of K (Mid only; 1: whole)
    int mt, nt;     // tiles
    double us;      // the estimate
    unsigned grid() const { return (unsigned)mt * (unsigned)nt * (unsigned)splits; }
};

// The cheapest plan of a rows x cols product over kbytes of K by an estimate
// in microseconds, from times measured on the card (256 compute units):
//   * a pair of 128 bytes of K takes a Big tile 0.93 us while at most 128 tiles
//     are at work (2048 cycles of MFMA) and 1.41 us at 256 (the clock falls
//     under the power limit); a Mid tile 0.36 and 0.47 us, a Shared one 0.38
//     and 0.48 us, a Small one 0.27 and 0.32 us, whatever its MFMAs: the loads
//     bound those;
//   * launch, first loads and epilogue: 9.5 (Big), 5.0 (Mid), 4.2 (Small) and 4.5
//     us (Shared), and 4, 4, 0.75 and 0.75 us for each further round of 256
//     tiles: two Small or Shared ones overlap on a CU, and Shared is meant for
//     products that have them;
//   * the operands come from memory at 4.9 TB/s (and 3.5 us of launch);
//   * splitting K (few tiles, long K) costs 1.5 us (a second kernel, less the
//     epilogue) and the partial sums' way to memory and back at 2.2 TB/s of them.
// Measured, with the operands in the memory-side cache (us, Big / Mid / Small /
// Shared / Mid with K in parts): 67 x 4096, K
// 7168 int8: 62.1 / 23.6 / 18.4 / - / 13.3 (4 parts); 512 x 4096, K 4096 int8:
// 39.4 / 16.5 / 13.7 / - / 17.9 (2); 1600 x 2048, K 7168 int8: - / 29.8 / 35.7
// / 31.9; gated fp16 509 x 2048, K 7168: 114 / 44.9 / 38.9 / - / 43.5 (2); gated
// bf16 2000 x 2048, K 4096: 71.1 / 63.6 / 78.1 / 57.5; 2048 x 8192, K 4096 int8:
// 54.9 / 73.8 / 85.9 / 63.9; 6000 x 704, K 512 int8: 12.4 / 10.8 / 9.0 / 7.6.
struct ShapeCost {
    int tm, tn;
    double fixed, round, pair, pair_all;
};
static constexpr ShapeCost kShapeCost[4] = {
    {256, 256, 9.5, 4.0, 0.93, 1.41}, {128, 128, 5.0, 4.0, 0.36, 0.47},
    {64, 128, 4.2, 0.75, 0.27, 0.32}, {128, 128, 4.5, 0.75, 0.38, 0.48}};

inline int64_t pairs_in(int64_t kbytes) { return kbytes > 128 ? (kbytes + 127) / 128 : 1; }

inline Plan plan_with(int shape, int splits, int64_t rows, int64_t cols, int64_t kbytes)
{
    const ShapeCost &c = kShapeCost[shape];
    const int64_t mt = (rows + c.tm - 1) / c.tm, nt = (cols + c.tn - 1) / c.tn;
    const int64_t tiles = mt * nt * splits, full = tiles / 256, rest = tiles % 256;
    const double part = rest > 128 ? c.pair + (c.pair_all - c.pair) * (double)(rest - 128) / 128 : c.pair;
    double t = c.fixed + (double)(full + (rest > 0) - 1) * c.round +
               (double)((pairs_in(kbytes) + splits - 1) / splits) * ((double)full * c.pair_all + (rest ? part : 0));
    t = std::max(t, 3.5 + (double)(rows + cols) * (double)kbytes / 4.9e6);
    if (splits > 1) t += 1.5 + (double)rows * (double)cols * splits * 4 / 2.2e6;
    return {shape, splits, (int)mt, (int)nt, t};
}

inline Plan plan_of(int64_t rows, int64_t cols, int64_t kbytes)
{
    Plan best = plan_with(0, 1, rows, cols, kbytes);
    auto offer = [&](const Plan &p) {
        if (p.us < best.us) best = p;
    };
    const int64_t mid = ((rows + 127) / 128) * ((cols + 127) / 128), pairs = pairs_in(kbytes);
    for (int s = 1; s < (mid > 256 ? 4 : 3); ++s) offer(plan_with(s, 1, rows, cols, kbytes));
    // a split keeps at least four pairs, and splits never make more workgroups than two rounds
    for (int n = 2; n <= 8 && pairs >= 4 * n && mid * n <= 512; ++n) offer(plan_with(1, n, rows, cols, kbytes));
    return best;
}

// Two products that do not depend on each other, x and w: with `together`
// set both have one shape and no splits and go out as one launch, whose
// workgroups fill the compute units that the last round of one of them alone
// would leave idle.  Measured for the gradients of a gated block (us, two
// launches / one): 1003 x 1408 x 2048 39.1 / 30.6, 256 x 512 x 1024 16.6 / 11.8,
// 8192 x 1408 x 2048 204 / 177; 700 x 4096 x 1024, whose dX has few tiles and
// long K, 44.1 (dX in parts) / 59.6.
struct PlanPair {
    Plan x, w;
    bool together;
};
inline PlanPair plan_pair(int64_t xr, int64_t xc, int64_t xk, int64_t wr, int64_t wc, int64_t wk)
{
    PlanPair best{plan_of(xr, xc, xk), plan_of(wr, wc, wk), false};
    double least = best.x.us + best.w.us;
    for (int s = 0; s < 4; ++s) {
        const ShapeCost &c = kShapeCost[s];
        const Plan x = plan_with(s, 1, xr, xc, xk), w = plan_with(s, 1, wr, wc, wk);
        const double xt = (double)x.mt * x.nt, wt = (double)w.mt * w.nt, xp = (double)pairs_in(xk), wp = (double)pairs_in(wk);
        // the longest tile among all the others (a Small or Shared one comes to
        // share its compute unit with a shorter one), or the compute units kept busy to the end
        const double share = std::min(1.0, std::max(0.0, (xt + wt - 256) / 256));
        if (s == 3 && share == 0) break;
        const double one = c.fixed + (s < 2 ? std::max(xp, wp) * (c.pair + c.pair_all) / 2
                                            : std::max(xp, wp) * c.pair + (c.round + std::min(xp, wp) * c.pair_all) * share);
        const double all = (xt * xp + wt * wp) / 256 * c.pair_all + c.fixed + c.round * ((xt + wt) / 256);
        const double t = std::max(one, all);
        if (t < least) {
            best = {x, w, true};
            least = t;
        }
    }
    return best;
}

// The same estimate for the kernel of a few tokens (up to 64), cols weight
// rows in all: the weights at 5.2 TB/s, and the tokens' rows, which every
// workgroup of 16 weight rows reads from the L2 at 45 bytes a nanosecond and
// compute unit (the first six hide behind the weights); the form for 33 to 64
// tokens, with less of the weights in flight, takes 1.3 us more.  Measured, few
// / tiles (us, the weights in the memory-side cache; from HBM the form that is
// taken needs 0.5 to 5 us more): int8 4096 x 7168, 16 tokens 8.6 / 11.2, 24 11.0 / 11.3, 40 15.3
// / 11.8; int8 7168 x 2048, 24 tokens 7.2 / 8.0, 40 9.7 / 8.1; gated bf16 2048 x
// 7168, 16 tokens 15.4 / 17.4, 24 18.7 / 17.5; gated bf16 8192 x 4096, 8 tokens
// 28.7 / 33.5, 16 35.6 / 35.3; gated bf16 512 x 512, 64 tokens 4.6 / 5.1.
inline double few_us(int64_t tokens, int64_t cols, int64_t kbytes)
{
    const double rounds = (double)((cols + 4095) / 4096);
    return (tokens > 32 ? 3.8 : 2.5) + (double)cols * (double)kbytes / 5.2e6 +
           rounds * (double)std::max<int64_t>(0, tokens - 6) * (double)kbytes / 45000.0;
}

// How a product goes out: in the few-token kernel's form for up to 16, 32 or
// 64 tokens, or (few = 0) in tiles.
struct Form {
    int few;
    Plan tiles;
};
inline Form form_of(int64_t tokens, int64_t cols, int64_t kbytes)
{
    const Plan p = plan_of(tokens, cols, kbytes);
    if (tokens > 64 || few_us(tokens, cols, kbytes) > p.us) return {0, p};
    return {tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64, p};
}

// The operators' products: their launches, workspace sizes and plan strings
// all come from these.
inline Form form_gemm_i8(int64_t m, int64_t n, int64_t k) { return form_of(m, n, k); }
inline Form form_gemm_glu(int64_t m, int64_t n, int64_t k, bool in_i8) { return form_of(m, 2 * n, in_i8 ? k : 2 * k); }
// x: dX, whose K is two ranges of n, each padded to whole pairs; w: both weight gradients
inline PlanPair pair_glu_bwd(int64_t m, int64_t n, int64_t k)
{
    return plan_pair(m, k, 2 * ((2 * n + 127) / 128 * 128), 2 * n, k, 2 * m);
}

}  // namespace ffn
}  // namespace bsg
