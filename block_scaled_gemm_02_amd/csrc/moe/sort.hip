// moe_sort: expert ids -> each expert's range of rows, and which row holds
// which pair (token, choice).
//
//   count[e] = #{p : expert[p] = e}        begin[e] = sum_{f < e} ceil256(count[f])
//   row_of[p] = begin[e] + #{q < p : expert[q] = e}    (p's expert e; -1 if it has none)
//
// The rank is a running count in the order of the pairs, so equal inputs give
// equal maps.  The pairs are cut into contiguous chunks, a workgroup each, and
// a chunk into contiguous runs, a wave each.  A wave counts its run's ids in
// the LDS, learns where each expert's rows of its run begin (the chunks before
// it, the waves before it), and goes through the run again, 64 pairs at a
// time: lanes with the same id find each other with one ballot a bit of the
// id, and a lane's rank among them is a count of the lower ones.
// One workgroup does all of up to kOne pairs in one launch; more take a first
// launch that leaves each chunk's counts in the workspace, 512 pairs a chunk up to
// 131072 pairs, so that a wave has its ids in one load each, and a chunk's
// workgroup sums the counts of the others in parallel slices.
// Bound by latency: 128 pairs 5.1 us, launch included; 32008 pairs over 64
// experts 13.5 us with 2048 pairs a chunk and one thread an expert, 11.4 us so.
#include "rows.hpp"

namespace bsg {
namespace moe {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64, kMaxExperts = 1024;
constexpr int kOne = 4096;          // pairs of one workgroup
constexpr int kChunks = 256;        // most workgroups of one launch
constexpr int kHeld = 8;            // ids of a wave's run that a lane keeps in registers

struct Cut {
    int chunks, size;               // pairs a chunk
};
__host__ __device__ inline Cut cut_of(int64_t pairs)
{
    if (pairs <= kOne) return {1, (int)pairs};
    const int64_t size = ((pairs + kChunks - 1) / kChunks + kThreads - 1) / kThreads * kThreads;
    return {(int)((pairs + size - 1) / size), (int)size};
}

// An id, or -1 for one that names no expert.
__device__ __forceinline__ int id_at(const SortArgs &p, int i)
{
    const int e = p.expert[i];
    return (unsigned)e < (unsigned)p.num_experts ? e : -1;
}

__global__ __launch_bounds__(kThreads) void k_count(SortArgs p, Cut cut)
{
    __shared__ int32_t count[kMaxExperts];
    for (int e = threadIdx.x; e < p.num_experts; e += kThreads) count[e] = 0;
    __syncthreads();
    const int lo = blockIdx.x * cut.size, hi = min(p.pairs, lo + cut.size);
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
        const int e = id_at(p, i);
        if (e >= 0) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.num_experts; e += kThreads) p.workspace[(int64_t)blockIdx.x * p.num_experts + e] = count[e];
}

__global__ __launch_bounds__(kThreads) void k_place(SortArgs p, Cut cut)
{
    // of[w][e]: wave w's count of expert e, then the next row of its pairs
    __shared__ int32_t of[kWaves][kMaxExperts], total[kMaxExperts], begin[kMaxExperts + 1];
    __shared__ int2 part[kThreads];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6, L = p.num_experts;
    for (int e = t; e < L; e += kThreads)
#pragma unroll
        for (int v = 0; v < kWaves; ++v) of[v][e] = 0;
    __syncthreads();
    const int run = (cut.size + kThreads - 1) / kThreads * 64;
    const int lo = blockIdx.x * cut.size + w * run, hi = min(min(p.pairs, (int)(blockIdx.x + 1) * cut.size), lo + run);
    int held[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int i = lo + 64 * j + lane;
        held[j] = i < hi ? id_at(p, i) : -1;
        if (held[j] >= 0) atomicAdd(&of[w][held[j]], 1);
    }
    for (int i = lo + 64 * kHeld + lane; i < hi; i += 64) {
        const int e = id_at(p, i);
        if (e >= 0) atomicAdd(&of[w][e], 1);
    }
    __syncthreads();
    // rows of the chunks before this one, and of all: `span` experts at a time,
    // the chunks in up to 16 slices
    const int bits = 32 - __clz(L - 1), span = min(1 << bits, kThreads), slices = cut.chunks > 1 ? min(kThreads / span, 16) : 1;
    for (int e0 = 0; e0 < L; e0 += span) {
        const int e = e0 + (t & (span - 1));
        int2 sum = {0, 0};          // before, all
        if (e < L && cut.chunks > 1 && t < span * slices) {
            const int32_t *c = p.workspace + e;
#pragma unroll 8
            for (int i = t / span; i < cut.chunks; i += slices) {
                const int n = c[(int64_t)i * L];
                sum.x += i < (int)blockIdx.x ? n : 0;
                sum.y += n;
            }
        }
        if (slices > 1) {
            part[t] = sum;
            __syncthreads();
        }
        if (t < span && e < L) {
            for (int i = 1; i < slices; ++i) {
                const int2 o = part[i * span + t];
                sum.x += o.x;
                sum.y += o.y;
            }
            int at = sum.x;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                const int n = of[v][e];
                of[v][e] = at;
                at += n;
            }
            total[e] = cut.chunks > 1 ? sum.y : at;
        }
        if (slices > 1 || e0 + span >= L) __syncthreads();
    }
    // where each expert begins: a lane of the first wave sums `each` experts
    if (w == 0) {
        const int each = (L + 63) / 64, e0 = min(lane * each, L), e1 = min(e0 + each, L);
        int s = 0;
        for (int e = e0; e < e1; ++e) s += (total[e] + 255) & ~255;
        int sum = s;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            sum += lane >= d ? o : 0;
        }
        int at = sum - s;
        for (int e = e0; e < e1; ++e) {
            begin[e] = at;
            at += (total[e] + 255) & ~255;
        }
        if (lane == 63) begin[L] = sum;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = t; e < L; e += kThreads) {
            p.padded_offsets[e] = begin[e + 1];
            p.expert_rows[e] = total[e];
        }
    volatile int32_t *const mine = of[w];
    auto place = [&](int q, int e) {
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        int row = -1;
        if (e >= 0) {
            const int rank = __popcll(same & ((1ull << lane) - 1)), at = mine[e];
            row = begin[e] + at + rank;
            __builtin_amdgcn_wave_barrier();
            if (rank == 0) mine[e] = at + __popcll(same);
            if (p.pair_of) p.pair_of[row] = q;
        }
        __builtin_amdgcn_wave_barrier();
        if (q < hi) p.row_of[q] = row;
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
        if (lo + 64 * j < hi) place(lo + 64 * j + lane, held[j]);
    for (int i = lo + 64 * kHeld; i < hi; i += 64) place(i + lane, i + lane < hi ? id_at(p, i + lane) : -1);
    // rows without a pair: each expert's last ones, and those past them all
    if (!p.pair_of) return;
    for (int e = blockIdx.x * kWaves + w; e < L; e += gridDim.x * kWaves)
        for (int r = begin[e] + total[e] + lane; r < begin[e + 1]; r += 64) p.pair_of[r] = -1;
    for (int64_t r = begin[L] + (int64_t)blockIdx.x * kThreads + t; r < p.m; r += (int64_t)gridDim.x * kThreads) p.pair_of[r] = -1;
}

}  // namespace

int64_t workspace_moe_sort(int64_t pairs, int64_t num_experts)
{
    const Cut c = cut_of(pairs);
    return c.chunks > 1 ? 4 * (int64_t)c.chunks * num_experts : 0;
}

hipError_t launch_moe_sort(const SortArgs &a, hipStream_t s)
{
    const Cut cut = cut_of(a.pairs);
    if (cut.chunks > 1) k_count<<<(unsigned)cut.chunks, kThreads, 0, s>>>(a, cut);
    k_place<<<(unsigned)cut.chunks, kThreads, 0, s>>>(a, cut);
    return hipGetLastError();
}

}  // namespace moe
}  // namespace bsg
