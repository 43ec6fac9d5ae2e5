// Eviction by accumulated attention weight: the weights of a decode added to
// each token's score, and the choice of the tokens a sequence keeps.
//
// "LLM推論の「見えないメモリ問題」を解く … vToken", section on token eviction:
// policies such as heavy hitters and sinks with a recent window pick the
// tokens a sequence drops; the token table then lists the survivors.
#include <cooperative_groups.h>

#include <mutex>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_merge.cuh"
#include "pkv_tc_common.cuh"
#include "pkv_units.cuh"

namespace pkv {
namespace {

// ------------------------------------------------------------------- scores
//
// score[s][t] += sum over the query heads h of 2^(x[s][h][t] - M) / L, with
// the logits x the scored decode stored and each row's (M, L), merged from
// its partitions.  One thread owns a token and adds its heads in order, so
// the sum is the same in every launch (no atomics).  The bound is the read
// of the logits, 4 bytes per token and head: a head set's row of a token is
// 4 * score_width(g) consecutive bytes (8 to 32, in 16-byte loads, in 8-byte
// ones where the width is 2 or 6), and a thread requests its next step's rows
// before it merges or uses the ones it has.  The decode's merge needs the same
// inputs and nothing of this, so the grid's first blocks do it: one launch
// instead of two (one sequence of 4,096 tokens: 22.7 -> 20.7 us; long launches
// the same).  Calls in a loop: 64 bf16 sequences of 512..4,096 tokens 31.4 us
// without scores and 34.8 with; 32 E4M3 ones of 256..16,384 67.7 and, with the
// same partitions (512), 79.0, with the scored decode's (800) 67.9; 34 MB of
// logits are read at a third of HBM's rate.  Four head sets per step with two
// blocks per SM are faster where that is one wave (one sequence of 4,096: 13.2
// us, 14.1 with three blocks and two sets), slower in a large launch by 1.3 us
// (32 E4M3 sequences in partitions of 512).

constexpr int kScoreThreads = 256, kScoreWarps = kScoreThreads / 32;
constexpr int kScoreRows = 512;          // (set, head) rows whose (M, 1 / L) are staged at a time

// (M, L) of another part of the same row joins (m, l).
__device__ __forceinline__ void join(float& m, float& l, float M, float L) {
    const float top = fmaxf(m, M);
    const float a = m == top ? 1.f : exp2f(m - top), b = M == top ? 1.f : exp2f(M - top);   // -inf: no -inf - -inf
    l = l * a + L * b;
    m = top;
}

// W: heads per row of logits; ONE: the grid is one wave of two blocks per SM
template <int W, int D, typename QF, bool ONE>
__global__ void __launch_bounds__(kScoreThreads, ONE ? 2 : 3)
    score_kernel(DecodeParams p, float* __restrict__ scores, int MT, int merge_blocks, int chunks, int chunk) {
    constexpr int kSets = ONE ? 4 : 2;   // head sets a thread loads at once
    __shared__ float2 ml[kScoreRows];    // (M, 1 / L); 1 / L = 0 for a row without weight or past the set's heads
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    if ((int)blockIdx.x < merge_blocks) {
        merge_row<D, QF>(p, (long long)blockIdx.x * kScoreWarps + warp, lane);
        return;
    }
    const int job = blockIdx.x - merge_blocks, s = job / chunks, t0 = (job - s * chunks) * chunk;
    int n = p.context_lens[s];
    n = n < 0 ? 0 : min(n, p.max_ctx);   // the decode's clamp
    if (t0 >= n) return;
    const int np = num_partitions(n, p.P, p.Q, p.hold);
    const int nsets = (p.g + kHeadsPerUnit - 1) / kHeadsPerUnit, sets = p.Hkv * nsets;
    constexpr int kTile = kScoreRows / W / kSets * kSets;    // head sets whose rows are staged
    const bool one_tile = sets <= kTile;
    const int end = min(n, t0 + chunk);
    // kSets head sets' logits of token tc + tid, from set b on
    const float* x = p.logits + ((size_t)s * sets * p.max_ctx + tid) * W;
    auto load = [&](float (&v)[kSets][W], int tc, int b) {
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            if (b + k >= sets || tc + tid >= n) continue;
            const float* src = x + ((size_t)(b + k) * p.max_ctx + tc) * W;
#pragma unroll
            for (int j = 0; j < W; j += (W % 4 ? 2 : 4)) {
                if constexpr (W % 4 == 0) {
                    const float4 q = __ldcs(reinterpret_cast<const float4*>(src + j));
                    v[k][j] = q.x; v[k][j + 1] = q.y; v[k][j + 2] = q.z; v[k][j + 3] = q.w;
                } else {
                    const float2 q = __ldcs(reinterpret_cast<const float2*>(src + j));
                    v[k][j] = q.x; v[k][j + 1] = q.y;
                }
            }
        }
    };
    // steps of kSets sets: a step's logits are requested before the rows of the step before are merged or used
    float v[kSets][W], next[kSets][W], sum = 0.f;
    load(v, t0, 0);
    for (int tc = t0, b = 0;;) {
        const int nb = b + kSets < sets ? b + kSets : 0, ntc = nb > 0 ? tc : tc + kScoreThreads;
        if (ntc < end) load(next, ntc, nb);
        if (b % kTile == 0 && (!one_tile || tc == t0)) {
            // eight lanes per row, over its partitions
            const int bn = min(kTile, sets - b);
            __syncthreads();
            for (int i = tid / 8; i - (lane / 8) < bn * W; i += kScoreThreads / 8) {
                const int set = b + i / W, kvh = set / nsets;
                const int hg = (set - kvh * nsets) * kHeadsPerUnit + i % W;
                const bool on = i < bn * W && hg < p.g;
                float m = -CUDART_INF_F, l = 0.f;
                if (on) {
                    const float2* src = reinterpret_cast<const float2*>(p.part_ml) +
                                        ((size_t)s * p.Hq + kvh * p.g + hg) * p.Pmax;
#pragma unroll 4
                    for (int q = lane % 8; q < np; q += 8) {
                        const float2 u = __ldcg(src + q);
                        join(m, l, u.x, u.y);
                    }
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    const float M = __shfl_xor_sync(0xffffffffu, m, o), L = __shfl_xor_sync(0xffffffffu, l, o);
                    join(m, l, M, L);
                }
                if (lane % 8 == 0 && i < bn * W) ml[i] = l != 0.f ? make_float2(m, 1.f / l) : make_float2(0.f, 0.f);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kSets; ++k)
            if (b + k < sets && tc + tid < n)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float2 a = ml[(b % kTile + k) * W + j];
                    // a row without weight adds nothing, whatever its logits are (one with a NaN: NaN)
                    if (a.y != 0.f) sum = fmaf(tc::fast_exp2(v[k][j] - a.x), a.y, sum);
                }
        if (nb == 0) {
            if (tc + tid < n) scores[(size_t)s * MT + tc + tid] += sum;
            sum = 0.f;
        }
        if (ntc >= end) break;
#pragma unroll
        for (int k = 0; k < kSets; ++k)
#pragma unroll
            for (int j = 0; j < W; ++j) v[k][j] = next[k][j];
        tc = ntc;
        b = nb;
    }
}

// ----------------------------------------------------------------- eviction
//
// A sequence of n > budget tokens keeps its first F, its last R and, of the
// rest, the `need` = budget - F - R with the largest scores, ties to the
// lowest index.  Scores are compared as 32-bit keys that order as the floats
// do (NaN lowest, -0 = +0).  The need-th largest key T is found digit by
// digit (histograms of 11, 11 and 10 bits); then a token is kept when its key
// is above T, or equals T and fewer than need - #(above T) equal ones come
// before it.  A kept token's place is the number kept before it, a dropped
// one's the number dropped before it: the order is preserved.
//
// The floor is 8 bytes in and 8 (kept) or 4 (dropped) out per token, 4 us for
// 64 sequences of 32,768; what costs is the chain of dependent steps, 19.3 us
// there (7.3 when nothing is dropped; one sequence of 1,000: 5.8, of 131,072:
// 14.5).  So a sequence is spread over a cluster of CTAs that keep their share
// of the keys in shared memory (one read of the scores), add up their
// histograms through distributed shared memory, and each find T for
// themselves, 2.5 us and a cluster barrier per digit.  The same histograms say
// how many of the CTAs before keep and how many of their keys equal T, so the
// places need no further exchange (one more barrier and its counts: 1.5 us).
// The cluster grows while the grid still fits the GPU in one wave (clusters of
// 8 for the 64 sequences: 28 us, of 2: 30); a share above kEvictHeld tokens is
// read again in every step instead.  Slower were: counting equal bins of a
// warp before the atomics, and a list of the first digit's candidates in every
// CTA so that the other digits need no cluster (20-22 us).

constexpr int kEvictThreads = 512, kEvictWarps = kEvictThreads / 32;
constexpr int kEvictHeld = 16384;                    // keys per CTA, in shared memory
constexpr int kBins = 2048, kMaxRanks = 16, kPortableRanks = 8;
static_assert(kBins == 4 * kEvictThreads && kBins == 64 * 32, "four bins per thread, 64 sums of 32 bins");

// Sum of the values of the lanes above this one.
__device__ __forceinline__ uint32_t lanes_above(uint32_t v, int lane) {
    uint32_t up = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_down_sync(0xffffffffu, up, o);
        if (lane + o < 32) up += u;
    }
    return up - v;
}

// Order of the floats as 32-bit keys: 2 for a NaN, then -inf = 0x007fffff up
// to +inf = 0xff800000.  The values outside are free for what has no score in
// the choice: kFixed is above every T and alone in the last bin, kNone (past
// the sequence's end) below every T.
constexpr uint32_t kFixed = 0xffffffffu, kNone = 0u;
__device__ __forceinline__ uint32_t score_key(float f) {
    if (f != f) return 2u;
    const uint32_t u = f == 0.f ? 0u : __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// HELD: every CTA's share fits its shared memory.
template <bool HELD>
__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const __grid_constant__ EvictParams p) {
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) uint32_t keys[];   // HELD: of this CTA's tokens, in order
    __shared__ __align__(16) uint32_t hist[3][kBins];
    __shared__ __align__(16) uint32_t coarse[3][kBins / 32];
    __shared__ uint2 warp_count[kEvictWarps];
    __shared__ uint32_t pick[4];
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int s = blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    for (int i = tid; i < 3 * kBins / 4; i += kEvictThreads)
        reinterpret_cast<uint4*>(&hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    pdl_wait();
    int n = p.num_tokens[s];
    if (n < 0 || n > p.MT) {
        if (rank == 0 && tid == 0) report(p.err, PKV_DEVERR_CONTEXT_LEN);
        n = n < 0 ? 0 : p.MT;
    }
    const size_t row = (size_t)s * p.MT;
    const bool all = n <= p.budget;
    if (rank == 0 && tid == 0) p.new_num[s] = all ? n : p.budget;
    const int lo = p.first, hi = n - p.recent;       // tokens [lo, hi) compete
    const uint32_t need = all ? 0u : (uint32_t)(p.budget - p.first - p.recent);

    // rank r's tokens are [r * 512 * turns, ...), warp w's 32 * turns of them in order
    const int turns = (n + ranks * kEvictThreads - 1) / (ranks * kEvictThreads);
    const int base = (rank * kEvictWarps + warp) * 32 * turns + lane;
    uint32_t* own = keys + warp * 32 * turns;        // this warp's
    // without a choice to make: every token is fixed (all), or only the first and the recent ones (need 0)
    auto key_of = [&](int t, float sc) {
        if (t >= n) return kNone;
        if (t < lo || t >= hi || all) return kFixed;
        return need > 0 ? score_key(sc) : 1u;
    };
    // fixed tokens among the first m
    auto fixed_before = [&](int m) { return m > n ? (all ? n : lo + n - hi) : all ? m : min(m, lo) + max(0, m - hi); };
    constexpr int kBatch = 8;                       // loads in flight per thread
    if (HELD && need > 0) {                          // the keys, and the first digit's histogram
        for (int i0 = 0; i0 < turns; i0 += kBatch) {
            float v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int t = base + 32 * (i0 + j);
                v[j] = i0 + j < turns && t < n ? __ldg(p.scores + row + t) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i0 + j < turns) {
                    const uint32_t k = key_of(base + 32 * (i0 + j), v[j]);
                    own[32 * (i0 + j) + lane] = k;
                    if (k != kFixed) atomicAdd(&hist[0][k >> 21], 1u);
                }
        }
        __syncwarp();
    }
    // f(key) for the keys of this warp's tokens, in no order
    auto each = [&](auto f) {
        if constexpr (HELD) {
            const uint4* k4 = reinterpret_cast<const uint4*>(own);
#pragma unroll 2
            for (int i = lane; i < 8 * turns; i += 32) {
                const uint4 k = k4[i];
                f(k.x);
                f(k.y);
                f(k.z);
                f(k.w);
            }
        } else {
#pragma unroll 4
            for (int i = 0; i < turns; ++i) {
                const int t = base + 32 * i;
                f(key_of(t, t < n ? __ldg(p.scores + row + t) : 0.f));
            }
        }
    };

    uint32_t T = kFixed - 1u, left = 0;              // keep keys above T, and `left` of key T
    uint32_t a = fixed_before(base - lane), b = 0;   // before this warp: kept for certain, and of key T
    uint32_t ties = 0;                               // of key T in this warp
    if (need > 0) {
        T = 0;
        left = need;
        uint32_t lower = 0;                          // warp 0: competing keys above T in the ranks before this one
        // one copy of the code for the three digits: a launch runs it once, and fetching it is part of the time
#pragma unroll 1
        for (int step = 0; step < 3; ++step) {
            const int shift = step == 0 ? 21 : step == 1 ? 10 : 0;
            const int width = step == 2 ? 10 : 11;
            const uint32_t mask = (1u << width) - 1u;
            uint32_t* bins = hist[step];
            if (step == 0) {                             // (the fixed tokens do not compete)
                if constexpr (!HELD)
                    each([&](uint32_t k) {
                        if (k != kFixed) atomicAdd(&bins[k >> 21], 1u);
                    });
            } else {
                const uint32_t prefix = T >> (shift + width);
                each([&](uint32_t k) {
                    if (k >> (shift + width) == prefix) atomicAdd(&bins[(k >> shift) & mask], 1u);
                });
            }
            __syncthreads();
            // sums of 32 bins: eight threads of four bins each
            const uint4 v = reinterpret_cast<const uint4*>(bins)[tid];
            uint32_t sum = v.x + v.y + v.z + v.w;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane % 8 == 0) coarse[step][tid / 8] = sum;
            if (ranks > 1) cluster.sync();
            else __syncthreads();
            // one warp reads the cluster's 64 sums, then the 32 bins of the sum that T's digit is in
            if (warp == 0) {
                uint32_t h0 = 0, h1 = 0, l0 = 0, l1 = 0; // sums 2 lane, 2 lane + 1; l: of the ranks before
#pragma unroll 8
                for (int r = 0; r < ranks; ++r) {
                    const uint2 u = reinterpret_cast<const uint2*>(cluster.map_shared_rank(&coarse[step][0], r))[lane];
                    h0 += u.x;
                    h1 += u.y;
                    l0 += r < rank ? u.x : 0u;
                    l1 += r < rank ? u.y : 0u;
                }
                uint32_t above = lanes_above(h0 + h1, lane);
                const bool here = above < left && above + h0 + h1 >= left;
                const bool upper = above + h1 >= left;   // of the two sums, the higher one
                if (!upper) above += h1;
                const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
                const int group = __shfl_sync(0xffffffffu, 2 * lane + (upper ? 1 : 0), src);
                const uint32_t want = left - __shfl_sync(0xffffffffu, above, src);
                uint32_t h = 0, l = 0;                   // bin 32 group + lane
#pragma unroll 8
                for (int r = 0; r < ranks; ++r) {
                    const uint32_t u = cluster.map_shared_rank(bins, r)[32 * group + lane];
                    h += u;
                    l += r < rank ? u : 0u;
                }
                above = lanes_above(h, lane);
                const int at = __ffs(__ballot_sync(0xffffffffu, above < want && above + h >= want)) - 1;
                lower += __reduce_add_sync(0xffffffffu, (2 * lane > group ? l0 : 0u) + (2 * lane + 1 > group ? l1 : 0u) +
                                                            (lane > at ? l : 0u));
                if (lane == at) {
                    pick[0] = (uint32_t)(32 * group + lane);
                    pick[1] = want - above;
                    pick[2] = lower;
                    pick[3] = l;                         // the last time: of key T in the ranks before this one
                }
            }
            __syncthreads();
            T |= pick[0] << shift;
            left = pick[1];
        }
        // no CTA leaves while another may still read its histograms
        if (ranks > 1) cluster.barrier_arrive();
        uint32_t ca = 0;
        each([&](uint32_t k) {
            ca += k > T;
            ties += k == T;
        });
        ca = __reduce_add_sync(0xffffffffu, ca);
        ties = __reduce_add_sync(0xffffffffu, ties);
        if (lane == 0) warp_count[warp] = make_uint2(ca, ties);
        __syncthreads();
        a = pick[2] + fixed_before(rank * kEvictThreads * turns);
        b = pick[3];
#pragma unroll
        for (int w = 0; w < kEvictWarps; ++w) {
            const uint2 c = warp_count[w];
            a += w < warp ? c.x : 0u;
            b += w < warp ? c.y : 0u;
        }
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = 0; i0 < turns; i0 += kBatch) {
        int slot[kBatch];
        float sc[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int t = base + 32 * (i0 + j);
            const bool on = i0 + j < turns && t < n;
            slot[j] = on ? __ldg(p.token_slots + row + t) : 0;
            sc[j] = on ? __ldg(p.scores + row + t) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (i0 + j >= turns) break;
            const int t = base + 32 * (i0 + j);
            uint32_t k;
            if (HELD && need > 0) k = own[32 * (i0 + j) + lane];
            else k = key_of(t, sc[j]);
            const bool in = k > T, tie = k == T;
            const uint32_t ba = __ballot_sync(0xffffffffu, in);
            const uint32_t bb = ties ? __ballot_sync(0xffffffffu, tie) : 0u;
            const uint32_t eq = b + __popc(bb & below);  // of key T before this token
            const uint32_t place = a + __popc(ba & below) + min(eq, left);
            if (in || (tie && eq < left)) {
                p.new_slots[row + place] = slot[j];
                p.new_scores[row + place] = sc[j];
            } else if (t < n && p.evicted != nullptr) {
                p.evicted[row + t - place] = slot[j];
            }
            a += __popc(ba);
            b += __popc(bb);
        }
    }
    if (ranks > 1 && need > 0) cluster.barrier_wait();
}

// Whether the device can place a cluster of kMaxRanks CTAs, more than the 8
// that every device can: a context with few SMs per GPC cannot.  Asked once
// per device and context.
class WideClusters {
  public:
    bool fit(const void* kernel, size_t smem) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return false;
        CUcontext ctx = current_context();
        std::lock_guard<std::mutex> lock(mu_);
        const bool cached = dev >= 0 && dev < kDevices && ctx != nullptr;
        if (cached && known_[dev] == ctx) return fits_[dev];
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMaxRanks);
        cfg.blockDim = dim3(kEvictThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxRanks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                  cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
        if (!ok) (void)cudaGetLastError();     // answered: no launch has failed
        if (cached) {
            known_[dev] = ctx;
            fits_[dev] = ok;
        }
        return ok;
    }

  private:
    static constexpr int kDevices = 64;
    CUcontext known_[kDevices] = {};
    bool fits_[kDevices] = {};
    std::mutex mu_;
};

// CTAs per sequence: a cluster of up to 16, doubled while a share is above
// 2,048 tokens and the grid still fits the GPU's two CTAs per SM.  Shares of
// 1,024 / 2,048 / 4,096: one sequence of 16,384 tokens 10.5 / 9.0 / 11.6 us,
// of 4,096 9.7 / 8.4 / 7.7, eight of 8,192 8.7 / 10.1 / 10.1.
int evict_cluster(int S, int MT, int num_sms, int most) {
    int c = 1;
    while (c < most && (MT + c - 1) / c > 2048 && (long long)S * c * 2 <= 2LL * num_sms) c *= 2;
    return c;
}

}  // namespace

template <int D, typename QF>
static cudaError_t launch_score_d(const DecodeParams& p, bool merge, float* scores, int MT, int num_sms, cudaStream_t st) {
    const int merge_blocks = merge ? (int)(((long long)p.S * p.Hq + kScoreWarps - 1) / kScoreWarps) : 0;
    // tokens per thread: as many as leave every SM a few blocks, so that the rows' (M, L) serve more (one / two / four,
    // calls in a replayed graph: 64 bf16 sequences of 512..4,096 40.0 / 38.5 / 40.3 us, 32 E4M3 ones of 256..16,384
    // 72.1 / 70.4 / 69.8, one of 4,096 16.5 / 16.6 / 18.6)
    const long long small = (long long)p.S * ((p.max_ctx + kScoreThreads - 1) / kScoreThreads);
    const int chunk = kScoreThreads * (small <= 4 * num_sms ? 1 : small <= 8 * num_sms ? 2 : 4);
    const int chunks = (p.max_ctx + chunk - 1) / chunk;
    const long long blocks = merge_blocks + (long long)p.S * chunks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(kScoreThreads);
    auto launch = [&](auto kernel) {
        return launch_pdl(kernel, grid, block, 0, st, p, scores, MT, merge_blocks, chunks, chunk);
    };
    const bool one = blocks <= 2 * num_sms;
    switch (score_width(p.g)) {
        case 2: return one ? launch(score_kernel<2, D, QF, true>) : launch(score_kernel<2, D, QF, false>);
        case 4: return one ? launch(score_kernel<4, D, QF, true>) : launch(score_kernel<4, D, QF, false>);
        case 6: return one ? launch(score_kernel<6, D, QF, true>) : launch(score_kernel<6, D, QF, false>);
        default: return one ? launch(score_kernel<8, D, QF, true>) : launch(score_kernel<8, D, QF, false>);
    }
}

cudaError_t launch_score(const DecodeParams& p, pkv_dtype q_dt, bool merge, float* scores, int MT, int num_sms,
                         cudaStream_t st) {
    if (p.S == 0 || p.max_ctx == 0) return cudaSuccess;
    if (p.d == 64)
        return q_dt == PKV_F32 ? launch_score_d<64, F32>(p, merge, scores, MT, num_sms, st)
                               : launch_score_d<64, BF16>(p, merge, scores, MT, num_sms, st);
    return q_dt == PKV_F32 ? launch_score_d<128, F32>(p, merge, scores, MT, num_sms, st)
                           : launch_score_d<128, BF16>(p, merge, scores, MT, num_sms, st);
}

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t st) {
    if (p.S == 0) return cudaSuccess;
    auto share_of = [&](int c) { return ((p.MT + c - 1) / c + kEvictThreads - 1) / kEvictThreads * kEvictThreads; };
    int c = evict_cluster(p.S, p.MT, num_sms, kMaxRanks);
    int share = share_of(c);
    bool held = share <= kEvictHeld;
    auto kern = held ? evict_kernel<true> : evict_kernel<false>;
    static SmemOptIn optin;
    auto opt_in = [&] {
        return held ? optin.ensure(reinterpret_cast<const void*>(kern), kEvictHeld * sizeof(uint32_t)) : cudaSuccess;
    };
    cudaError_t e = opt_in();
    if (e != cudaSuccess) return e;
    if (c > kPortableRanks) {
        static WideClusters wide[2];
        if (!wide[held].fit(reinterpret_cast<const void*>(kern), held ? kEvictHeld * sizeof(uint32_t) : 0)) {
            c = evict_cluster(p.S, p.MT, num_sms, kPortableRanks);
            share = share_of(c);
            held = share <= kEvictHeld;
            kern = held ? evict_kernel<true> : evict_kernel<false>;
            if ((e = opt_in()) != cudaSuccess) return e;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.S * c));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = held ? share * sizeof(uint32_t) : 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace pkv
