// Eviction by accumulated attention weight: the weights of a decode added to
// each token's score, and the choice of the tokens a sequence keeps.
//
// "LLM推論の「見えないメモリ問題」を解く … vToken", section on token eviction:
// policies such as heavy hitters and sinks with a recent window pick the
// tokens a sequence drops; the token table then lists the survivors.
#include <math_constants.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_tc_common.cuh"
#include "pkv_units.cuh"

namespace pkv {
namespace {

// ------------------------------------------------------------------- scores
//
// score[s][t] += sum over the query heads h of 2^(x[s][h][t] - M) / L, with
// the logits x the scored decode stored and the (M, L) of row (s, h) merged
// from its partitions.  One thread owns a token and adds its heads in order,
// so the sum is the same in every launch (no atomics).

constexpr int kScoreThreads = 256;
constexpr int kScoreTokens = 1024;       // per CTA
constexpr int kScoreRows = 512;          // (set, head) rows whose (M, 1 / L) are staged at a time

__global__ void __launch_bounds__(kScoreThreads) score_kernel(DecodeParams p, float* __restrict__ scores, int MT) {
    __shared__ float2 ml[kScoreRows];    // (M, 1 / L); (0, 0) for a row without tokens or past the set's heads
    const int s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    int n = p.context_lens[s];
    n = n < 0 ? 0 : min(n, p.max_ctx);   // the decode's clamp
    const int t0 = blockIdx.x * kScoreTokens;
    if (t0 >= n) return;
    const int np = num_partitions(n, p.P, p.Q, p.hold);
    const int W = score_width(p.g), nsets = (p.g + kHeadsPerUnit - 1) / kHeadsPerUnit;
    const int sets = p.Hkv * nsets, tile = kScoreRows / W;
    constexpr int K = kScoreTokens / kScoreThreads;
    float sum[K];
#pragma unroll
    for (int k = 0; k < K; ++k) sum[k] = 0.f;
    for (int b0 = 0; b0 < sets; b0 += tile) {
        const int bn = min(tile, sets - b0);
        __syncthreads();
        for (int i = warp; i < bn * W; i += kScoreThreads / 32) {
            const int set = b0 + i / W, j = i % W;
            const int kvh = set / nsets, hg = (set - kvh * nsets) * kHeadsPerUnit + j;
            float M = -CUDART_INF_F, L = 0.f;
            if (hg < p.g) {
                const float2* src = reinterpret_cast<const float2*>(p.part_ml) + ((size_t)s * p.Hq + kvh * p.g + hg) * p.Pmax;
                for (int q = lane; q < np; q += 32) M = fmaxf(M, src[q].x);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                if (M != -CUDART_INF_F)
                    for (int q = lane; q < np; q += 32) L += src[q].y * exp2f(src[q].x - M);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
            }
            if (lane == 0) ml[i] = L > 0.f ? make_float2(M, 1.f / L) : make_float2(0.f, 0.f);
        }
        __syncthreads();
        for (int b = 0; b < bn; ++b) {
            const float* x = p.logits + ((size_t)s * sets + b0 + b) * p.max_ctx * W;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int t = t0 + tid + k * kScoreThreads;
                if (t >= n) continue;
                for (int j = 0; j < W; j += 2) {
                    const float2 v = *reinterpret_cast<const float2*>(x + (size_t)t * W + j);
                    const float2 a = ml[b * W + j], c = ml[b * W + j + 1];
                    // a row without weight (L = 0) adds nothing, whatever its logits are
                    if (a.y > 0.f) sum[k] = fmaf(tc::fast_exp2(v.x - a.x), a.y, sum[k]);
                    if (c.y > 0.f) sum[k] = fmaf(tc::fast_exp2(v.y - c.x), c.y, sum[k]);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int t = t0 + tid + k * kScoreThreads;
        if (t < n) scores[(size_t)s * MT + t] += sum[k];
    }
}

// ----------------------------------------------------------------- eviction
//
// A sequence of n > budget tokens keeps its first F, its last R and, of the
// rest, the `need` = budget - F - R with the largest scores, ties to the
// lowest index.  Scores are compared as 32-bit keys that order as the floats
// do (NaN lowest, -0 = +0).  The need-th largest key T is found digit by
// digit (four 8-bit histograms); then one pass in token order keeps a token
// when its key is above T, or equals T and fewer than need - #(above T)
// equal ones came before it.  A kept token's place is the number kept before
// it, a dropped one's the number dropped before it: the order is preserved.

constexpr int kEvictThreads = 1024;

__device__ __forceinline__ uint32_t score_key(float f) {
    if (f != f) return 0u;
    const uint32_t u = f == 0.f ? 0u : __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t pick[2];          // digit of T, tokens still to find at or below it
    __shared__ uint32_t warp_sum[32];
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    int n = p.num_tokens[s];
    if (n < 0 || n > p.MT) {
        if (tid == 0) report(p.err, PKV_DEVERR_CONTEXT_LEN);
        n = n < 0 ? 0 : p.MT;
    }
    const size_t row = (size_t)s * p.MT;
    const bool all = n <= p.budget;
    if (tid == 0) p.new_num[s] = all ? n : p.budget;
    const int lo = p.first, hi = n - p.recent;       // tokens [lo, hi) compete
    const uint32_t need = all ? 0u : (uint32_t)(p.budget - p.first - p.recent);
    uint32_t T = 0xffffffffu, left = 0;              // left: tokens of key T to keep
    if (need > 0) {
        T = 0;
        left = need;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
            __syncthreads();
            for (int t = lo + tid; t < hi; t += kEvictThreads) {
                const uint32_t k = score_key(p.scores[row + t]);
                if (shift == 24 || (k >> (shift + 8)) == (T >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                int dg = 255;
                uint32_t want = left;
                while (dg > 0 && hist[dg] < want) want -= hist[dg--];
                pick[0] = (uint32_t)dg;
                pick[1] = want;
            }
            __syncthreads();
            T |= pick[0] << shift;
            left = pick[1];
        }
    }
    uint32_t above = 0, equal = 0;                   // kept above T, and of key T, before this pass
    for (int c0 = 0; c0 < n; c0 += kEvictThreads) {
        const int t = c0 + tid;
        const bool fixed = t < lo || t >= hi || all;
        float sc = 0.f;
        int slot = 0;
        uint32_t v = 0;                              // (equal to T) << 16 | above T or fixed
        if (t < n) {
            sc = p.scores[row + t];
            slot = p.token_slots[row + t];
            const uint32_t k = score_key(sc);
            v = fixed ? 1u : (need == 0 ? 0u : (k > T ? 1u : (k == T ? 0x10000u : 0u)));
        }
        uint32_t inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        uint32_t before = 0, total = 0;
        for (int w = 0; w < kEvictThreads / 32; ++w) {
            const uint32_t x = warp_sum[w];
            before += w < warp ? x : 0u;
            total += x;
        }
        __syncthreads();
        const uint32_t ex = before + inc - v;
        const uint32_t eq0 = equal + (ex >> 16);
        const uint32_t place = above + (ex & 0xffffu) + min(eq0, left);
        if (t < n) {
            const bool keep = (v & 0xffffu) || (v != 0 && eq0 < left);
            if (keep) {
                p.new_slots[row + place] = slot;
                p.new_scores[row + place] = sc;
            } else if (p.evicted != nullptr) {
                p.evicted[row + t - place] = slot;
            }
        }
        above += total & 0xffffu;
        equal += total >> 16;
    }
}

}  // namespace

cudaError_t launch_score(const DecodeParams& p, float* scores, int MT, cudaStream_t st) {
    if (p.S == 0 || p.max_ctx == 0) return cudaSuccess;
    const dim3 grid((unsigned)((p.max_ctx + kScoreTokens - 1) / kScoreTokens), (unsigned)p.S);
    return launch_pdl(score_kernel, grid, dim3(kScoreThreads), 0, st, p, scores, MT);
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t st) {
    if (p.S == 0) return cudaSuccess;
    return launch_pdl(evict_kernel, dim3((unsigned)p.S), dim3(kEvictThreads), 0, st, p);
}

}  // namespace pkv
