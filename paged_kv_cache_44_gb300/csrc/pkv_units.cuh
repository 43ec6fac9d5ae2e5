// Work units of the tensor-core decodes: a partition (or chunk) of one
// sequence's tokens for up to 8 query heads of one K/V head, and the order
// in which a launch hands them out.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_merge.cuh"

namespace pkv {

constexpr int kHeadsPerUnit = 8;

// Tokens of the longest sequence, in window_span's numbering with a window.
inline int max_visible(const DecodeParams& p) {
    return p.window > 0 ? window_bound(p.max_ctx, p.window, p.sinks, p.bs, 1) : p.max_ctx;
}

// Heads per row of the scored decode's logits: a head set's, an even number.
__host__ __device__ __forceinline__ int score_width(int g) { return g >= kHeadsPerUnit ? kHeadsPerUnit : (g + 1) & ~1; }

// Region B ids per (sequence, head set): the full-size chunks of the longest
// remainder (hold * P + P - 1 tokens), then one for the partial chunk.
__host__ __device__ __forceinline__ int chunk_slots(int P, int Q, int hold) {
    const int held = Q < P ? hold : 0;
    return (held * P + P - 1) / Q + 1;
}

struct __align__(16) Unit {
    int s, kvh, h0, nh, part, t0, t1, np;
};

// Unit id -> coordinates.  The ids run over two regions:
//   A: every full partition (P tokens) not held back, partition-major -- the same
//      partition of every sequence is claimed close together in time, so
//      shared prefix blocks are read while still in L2;
//   B: the chunks of each sequence's last, partial partition (and, with
//      p.hold, of the full partitions held back before it): first every
//      full-size chunk (Q tokens), chunk-major, then each sequence's
//      shorter last chunk (and the empty unit of a sequence with no tokens).
// Claimed in id order, the long units go first and the short ones last, so
// the tail of the launch is short.  Returns false for ids that name no
// work (a partition past the sequence's full ones, a chunk past its
// remainder, or a last chunk that does not exist).  With a window (WIN) the
// tokens t0, t1 are those of window_span's numbering.  SUFFIX: numbered from
// p.begin[s]; where that is not 0 there are other partial results beside this
// launch's, and np is never 1.
template <bool WIN, bool SUFFIX = false>
__device__ __forceinline__ bool unit_of(const DecodeParams& p, unsigned long long u, int nsets,
                                        unsigned long long region_a, Unit& x) {
    const unsigned long long per_part = (unsigned long long)p.S * p.Hkv * nsets;
    const bool in_a = u < region_a;
    const unsigned long long v = in_a ? u : u - region_a;
    const int idx = (int)(v / per_part);                  // partition (A) or chunk (B) index
    const unsigned long long rem = v - (unsigned long long)idx * per_part;
    x.s = (int)(rem / (unsigned)(p.Hkv * nsets));
    const int r2 = (int)(rem - (unsigned long long)x.s * (p.Hkv * nsets));
    x.kvh = r2 / nsets;
    const int set = r2 - x.kvh * nsets;
    x.h0 = x.kvh * p.g + set * kHeadsPerUnit;
    x.nh = min(kHeadsPerUnit, p.g - set * kHeadsPerUnit);
    int n = load_behind_wait(p.context_lens + x.s);
    if (n < 0 || n > p.max_ctx) {
        if (!in_a && idx == 0 && r2 == 0) report(p.err, PKV_DEVERR_CONTEXT_LEN);
        n = n < 0 ? 0 : p.max_ctx;
    }
    if constexpr (WIN) n -= window_span(n - p.window, p.sinks, p.bs).gap;
    int begin = 0;
    if constexpr (SUFFIX) {
        begin = load_behind_wait(p.begin + x.s);
        n = max(n - begin, 0);
    }
    x.np = num_partitions(n, p.P, p.Q, p.hold);
    if (SUFFIX && begin > 0) x.np = max(x.np, 2);
    const int full = whole_partitions(n, p.P, p.Q, p.hold);
    const int tail = n - full * p.P;
    const int cfull = chunk_slots(p.P, p.Q, p.hold) - 1;   // full-size chunks of the longest remainder
    if (in_a) {
        if (idx >= full) return false;
        x.part = idx;
    } else if (idx < cfull) {
        if ((idx + 1) * p.Q > tail) return false;          // full-size chunks first
        x.part = full + idx;
    } else {
        if (idx > cfull) return false;
        if (n > 0 && tail % p.Q == 0) return false;        // then the remainder's partial chunk
        x.part = full + tail / p.Q;
    }
    partition_range(n, p.P, p.Q, p.hold, x.part, x.t0, x.t1);
    return true;
}

// A launch of at most one CTA per (sequence, head set) and one warp per
// partition: warp w of CTA b then takes, as its first and only unit, unit
// w * CTAs + b, which is partition w of set b (the ids above), so a set's
// partial results are all its CTA's, and the CTA merges them without a second
// launch.  One 4-bit sequence of 301 tokens: 8.9 us with the merge kernel, 7.9
// without (and 2 us less of the host's time).  `warps` is what a set may take
// on one SM: a bf16, fp32 or 4-bit worker waits mostly for its own copies and
// sums, an E4M3 one is busy converting, and from five on the spread launch
// with its merge kernel is faster (640 tokens in 10 partitions: 9.3 and 12.8 us).
inline bool merges_itself(const DecodeParams& p, unsigned long long per_part, unsigned long long units, int warps,
                          int num_sms) {
    return p.Pmax > 1 && per_part <= (unsigned long long)num_sms && units <= per_part * warps;
}

// The merge of such a CTA's set, by all its warps.
template <int D, typename QF>
__device__ __forceinline__ void merge_set(const DecodeParams& p, int nsets, int warps) {
    __threadfence();
    __syncthreads();
    const int set = blockIdx.x % nsets, kvh = blockIdx.x / nsets % p.Hkv, s = blockIdx.x / (nsets * p.Hkv);
    const int nh = min(kHeadsPerUnit, p.g - set * kHeadsPerUnit);
    for (int h = threadIdx.x / 32; h < nh; h += warps)
        merge_row<D, QF>(p, (long long)s * p.Hq + kvh * p.g + set * kHeadsPerUnit + h, threadIdx.x & 31);
}

}  // namespace pkv
