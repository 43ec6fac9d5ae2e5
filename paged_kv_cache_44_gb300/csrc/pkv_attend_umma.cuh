// Attention of many query rows over the same keys on the fifth-generation
// tensor cores: whole packed prompts with K and V contiguous (pkv_prompt.cu),
// and the shared blocks of a group of decoding sequences, read through a block
// table (kShared; pkv_shared.cu).
//
// "LLM推論の基礎とvLLMの内部", section 6: a step computes prompts next to
// decodes; section 2: GQA lets several query heads share one K/V head.
// Sequence s has queries query_start[s] .. query_start[s + 1] of q and keys
// key_start[s] .. key_start[s + 1] of k and v; its last query sits at its last
// key.  out = softmax(scale q k^T) v over the keys a query sees: all of them,
// those up to its own position, or of these the first `sinks` and the last
// `window`.
//
// Two products of 128 x 128 x d per 128 queries, 128 keys and head, and 16,384
// exponentials between them: bound by the tensor cores, if the softmax of one
// tile hides behind the products of another.  A work unit is two tiles of 128
// queries of one head each (two heads of a K/V head, or two query blocks of
// one) over the same keys, so each K/V stage is read once for both; one
// persistent block per SM.  Roles:
//   warps 0-3   softmax of tile 0, warps 4-7 of tile 1, one thread per row (TMEM
//               lane): P = 2^(x - m) in bf16 goes over the first half of S's
//               columns
//   warp 8      claims units, K tiles by TMA into a ring
//   warps 9, 10 issue a tile's products each (one warp for both, waiting for the two
//               tiles in a fixed order: one prompt of 32,768 tokens 4,893 us, not 4,705;
//               one of 1 token 0.2 us less), and gather its rows where it is packed:
//                 S_t = Q_t . K_j^T       M 128, N 128, K d
//                 O_t (+)= P_t . V_j      M 128, N d, K 128 (P_t in TMEM)
//   warp 11     V tiles, and Q tiles of one head, by TMA; zeroes rows that no query of the sequence sees
//               (other sequences' in its last tile, those before every window: 0 times what they hold may be NaN)
// A row's reference maximum m moves only when a stage's maximum exceeds it by
// more than 8 (log2 units); O is then rescaled in TMEM.  Every weight stays <=
// 2^8 and O / l is the same softmax whatever m was.  P is rounded to bf16 (by
// 2^-8 of a weight at most): the tensor cores take 16-bit operands; sums stay in
// fp32.
//
// Units are numbered longest first: query blocks from the last to the first
// over all sequences, so the end of a launch is made of short ones.  A block
// takes tickets from a counter and walks (block, 32 sequences at a time) to
// the unit of its ticket, so ragged lengths cost no empty tickets.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include <mutex>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_qtile.cuh"
#include "pkv_tc_common.cuh"
#include "pkv_umma.cuh"

namespace pkv {
namespace {

using namespace tc;

constexpr int kTok = kPromptStage;    // key tokens per stage
constexpr int kRows = kPromptStage;   // queries per tile
constexpr int kSoftWarps = 8, kThreads = 384;
constexpr int kKWarp = 8, kMmaWarp = 9 /* and 10: a tile each */, kVWarp = 11;
constexpr int kTurnStages = 16, kTurnTail = 8;
constexpr float kRescaleLog2 = 8.f;
constexpr long long kTurnLimit = 16384;           // cycles: some five stages
constexpr long long kWaitLimit = 4000000000LL;    // ~2 s: a barrier that never completes
constexpr uint32_t kTmemCols = 512;               // O_0, O_1, S_0, S_1; P_t over the first half of S_t
__host__ __device__ constexpr uint32_t tmem_o(int t) { return 128u * t; }
__host__ __device__ constexpr uint32_t tmem_s(int t) { return 256u + 128u * t; }
// Registers: launched with kThreads x kLaunchRegs; the softmax warps raise
// theirs, the others lower theirs, within the launch's total.
constexpr int kLaunchRegs = 168, kSoftRegs = 200, kOtherRegs = 104;
static_assert(32 * kSoftWarps * kSoftRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");

// control block, in front of the tiles (byte offsets)
constexpr uint32_t kKFull = 0;         // [4]
constexpr uint32_t kKEmpty = 32;       // [4]
constexpr uint32_t kVFull = 64;        // [4]
constexpr uint32_t kVEmpty = 96;       // [4]
constexpr uint32_t kSFull = 128;       // [2 tiles]: S_t of the tile's stage done
constexpr uint32_t kPFull = 144;       // [2 tiles]: P_t written (4 warps)
constexpr uint32_t kPVDone = 160;      // [2 tiles]: P_t . V done
constexpr uint32_t kQFull = 176;       // [2 tiles]
constexpr uint32_t kQEmpty = 192;      // [2 tiles]
constexpr uint32_t kUFull = 208;       // [2]: unit records
constexpr uint32_t kUEmpty = 224;      // [2]
constexpr uint32_t kTail = 240;        // the V tile whose rows are to be zeroed has landed
constexpr uint32_t kFin = 248;
constexpr uint32_t kPFull2 = 256;      // [2 tiles]: ... of the second half of the keys
constexpr uint32_t kTmemSlot = 272, kAbort = 276, kTurn = 280 /* [2 tiles] */, kRing = 288 /* [2][4] int4 */;
constexpr uint32_t kMasks = kRing + 128 /* [8 stages][4 words] */, kCtlBytes = kMasks + 128;

// The rows of a tile: 128 queries of one head (kHeads: K and V of a head are
// read for two tiles), or the (query, head) pairs of a K/V head in order, 128 at
// a time (kPacked, kShared: few queries fill a tile between them).
enum Mode { kHeads, kPacked, kShared };

template <int D, int MODE>
struct Cfg {
    static constexpr int kHalves = D / 64;                 // 128-byte halves of a row
    static constexpr int kItemBytes = kTok * 2 * D;        // a K, V or Q tile
    // kHeads: an item of K less, and room for 64 columns of each tile's output, which leaves by TMA
    static constexpr int kKItems = D == 128 ? (MODE == kHeads ? 2 : 3) : 4, kVItems = D == 128 ? 2 : 4;
    static constexpr int kOutBytes = MODE == kHeads ? kRows * 128 : 0;
    static constexpr int kVOff = kKItems * kItemBytes;
    static constexpr int kQOff = (kKItems + kVItems) * kItemBytes;
    static constexpr int kOutOff = kQOff + 2 * kItemBytes, kTileBytes = kOutOff + 2 * kOutBytes;
    // the control block, up to the next 1,024 bytes (the dynamic shared memory starts on such a boundary;
    // the kernel checks it)
    static constexpr int kSmemBytes = ((int)kCtlBytes + 1023) / 1024 * 1024 + kTileBytes;
    static_assert(kSmemBytes <= 232448, "shared memory per block");
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// a box of shared memory into global memory, a bulk group of its own
__device__ __forceinline__ void tensor_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(src)
        : "memory");
}

// true in one thread of the (converged) warp, always the same one
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(is));
    return is != 0;
}

// D[tmem] (+)= A[tmem] . B[smem]
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "r"(tmem_a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u));
}

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A sequence's rows; false when a bound is broken (it is skipped then).
// kShared: a group of sequences, its members q0 .. q0 + ql, whose first kl
// tokens (whole blocks) are read through the table of the first of them.
struct Seq {
    int q0, ql, k0, kl;
};
template <int MODE>
__device__ __forceinline__ bool sequence(const PromptParams& p, int s, Seq& x) {
    if constexpr (MODE == kShared) {
        x.q0 = load_behind_wait(p.query_start + s);
        const long long members = (long long)load_behind_wait(p.query_start + s + 1) - x.q0;
        const int shared = load_behind_wait(p.key_start + s);
        x.ql = (int)members;
        x.k0 = 0;
        x.kl = shared / p.bs * p.bs;
        const bool ok = x.q0 >= 0 && members >= 0 && x.q0 + members <= p.Tq && shared >= 0 && shared <= p.max_k &&
                        (x.kl == 0 || members <= p.max_q);
        if (!ok) x.kl = 0;
        return ok;
    }
    x.q0 = load_behind_wait(p.query_start + s);
    x.k0 = load_behind_wait(p.key_start + s);
    const long long ql = (long long)load_behind_wait(p.query_start + s + 1) - x.q0, kl = (long long)load_behind_wait(p.key_start + s + 1) - x.k0;
    x.ql = (int)ql;
    x.kl = (int)kl;
    return x.q0 >= 0 && x.k0 >= 0 && ql >= 0 && kl >= 0 && ql <= p.max_q && kl <= p.max_k && x.q0 + ql <= p.Tq &&
           x.k0 + kl <= p.Tk;
}

// kHeads: query blocks come in groups of p.group (two where the heads per K/V
// head are odd, so that tiles pair up), one group a level; else a sequence's
// tiles are one group.  The keys of a group's stages: the blocks of 128 that
// hold sinks, then those from the first query's window on.  A sequence of one
// packed tile and several partitions pairs the partitions instead: the unit's
// two tiles then hold the same rows and take turns at the stages: one tile
// alone waits for its own products (5 and 9 queries over 16,384 and 32,768
// keys, 12 / 2 heads: 26.9 us; with tiles of one head's rows, unpaired, 44.6).
struct Group {
    int blocks, units, sinks, low, np;      // query blocks (tiles) here; units per K/V head; key blocks; partitions
    bool pairs;
    __device__ __forceinline__ int per_head() const { return pairs ? (np + 1) / 2 : np * units; }
};
// keys that the queries of a block (a packed tile) see
template <int MODE>
__device__ __forceinline__ int key_end(const PromptParams& p, const Seq& x, int block) {
    if (MODE == kShared || !p.causal) return x.kl;
    int last = (block + 1) * kRows;
    if constexpr (MODE == kPacked) last = (last - 1) / p.g + 1;
    return max(x.kl - x.ql + min(x.ql, last), 0);
}
__device__ __forceinline__ int stages_to(const Group& g, int end) {
    const int blocks = ceil_div(end, kTok);
    return min(g.sinks, blocks) + max(0, blocks - max(g.low, g.sinks));
}
template <int MODE>
__device__ __forceinline__ bool group_of(const PromptParams& p, const Seq& x, int level, Group& g) {
    int first = 0;                          // the group's first query, and its last block
    if constexpr (MODE == kHeads) {
        first = level * p.group;
        g.blocks = min(p.group, ceil_div(x.ql, kRows) - first);
        g.units = (p.g * g.blocks + 1) / 2;
    } else {
        g.blocks = (int)(((long long)x.ql * p.g + kRows - 1) / kRows);
        g.units = (g.blocks + 1) / 2;
    }
    if (g.blocks <= 0 || (MODE == kShared && x.kl == 0)) return false;
    g.sinks = 0;
    g.low = 0;
    if (MODE != kShared && p.window > 0) {
        g.low = max(0, x.kl - x.ql + first * kRows - p.window + 1) / kTok;
        g.sinks = min(ceil_div(p.sinks, kTok), g.low);
    }
    const int n = stages_to(g, key_end<MODE>(p, x, first + g.blocks - 1));
    g.np = p.P > 0 && n > p.P ? ceil_div(n, p.P) : 1;
    g.pairs = MODE != kHeads && g.blocks == 1 && g.np > 1;
    return true;
}

// Tokens that sequence s shares with its group, by the bounds that attend_kernel keeps (0 for a group it skips).
__device__ __forceinline__ int shared_tokens(const PromptParams& p, int s) {
    int lo = 0, hi = p.S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (load_behind_wait(p.query_start + mid) <= s) lo = mid; else hi = mid;
    }
    Seq x;
    return p.S > 0 && sequence<kShared>(p, lo, x) && s >= x.q0 && s < x.q0 + x.ql ? x.kl : 0;
}

// A group's block ids, stage by stage, of one run of stages or two that are
// `apart` stages apart: 32 entries of the table at a time, one per lane, the
// next 32 on their way.
struct BlockIds {
    const int32_t* row;
    int blocks, next[2], tab[2], tab_next[2];      // blocks of the group; a run's next one and its entries
    __device__ __forceinline__ int load(int at) const {
        const int b = at + (int)(threadIdx.x & 31);
        return b < blocks ? __ldg(row + b) : 0;
    }
    __device__ __forceinline__ void start(const PromptParams& p, int member, int n, int stage, int apart) {
        row = p.tables + (size_t)member * p.MB;
        blocks = n;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            next[r] = (stage + r * apart) * (kTok / p.bs);
            if (r > 0 && apart == 0) break;
            tab[r] = load(next[r] & ~31);
            tab_next[r] = load((next[r] & ~31) + 32);
        }
    }
    // the next stage of run r; lane i: block i of its 8 or 4; -1 past the group's last, -2 out of the pool
    __device__ __forceinline__ int stage(const PromptParams& p, int r) { return r ? take(p, next[1], tab[1], tab_next[1]) : take(p, next[0], tab[0], tab_next[0]); }
    __device__ __forceinline__ int take(const PromptParams& p, int& at, int& now, int& then) {
        const int n = kTok / p.bs, i = threadIdx.x & 31;
        int pb = __shfl_sync(0xffffffffu, now, (at + i) & 31);
        if (i >= n || at + i >= blocks) pb = -1;
        else if (pb < 0 || pb >= p.NB) pb = -2;
        at += n;
        if ((at & 31) == 0) {
            now = then;
            then = load(at + 32);
        }
        return pb;
    }
};

// The blocks of a stage into a tile: a box per block and 64 values, one lane each.
template <int D>
__device__ __forceinline__ void load_blocks(const PromptParams& p, const CUtensorMap* map, uint32_t tile, int kvh, int pb,
                                            uint32_t there, uint32_t full) {
    constexpr int H = D / 64;
    const int lane = threadIdx.x & 31, b = lane / H, h = lane % H;
    const int id = __shfl_sync(0xffffffffu, pb, b);
    if (lane == 0) mbar_arrive_expect_tx(full, __popc(there) * (uint32_t)p.bs * 2 * D);
    __syncwarp();
    if (b < kTok / p.bs && id >= 0) tensor_load_2d(tile + h * (kTok * 128) + b * p.bs * 128, map, kvh * D + h * 64, id * p.bs, full);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap omap) {
    using C = Cfg<D, MODE>;
    constexpr bool SHARED = MODE == kShared, PACKED = MODE != kHeads;
    constexpr int NK = C::kKItems, NV = C::kVItems;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t ctl = smem_addr(smem_raw);
    const uint32_t base = (ctl + kCtlBytes + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (base + C::kTileBytes > ctl + C::kSmemBytes) {        // not on the boundary the layout counts on
        pdl_wait();
        if (tid == 0) report(p.err, PKV_DEVERR_TIMEOUT);
        return;
    }
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + kAbort);
    int4* ring = reinterpret_cast<int4*>(smem_raw + kRing);              // [2 units][4]
    volatile uint32_t* turns = reinterpret_cast<volatile uint32_t*>(smem_raw + kTurn);   // stages of each tile that had their turn
    uint32_t* masks = reinterpret_cast<uint32_t*>(smem_raw + kMasks);    // SHARED: tokens there are, stage g in slot g % 8
    auto ktile = [&](uint32_t j) { return base + (j % NK) * C::kItemBytes; };
    auto vtile = [&](uint32_t j) { return base + C::kVOff + (j % NV) * C::kItemBytes; };
    auto qbuf = [&](int t) { return base + C::kQOff + t * C::kItemBytes; };
    auto bar = [&](uint32_t off, int i) { return ctl + off + 8 * i; };
    pdl_trigger();

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kKFull, i), 1);
            mbar_init(bar(kKEmpty, i), 2);
            mbar_init(bar(kVFull, i), 1);
            mbar_init(bar(kVEmpty, i), 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(kSFull, t), 1);
            mbar_init(bar(kPFull, t), kSoftWarps / 2);
            mbar_init(bar(kPFull2, t), kSoftWarps / 2);
            mbar_init(bar(kPVDone, t), 1);
            mbar_init(bar(kQFull, t), 1);
            mbar_init(bar(kQEmpty, t), 1);
            mbar_init(bar(kUFull, t), 1);
            mbar_init(bar(kUEmpty, t), kSoftWarps + 3);
        }
        mbar_init(bar(kTail, 0), 1);
        mbar_init(bar(kFin, 0), 2);
        *abort_flag = 0;
        turns[0] = turns[1] = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) umma::tmem_alloc(ctl + kTmemSlot, kTmemCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem_raw + kTmemSlot);
    pdl_wait();

    // bounded wait; false once the limit passes or another role gave up
    auto wait = [&](uint32_t b, uint32_t parity, bool abortable) -> bool {
        if (mbar_try_wait(b, parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try_wait(b, parity)) {
            if (abortable && *abort_flag) return false;
            if (clock64() - t0 > kWaitLimit) {
                report(p.err, PKV_DEVERR_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
        return true;
    };
    if constexpr (SHARED) {
        // where each sequence's own part begins, and the longest one, for the kernels behind this one
        int own = 0;
        for (int s = blockIdx.x * kThreads + tid; s < p.Tq; s += gridDim.x * kThreads) {
            // A member that ends inside the shared tokens is decoded on its own (what its rows give here is not used):
            // tokens it does not see would weigh 0, but may hold what is not finite, or have never been written.
            const int n = min(load_behind_wait(p.lens + s), p.max_ctx), whole = shared_tokens(p, s);
            const int begin = n < whole ? 0 : whole;
            p.begin[s] = begin;
            own = max(own, n - begin);
        }
        own = __reduce_max_sync(0xffffffffu, own);
        if (lane == 0 && own > 0) atomicMax(p.own_max, own);
    }
    // Tiles take turns so that one's softmax runs beside the other's products,
    // not beside its softmax.  Only their pace depends on it: a tile that has
    // waited for as long as several stages goes on.  Tile t's stage j follows
    // the other's stage j (t 1) or j - 1 (t 0), `before` stages of the other in
    // the units before and `here` in this one.
    //
    // In turn go the products (by_products), or in long lists of 128-wide heads
    // the softmaxes, but for the last kTurnTail stages.  TFLOP/s with turns of
    // the softmaxes, of the products, without: d 128, 16,384 tokens both ways
    // 1,781, 1,574, 1,725; d 64, 4 x 4,096 tokens causal 878, 1,011, 941 (both
    // ways 783, 920, 881).  1,000 tokens alone (8 stages): turns of the products
    // 18.5 us, without 20.8.  kTurnStages 10, 16, 32: 8 x 6,000 tokens with a
    // window of 1,024 at 1,084, 1,136, 1,124, 16,384 at 1,754, 1,763, 1,680.
    auto by_products = [](int c0, int c1) { return D == 64 || min(c0, c1) < kTurnStages; };
    auto my_turn = [&](int t, int j, uint32_t before, int here) {
        const uint32_t need = before + min(t == 0 ? j : j + 1, here);
        const long long t0 = clock64();
        while ((int)(turns[t ^ 1] - need) < 0 && clock64() - t0 < kTurnLimit) {
        }
        __syncwarp();
    };
    // the first key of stage j of a unit's list
    auto stage_key = [](int j, int sinks, int low) { return (j < sinks ? j : j - sinks + low) * kTok; };
    // Stages of a unit whose tiles take c0 and c1 of them: the same ones, or
    // (paired partitions, c0 >= c1) each its own, in turn.  order: which of the
    // unit's stages tile t's stage j is; turn: the other way round, as the
    // tile's stage, plus p.P in tile 1's.
    auto count = [](bool pair, int c0, int c1) { return PACKED && pair ? c0 + c1 : max(c0, c1); };
    auto order = [](bool pair, int c1, int t, int j) { return PACKED && pair ? (j < c1 ? 2 * j + t : c1 + j) : j; };
    auto turn = [&](bool pair, int c1, int m) {
        return PACKED && pair ? (m < 2 * c1 ? m / 2 + (m & 1) * p.P : m - c1) : m;
    };
    // A parity wait is exact while the barrier is within one phase of the
    // awaited one; every wait below is by construction (a slot is filled again
    // once both tiles' products have gone past it).  K_j and V_j sit in
    // slots j % NK, j % NV (j counted over the block's stages); the per-tile
    // barriers count the stages that tile took part in.

    if (warp == kKWarp) {
        // ------------------------------------------------- units and K tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // the highest query block group of any sequence
        int level = 0;
        // this lane's sequence of the current 32, its group at this level, and the units up to its own
        Seq x{};
        Group gr{};
        bool there = false;
        for (int s = lane; s < p.S; s += 32) {
            there = sequence<MODE>(p, s, x);
            if (there) level = max(level, PACKED ? 1 : ceil_div(x.ql, p.group * kRows));
            else if (blockIdx.x == 0) report(p.err, PKV_DEVERR_QUERY_LEN);
        }
        level = __reduce_max_sync(0xffffffffu, level) - 1;
        int at = -32;
        long long before = 0, mine = 0, upto = 0, total = 0;
        auto next_batch = [&]() -> bool {
            before += total;
            at += 32;
            if (at >= p.S) {
                at = 0;
                --level;
            }
            if (level < 0) return false;
            mine = 0;
            if (p.S > 32) there = at + lane < p.S && sequence<MODE>(p, at + lane, x);
            if (there && group_of<MODE>(p, x, level, gr)) mine = (long long)p.Hkv * gr.per_head();
            upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            total = __shfl_sync(0xffffffffu, upto, 31);
            return true;
        };
        long long ticket = blockIdx.x;
        uint32_t g = 0, un = 0;
        bool ok = true, bad = false, more = level >= 0 && next_batch();
        for (;;) {
            while (more && ticket >= before + total) more = next_batch();
            const int slot = un & 1;
            if (un >= 2) ok = wait(bar(kUEmpty, slot), ((un >> 1) - 1) & 1, true);
            if (__any_sync(0xffffffffu, !ok)) break;
            if (!more) {
                if (lane == 0) {
                    ring[4 * slot + 1] = make_int4(-1, 0, 0, 0);
                    umma::mbar_arrive(bar(kUFull, slot));
                }
                break;
            }
            const int owner = __ffs(__ballot_sync(0xffffffffu, ticket < before + upto)) - 1;
            int4 e0, e1, e2, e3;
            if (lane == owner) {
                const int rel = (int)(ticket - before - (upto - mine)), per = gr.per_head(), kvh = rel / per;
                int part = gr.pairs ? 2 * (rel - kvh * per) : (rel - kvh * per) / gr.units;
                const int u = gr.pairs ? 0 : rel - kvh * per - part * gr.units;
                const int j0 = gr.np > 1 ? part * p.P : 0, cap = gr.np > 1 ? p.P : 0x7fffffff;
                // the tiles' query blocks (packed: tiles) and heads; -1: no second tile; packed, 1: paired partitions
                int b0 = 2 * u, h0 = 0, b1 = 2 * u + 1, h1 = 2 * u + 1 < gr.blocks ? 0 : -1;
                if constexpr (!PACKED) {
                    b0 = level * p.group + 2 * u / p.g;
                    h0 = 2 * u % p.g;
                    b1 = level * p.group + (2 * u + 1) / p.g;
                    h1 = 2 * u + 1 < p.g * gr.blocks ? (2 * u + 1) % p.g : -1;
                }
                const int n0 = stages_to(gr, key_end<MODE>(p, x, b0)) - j0;
                int n1 = stages_to(gr, key_end<MODE>(p, x, b1)) - j0;
                if (gr.pairs) {
                    b1 = 0;
                    h1 = part + 1 < gr.np ? 1 : -1;
                    n1 = n0 - p.P;
                }
                e0 = make_int4(x.q0, x.k0, x.ql, x.kl);
                e1 = make_int4(kvh, gr.np, part, j0);
                e2 = make_int4(gr.sinks, max(gr.low, gr.sinks), min(max(n0, 0), cap), h1 < 0 ? 0 : min(max(n1, 0), cap));
                e3 = make_int4(b0, h0, b1, h1);
                int4* e = ring + 4 * slot;
                e[0] = e0;
                e[1] = e1;
                e[2] = e2;
                e[3] = e3;
                umma::mbar_arrive(bar(kUFull, slot));
            }
            const int k0 = __shfl_sync(0xffffffffu, e0.y, owner), kvh = __shfl_sync(0xffffffffu, e1.x, owner);
            const int j0 = __shfl_sync(0xffffffffu, e1.w, owner), sinks = __shfl_sync(0xffffffffu, e2.x, owner);
            const int low = __shfl_sync(0xffffffffu, e2.y, owner);
            const int c1 = __shfl_sync(0xffffffffu, e2.w, owner);
            const bool pair = PACKED && __shfl_sync(0xffffffffu, e3.w, owner) > 0;
            const int n = count(pair, __shfl_sync(0xffffffffu, e2.z, owner), c1);
            BlockIds ids;
            if constexpr (SHARED)
                ids.start(p, __shfl_sync(0xffffffffu, e0.x, owner), __shfl_sync(0xffffffffu, e0.w, owner) / p.bs, j0,
                          pair ? p.P : 0);
            // the next ticket, on its way while the tiles are requested
            long long claimed = 0;
            if (p.sched != nullptr && lane == 0)
                claimed = (long long)atomicAdd(reinterpret_cast<unsigned long long*>(p.sched), 1ull);
            for (int j = 0; j < n; ++j, ++g) {
                if (g >= (uint32_t)NK) ok = wait(bar(kKEmpty, g % NK), (g / NK - 1) & 1, true);
                if (__any_sync(0xffffffffu, !ok)) {
                    bad = true;
                    break;
                }
                if constexpr (SHARED) {
                    // which of the stage's tokens there are: a block whose id is out of the pool is absent
                    // (stage g - 8's were read: both tiles' products have gone past stage g - NK, NK < 8)
                    const int pb = ids.stage(p, pair && j < 2 * c1 ? j & 1 : 0);
                    const uint32_t there = __ballot_sync(0xffffffffu, pb >= 0);
                    if (pb == -2) report(p.err, PKV_DEVERR_BLOCK_ID);
                    if (lane < 4) {
                        uint32_t w = (there >> lane) & 1u ? 0xffffffffu : 0u;
                        if (p.bs == 16) w = ((there >> (2 * lane)) & 1u ? 0xffffu : 0u) | ((there >> (2 * lane)) & 2u ? 0xffff0000u : 0u);
                        masks[4 * (g & 7) + lane] = w;
                    }
                    __syncwarp();
                    load_blocks<D>(p, &kmap, ktile(g), kvh, pb, there, bar(kKFull, g % NK));
                    continue;
                }
                if (lane == 0) {
                    const uint32_t full = bar(kKFull, g % NK);
                    mbar_arrive_expect_tx(full, C::kItemBytes);
                    const int row = k0 + stage_key(j0 + turn(pair, c1, j), sinks, low);
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        tensor_load_2d(ktile(g) + h * (kTok * 128), &kmap, kvh * D + h * 64, row, full);
                }
                __syncwarp();
            }
            if (bad) break;
            ticket = p.sched != nullptr ? (long long)gridDim.x + __shfl_sync(0xffffffffu, claimed, 0) : ticket + gridDim.x;
            ++un;
        }
        // copies still in flight land before the block leaves
        for (uint32_t k = 1; k <= (uint32_t)NK && k <= g; ++k)
            wait(bar(kKFull, (g - k) % NK), ((g - k) / NK) & 1, false);
        if (p.sched != nullptr && lane == 0) {
            unsigned long long* ctr = reinterpret_cast<unsigned long long*>(p.sched);
            __threadfence();
            if (atomicAdd(ctr + 1, 1ull) == gridDim.x - 1) {
                atomicExch(ctr, 0ull);
                atomicExch(ctr + 1, 0ull);
            }
        }
    } else if (warp == kVWarp) {
        // ------------------------------------------------------ Q and V tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        uint32_t g = 0, un = 0, tails = 0, qu[2] = {0u, 0u};
        bool ok = true, bad = false;
        for (;;) {
            const int slot = un & 1;
            ok = wait(bar(kUFull, slot), (un >> 1) & 1, true);
            if (__any_sync(0xffffffffu, !ok)) break;
            const int4 e0 = ring[4 * slot], e1 = ring[4 * slot + 1], e2 = ring[4 * slot + 2], e3 = ring[4 * slot + 3];
            const bool pair = PACKED && e3.w > 0;
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(bar(kUEmpty, slot));
            if (e1.x < 0) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (PACKED || (t == 0 ? e2.z : e2.w) == 0) continue;       // no keys, or no tile
                if (qu[t] >= 1) ok = wait(bar(kQEmpty, t), (qu[t] - 1) & 1, true);
                if (__any_sync(0xffffffffu, !ok)) {
                    bad = true;
                    break;
                }
                if (lane == 0) {
                    // rows past the sequence's last are other sequences' or zeros: their results are not stored
                    mbar_arrive_expect_tx(bar(kQFull, t), C::kItemBytes);
                    const int head = e1.x * p.g + (t == 0 ? e3.y : e3.w), row = e0.x + (t == 0 ? e3.x : e3.z) * kRows;
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        tensor_load_2d(qbuf(t) + h * (kRows * 128), &qmap, head * D + h * 64, row, bar(kQFull, t));
                }
                __syncwarp();
                ++qu[t];
            }
            if (bad) break;
            const int n = count(pair, e2.z, e2.w);
            // keys between the sinks and the first query's window: no query of the sequence sees them
            const int hidden0 = p.sinks, hidden1 = !SHARED && p.window > 0 ? e0.w - e0.z - p.window + 1 : 0;
            BlockIds ids;
            if constexpr (SHARED) ids.start(p, e0.x, e0.w / p.bs, e1.w, pair ? p.P : 0);
            for (int j = 0; j < n; ++j, ++g) {
                if (g >= (uint32_t)NV) ok = wait(bar(kVEmpty, g % NV), (g / NV - 1) & 1, true);
                if (__any_sync(0xffffffffu, !ok)) {
                    bad = true;
                    break;
                }
                const int key = stage_key(e1.w + turn(pair, e2.w, j), e2.x, e2.y);
                // rows of the tile, in eighths (SHARED: a block or half of one) or counted, that hold something, and whether
                // some of them are unseen
                const int here = e0.w - key;
                uint32_t there = 0xffu;
                int pb = 0;
                if constexpr (SHARED) {
                    pb = ids.stage(p, pair && j < 2 * e2.w ? j & 1 : 0);
                    there = __ballot_sync(0xffffffffu, pb >= 0);
                }
                const bool unseen = hidden0 < hidden1 && key < hidden1 && key + kTok > hidden0;
                const bool part = SHARED ? there != (p.bs == 16 ? 0xffu : 0xfu) : here < kTok || unseen;
                const uint32_t full = bar(kVFull, g % NV), landed = part ? bar(kTail, 0) : full;
                if constexpr (SHARED) {
                    load_blocks<D>(p, &vmap, vtile(g), e1.x, pb, there, landed);
                } else if (lane == 0) {
                    mbar_arrive_expect_tx(landed, C::kItemBytes);
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        tensor_load_2d(vtile(g) + h * (kTok * 128), &vmap, e1.x * D + h * 64, e0.y + key, landed);
                }
                __syncwarp();
                if (part) {
                    ok = wait(landed, tails & 1, false);
                    ++tails;
                    if (__any_sync(0xffffffffu, !ok)) {
                        bad = true;
                        break;
                    }
                    const uint32_t vb = vtile(g);
                    for (int i = (SHARED || unseen ? 0 : here * 8) + lane; i < kTok * 8; i += 32) {
                        if (SHARED && ((there >> (i / 8 / p.bs)) & 1u)) continue;
                        if (!SHARED && i < here * 8 && (key + i / 8 < hidden0 || key + i / 8 >= hidden1)) continue;
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vb + h * (kTok * 128) + i * 16), "r"(0u)
                                         : "memory");
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(full);
                }
            }
            if (bad) break;
            ++un;
        }
        for (uint32_t k = 1; k <= (uint32_t)NV && k <= g; ++k)
            wait(bar(kVFull, (g - k) % NV), ((g - k) / NV) & 1, false);
        for (int t = 0; t < 2; ++t)
            if (qu[t] > 0) wait(bar(kQFull, t), (qu[t] - 1) & 1, false);
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ----------------------------------------------------------- products
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // The whole warp walks the loop and one elected thread issues: the
        // operands are then uniform, and a product takes its 64 clocks.  Issued
        // by `if (lane == 0)` every operand goes through a vector register, and
        // a product took 123-147 clocks to issue.
        constexpr uint32_t idS = umma::idesc_bf16_f32(kRows, kTok, false);
        constexpr uint32_t idPV = umma::idesc_bf16_f32(kRows, D, true);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        // descriptors of the first K step of slot 0; a slot or K step on adds to the address, in 16 bytes
        const uint64_t q_desc = umma::desc_sw128(qbuf(0), 16, 1024), k_desc = umma::desc_sw128(base, 16, 1024);
        const uint64_t v_desc = umma::desc_sw128(base + C::kVOff, kTok * 128, 1024);
        const int t = __shfl_sync(0xffffffffu, warp - kMmaWarp, 0);
        uint32_t g = 0, un = 0, gt = 0, qu = 0, before = 0;
        bool ok = true;
        // waits of the whole warp
        auto all = [&](uint32_t b, uint32_t parity) -> bool { return !__any_sync(0xffffffffu, !wait(b, parity, true)); };
        // a slot, once what was issued before has read it
        auto release = [&](uint32_t b) {
            if (elect_one()) umma::commit(b);
            __syncwarp();
        };
        // The other tile's stages, before stage `to`: each is waited for and released like the tile's own, so
        // that no slot is filled twice between two waits (of one parity), nor while this tile counts on it
        uint32_t ks = 0, vs = 0;                             // the next K and V stages of the block
        auto skip_k = [&](uint32_t to) -> bool {
            for (; ks != to; ++ks) {
                if (!all(bar(kKFull, ks % NK), (ks / NK) & 1)) return false;
                if (lane == 0) umma::mbar_arrive(bar(kKEmpty, ks % NK));
            }
            return true;
        };
        auto skip_v = [&](uint32_t to) -> bool {
            for (; vs != to; ++vs) {
                if (!all(bar(kVFull, vs % NV), (vs / NV) & 1)) return false;
                if (lane == 0) umma::mbar_arrive(bar(kVEmpty, vs % NV));
            }
            return true;
        };
        auto issue_s = [&](uint32_t gs, bool last) {
            const uint64_t kd = k_desc + (gs % NK) * (C::kItemBytes / 16), qd = q_desc + t * (C::kItemBytes / 16);
            umma::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) / 16;
                    umma::mma_bf16(tm + tmem_s(t), qd + off, kd + off, idS, kk > 0);
                }
                umma::commit(bar(kSFull, t));
                if (last && !PACKED) umma::commit(bar(kQEmpty, t));
            }
            __syncwarp();
            release(bar(kKEmpty, gs % NK));
            ks = gs + 1;
        };
        // half of a stage's keys
        auto issue_pv = [&](uint32_t gs, int half, bool first) {
            const uint64_t vd = v_desc + (gs % NV) * (C::kItemBytes / 16) + half * (kTok / 2 * 128 / 16);
            umma::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTok / 32; ++kk)
                    mma_ts(tm + tmem_o(t), tm + tmem_s(t) + half * (kTok / 4) + kk * 8, vd + kk * (2048 / 16), idPV,
                           !(first && kk == 0));
                if (half) umma::commit(bar(kPVDone, t));
            }
            __syncwarp();
        };
        for (;;) {
            const int slot = un & 1;
            if (!all(bar(kUFull, slot), (un >> 1) & 1)) break;
            const int kvh = __shfl_sync(0xffffffffu, ring[4 * slot + 1].x, 0);
            const int c0 = __shfl_sync(0xffffffffu, ring[4 * slot + 2].z, 0), c1 = __shfl_sync(0xffffffffu, ring[4 * slot + 2].w, 0);
            const bool pair = PACKED && __shfl_sync(0xffffffffu, ring[4 * slot + 3].w, 0) > 0;
            __syncwarp();
            if (lane == 0 && (!PACKED || kvh < 0)) umma::mbar_arrive(bar(kUEmpty, slot));
            if (kvh < 0) break;
            const int c = t ? c1 : c0;
            const bool in_turn = by_products(c0, c1);
            const uint32_t end = g + count(pair, c0, c1);
            if (c > 0) {
                const uint32_t s0 = g + order(pair, c1, t, 0);
                // the tile's last P . V has read S's buffer (and its last S was before that)
                if (gt > 0) ok = all(bar(kPVDone, t), (gt - 1) & 1);
                if (!ok) break;
                if constexpr (PACKED) {
                    // rows of (query, head) pairs are gathered: by this warp, which waits for them anyway
                    DecodeParams q{};
                    q.q = p.q;
                    q.Hq = (int)(p.q_stride / D);                // (heads from one token to the next)
                    q.g = p.g;
                    const int4 e0 = ring[4 * slot], e3 = ring[4 * slot + 3];
                    const int r0 = (t == 0 ? e3.x : e3.z) * kRows;
                    load_q_rows<D, kRows>(q, e0.x, kvh, r0, 0, kRows, e0.z * p.g - r0, qbuf(t));
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    fence_proxy_async();
                    __syncwarp();
                } else {
                    ok = all(bar(kQFull, t), qu & 1);
                }
                ok = ok && skip_k(s0) && all(bar(kKFull, s0 % NK), (s0 / NK) & 1);
                if (!ok) break;
                issue_s(s0, c == 1);
            }
            if constexpr (PACKED) {
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(bar(kUEmpty, slot));
            }
            for (int j = 0; j < c; ++j, ++gt) {
                const uint32_t s0 = g + order(pair, c1, t, j);
                ok = skip_v(s0) && all(bar(kVFull, s0 % NV), (s0 / NV) & 1) && all(bar(kPFull, t), gt & 1);
                if (!ok) break;
                if (in_turn) my_turn(t, j, before, t ? c0 : c1);
                issue_pv(s0, 0, j == 0);
                ok = all(bar(kPFull2, t), gt & 1);
                if (!ok) break;
                issue_pv(s0, 1, false);
                release(bar(kVEmpty, s0 % NV));
                vs = s0 + 1;
                if (j + 1 < c) {
                    // the next S_t overwrites P_t: only after P_t . V_j is done
                    const uint32_t s1 = g + order(pair, c1, t, j + 1);
                    ok = skip_k(s1) && all(bar(kKFull, s1 % NK), (s1 / NK) & 1) && all(bar(kPVDone, t), gt & 1);
                    if (!ok) break;
                    issue_s(s1, j + 2 == c);
                }
                if (in_turn && lane == 0) turns[t] = gt + 1;
            }
            while (ok && ks != end) ok = skip_k(ks + 1) && skip_v(ks);
            if (!ok) break;
            before += t ? c0 : c1;
            g = end;
            qu += c > 0;
            ++un;
        }
        // every product issued here completes before the block releases TMEM
        release(bar(kFin, 0));
        wait(bar(kFin, 0), 0, false);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int t = warp >> 2;                              // tile
        const int i = (warp & 3) * 32 + lane;                // row of the tile, TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + lane_base + tmem_s(t);
        const uint32_t o_col = tmem + lane_base + tmem_o(t);
        uint32_t gt = 0, un = 0, gs = 0, before = 0;
        bool ok = true, bad = false;
        for (;;) {
            const int slot = un & 1;
            ok = wait(bar(kUFull, slot), (un >> 1) & 1, true);
            if (__any_sync(0xffffffffu, !ok)) break;
            const int4 e0 = ring[4 * slot], e1 = ring[4 * slot + 1], e2 = ring[4 * slot + 2], e3 = ring[4 * slot + 3];
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(bar(kUEmpty, slot));
            if (e1.x < 0) break;
            ++un;
            const int head = t == 0 ? e3.y : e3.w, n = t == 0 ? e2.z : e2.w;
            const bool pair = PACKED && e3.w > 0;
            const uint32_t stages = gs;                          // the unit's first in the block's count (SHARED's masks)
            gs += count(pair, e2.z, e2.w);
            const int here = t == 0 ? e2.w : e2.z;               // the other tile's stages
            const uint32_t before_here = before;
            before += here;
            if (head < 0) continue;                              // the unit has one tile
            const bool in_turn = by_products(n, here);
            const int block = t == 0 ? e3.x : e3.z;
            const int ql = e0.z, kl = e0.w;
            int qi = block * kRows + i, hh = head;               // this row's query and head of the K/V head's
            bool rv = qi < ql;
            int first = p.causal ? kl - ql + block * kRows : kl - 1;             // position of the tile's first row
            int pos = p.causal ? first + i : kl - 1;
            int far = p.causal ? first + kRows - 1 : kl - 1;               // and of its last
            if constexpr (PACKED) {
                hh = qi % p.g;
                qi /= p.g;
                rv = qi < ql;
                first = p.causal ? kl - ql + block * kRows / p.g : kl - 1;
                pos = p.causal ? kl - ql + qi : kl - 1;
                far = p.causal ? kl - ql + (block * kRows + kRows - 1) / p.g : kl - 1;
            }
            const int j0 = e1.w + (pair && t ? p.P : 0);         // the tile's first stage
            const bool flip = !(p.scale_log2 > 0.f);
            const float scl = flip ? 1.f : p.scale_log2;
            float m_ref = -CUDART_INF_F, l = 0.f;
            for (int j = 0; j < n; ++j, ++gt) {
                ok = wait(bar(kSFull, t), gt & 1, true);
                if (__any_sync(0xffffffffu, !ok)) {
                    bad = true;
                    break;
                }
                umma::fence_after_sync();
                if (!in_turn && n - j >= kTurnTail) my_turn(t, j, before_here, here);
                const int key = stage_key(j0 + j, e2.x, e2.y);
                const uint32_t* there = masks + 4 * ((stages + order(pair, e2.w, t, j)) & 7);
                bool whole = !flip && key + kTok - 1 <= min(first, kl - 1) &&
                             (p.window == 0 || key + kTok <= p.sinks || key > far - p.window);
                if constexpr (SHARED) whole = whole && (there[0] & there[1] & there[2] & there[3]) == 0xffffffffu;
                if (!whole) {
                    // -inf where this row does not see the key, in place: few stages need it, and their code, a
                    // word of 32 keys at a time, stays out of the others' way
#pragma unroll 1
                    for (int w = 0; w < kTok / 32; ++w) {
                        const int v0 = key + 32 * w;
                        uint32_t seen = bits_below(min(pos, kl - 1) + 1 - v0);
                        if constexpr (SHARED) seen &= there[w];
                        else if (p.window > 0) seen &= ~bits_between(v0, p.sinks, pos - p.window + 1);
                        if (!flip && __all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
                        uint32_t x[32];
#pragma unroll
                        for (int b = 0; b < 32; ++b) x[b] = 0xff800000u;
                        if (!__any_sync(0xffffffffu, seen != 0)) {
                            // hidden from the whole warp (8 x 6,000 tokens with a window of 1,024 at 1,153 TFLOP/s, read
                            // all the same at 1,123)
                            umma::tmem_st32(s_col + 32 * w, x);
                            continue;
                        }
                        umma::tmem_ld32(s_col + 32 * w, x);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int b = 0; b < 32; ++b) {
                            if (flip) x[b] = __float_as_uint(__uint_as_float(x[b]) * p.scale_log2);
                            if (!((seen >> b) & 1u)) x[b] = 0xff800000u;
                        }
                        umma::tmem_st32(s_col + 32 * w, x);
                    }
                    umma::tmem_wait_st();
                }
                uint32_t sr[kTok / 32][32];
#pragma unroll
                for (int w = 0; w < kTok / 32; ++w) umma::tmem_ld32(s_col + 32 * w, sr[w]);
                umma::tmem_wait_ld();
                float mx8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mx8[k] = __uint_as_float(sr[0][k]);
#pragma unroll
                for (int b = 8; b < kTok; ++b) mx8[b & 7] = fmaxf(mx8[b & 7], __uint_as_float(sr[b >> 5][b & 31]));
                const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                       fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))) * scl;
                float alpha = 1.f;
                bool resc = false;
                if (j == 0) {
                    m_ref = mx;
                } else if (mx > m_ref + kRescaleLog2) {
                    if (m_ref != -CUDART_INF_F) {
                        alpha = fast_exp2(m_ref - mx);
                        resc = true;
                    }
                    m_ref = mx;
                }
                l *= alpha;
                const float mb = m_ref == -CUDART_INF_F ? 0.f : m_ref;
                const uint64_t xs2 = umma::f2_pack(scl, scl), nmb2 = umma::f2_pack(-mb, -mb);
                uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
                if (__any_sync(0xffffffffu, resc)) {
                    // O_t holds the products up to the previous stage
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t ov[16];
                        tmem_ld16(o_col + c0, ov);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
                        tmem_st16(o_col + c0, ov);
                    }
                }
                // P in two halves: the product with the first 64 keys runs while the others are weighed
#pragma unroll
                for (int w = 0; w < kTok / 32; ++w) {
                    uint32_t pw[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const uint64_t s01 = umma::f2_pack(__uint_as_float(sr[w][2 * k]), __uint_as_float(sr[w][2 * k + 1]));
                        float x0, x1;
                        umma::f2_unpack(umma::f2_fma(s01, xs2, nmb2), x0, x1);
                        const float a0 = fast_exp2(x0), a1 = fast_exp2(x1);
                        ls2[k & 3] = umma::f2_add(ls2[k & 3], umma::f2_pack(a0, a1));
                        pw[k] = pack2<false>(a0, a1);
                    }
                    tmem_st16(s_col + 16 * w, pw);
                    if (w & 1) {
                        umma::tmem_wait_st();
                        umma::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(bar(w == 1 ? kPFull : kPFull2, t));
                    }
                }
                if (!in_turn && (tid & 127) == 0) turns[t] = gt + 1;
                float ls[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) umma::f2_unpack(ls2[k], ls[2 * k], ls[2 * k + 1]);
                l += ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
            }
            if (bad) break;

            // O / l, or the partition's (m, l, O), once the tile's last product is done
            if (n > 0) {
                ok = wait(bar(kPVDone, t), (gt - 1) & 1, true);
                if (__any_sync(0xffffffffu, !ok)) break;
                umma::fence_after_sync();
            }
            const int np = e1.y, part = e1.z + (pair && t ? 1 : 0);
            const size_t row = (size_t)(e0.x + qi), hrow = row * p.Hq + e1.x * p.g + hh;
            const float f = l > 0.f || l != l ? 1.f / l : 0.f;
            // A row that sees no key here is zeros: its weights are, but 0 times a V value that is not finite is not (and
            // O_t holds anything where there were no keys).
            const bool unseen = l == 0.f;
            // Whole warps of rows leave by TMA, 64 columns at a time through shared memory: stored by the threads, a row
            // each, 32 lines per instruction, 64 x 512 tokens take 204 us in both directions, not 189; 32 columns at a time
            // they run at 1,308 TFLOP/s, not 1,360.  (Loops: unrolled they are 4 KB of code that a unit runs once; 64 x 512
            // tokens 178 us, not 159.)
            const bool whole_rows = MODE == kHeads && np == 1 && block * kRows + (warp & 3) * 32 + 31 < ql;
            if (whole_rows) {
                const uint32_t keep = unseen ? 0u : 0xffffffffu;
                const uint32_t out = base + C::kOutOff + t * C::kOutBytes + (warp & 3) * 4096;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 64) {
                    uint32_t oa[32], ob[32];
                    umma::tmem_ld32(o_col + c0, oa);
                    umma::tmem_ld32(o_col + c0 + 32, ob);
                    // what was stored from here before has been read
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
                    umma::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int q = 8 * (k & 3) + 2 * e;
                            w[e] = keep & pack2<false>(__uint_as_float(k < 4 ? oa[q] : ob[q]) * f,
                                                       __uint_as_float(k < 4 ? oa[q + 1] : ob[q + 1]) * f);
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(out + lane * 128 + (k ^ (lane & 7)) * 16),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0)
                        tensor_store_2d(&omap, out, (e1.x * p.g + head) * D + c0, e0.x + block * kRows + (warp & 3) * 32);
                }
            } else
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t ov[32];
                umma::tmem_ld32(o_col + c0, ov);
                umma::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) ov[k] = unseen ? 0u : ov[k];
                if (rv) {
                    if (!SHARED && np == 1) {
                        store_row32(static_cast<__nv_bfloat16*>(p.out) + hrow * D + c0, ov, f,
                                    (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0);
                    } else {
                        store_part32(p.part_acc + (hrow * p.Pmax + part) * D + c0, ov,
                                     (reinterpret_cast<uintptr_t>(p.part_acc) & 31u) == 0);
                    }
                }
                __syncwarp();
            }
            if (rv && (SHARED || np > 1)) {
                const size_t u = hrow * p.Pmax + part;
                p.part_ml[2 * u] = m_ref;
                p.part_ml[2 * u + 1] = l;
            }
            umma::fence_before_sync();
        }
        // the output stored from shared memory is in place before the block leaves
        if (MODE == kHeads && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    umma::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, int MODE>
cudaError_t launch_attend(const PromptParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          const CUtensorMap& omap, long long units, int num_sms, cudaStream_t st) {
    using C = Cfg<D, MODE>;
    auto kern = attend_kernel<D, MODE>;
    // the register shares must fit in what the block is launched with
    // (setmaxnreg waits forever otherwise): checked once, on the binary
    static std::once_flag checked;
    static cudaError_t check = cudaSuccess;
    std::call_once(checked, [&] {
        cudaFuncAttributes fa;
        check = cudaFuncGetAttributes(&fa, kern);
        if (check == cudaSuccess &&
            (fa.numRegs * kThreads < 32 * kSoftWarps * kSoftRegs + 128 * kOtherRegs || fa.maxThreadsPerBlock < kThreads))
            check = cudaErrorInvalidConfiguration;
    });
    if (check != cudaSuccess) return check;
    static SmemOptIn optin;
    cudaError_t e = optin.ensure(reinterpret_cast<const void*>(kern), C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const int grid = (int)(units < num_sms ? (units > 0 ? units : 1) : num_sms);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), C::kSmemBytes, st, p, qmap, kmap, vmap, omap);
}

}  // namespace
}  // namespace pkv
