// paged_attention_decode_kv4: one query per sequence over a 4-bit cache
// (sm_103a), under an optional sliding window.
//
// "LLM推論の基礎とvLLMの内部", section 1: decode is bound by memory bandwidth;
// section 2: fewer bytes per K/V element are read faster, as long as the
// arithmetic per element keeps up.  The format is in pkv_kv4.cuh.
//
// Work units, their order and the ring of stages per warp are the
// tensor-core decode's (pkv_units.cuh); a stage is kTok tokens of one K/V
// head, each block's K and V one bulk copy of bs * 5 d / 8 contiguous bytes
// (cp.async.bulk onto the stage's mbarrier).
//
// The bound is HBM for the bytes (160 per token and K/V head of 128 values)
// and, close behind, the instruction issue: an SM must take a 16-token tile
// of K and V every ~109 cycles to keep up, 436 issue slots over its four
// schedulers.  So nothing is unpacked value by value:
//
//  - A 4-bit code in the low bits of a 16-bit half is itself an fp16 number,
//    the subnormal code * 2^-24 (* 2^-20 one nibble higher), which the matrix
//    instructions take exactly.  Two codes of a register are one AND.  Of the
//    two operand registers of a k-step, one holds codes at 2^-24 and one at
//    2^-20; the query's fragments carry 4 and 1/4, so both products are
//    code * q * 2^-22.  For V the two registers are different rows of the
//    result, whose factor is applied once at the end.
//  - K: x = sum_g s_g (sum_{d in g} code q) + sum_g z_g (sum_{d in g} q).  The
//    scale multiplies the four accumulators of a group's two products, not
//    the 64 codes; the zeros meet the query's group sums in one m16n8k8
//    product, the sums split into two fp16 parts (22 bits together).
//  - V: o_d = sum_t code_td (s_tg p_t) + sum_t z_tg p_t.  The scale goes onto
//    the 16-token fragment of the weights (two products of pairs per group);
//    the zeros' part of all groups is one more product, z^T . P^T, whose row
//    g is added to the group's values at the end.
//
// Rounding: p to fp16 and s * p to fp16 (2^-11 each); everything else
// accumulates in fp32.  The weights carry 2^12 (into the exponential's
// argument, off again at the unit's end), so that neither p nor s * p is below
// fp16's smallest normal number where it counts: of the zeros' part a token of
// weight p then loses no more than of the codes' part, whose loss would pull
// the result towards the groups' minima (values of 1e-3, 32,768 tokens whose
// logits have a deviation of 3: 37% off without it).  A group with a scale of
// 2 or more (values that span 30 tensor scales) takes its weights times 2^-j,
// so that s * p stays below 2^16, and its accumulators carry the 2^-j.  The
// test for such scales is two loads, four ORs and a vote per stage: 32 x 32,768
// tokens take 223.8 us with and without all this, 267 with a scale of 2 or more
// in every stage.  The query goes to fp16 after a power of two per unit (256 x
// 1..4,096 tokens: 80.3 us without and 80.7 with it, others the same).
//
// 32 sequences of 32,768 tokens (64 / 8 heads of 128, 1.34 GB): 221 us a call
// in a loop, 228 where every call has other inputs, 5.9-6.1 TB/s, 87-90% of the
// measured copy rate; the same tokens take 378 us from an E4M3 cache and 630
// from a bf16 one (in a loop).  A 16-token tile is 268 instructions of those
// 436 slots.  Warps x tokens per stage (two stages each, what shared memory
// holds; measured before the weights carried 2^12): 11 x 64 226 us, 10 x 64
// 226, 8 x 64 254, 16 x 32 270, 14 x 32 284.  The whole launch is one kernel
// and the partitions' merge.
#include <cuda_fp16.h>
#include <math_constants.h>

#include <type_traits>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_kv4.cuh"
#include "pkv_tc_common.cuh"
#include "pkv_units.cuh"

namespace pkv {
namespace {

using namespace tc;

#ifndef PKV_KV4_WARPS
#define PKV_KV4_WARPS 11
#endif
#ifndef PKV_KV4_STAGES
#define PKV_KV4_STAGES 2
#endif
#ifndef PKV_KV4_TOK
#define PKV_KV4_TOK 64
#endif

constexpr long long kWaitLimitCycles = 4000000000LL;   // ~2 s: a stage that never lands

template <int D>
struct KCfg {
    static constexpr int kWarps = PKV_KV4_WARPS, kStages = PKV_KV4_STAGES, kTok = PKV_KV4_TOK;
    static constexpr int kMT = kTok / 16, kMasks = kTok / 32;
    static constexpr int G = D / kKv4Group;
    static constexpr int kPartBytes = kTok * (D / 2 + D / 8);       // K (or V) of a stage
    static constexpr int kStageBytes = 2 * kPartBytes;
    static constexpr int kQueue = kStages;
    // trailer per worker: barriers, stage masks, the queue of claimed units (16-byte aligned), the unit's shifts
    static constexpr int kQueueOff = (8 * kStages + 4 * kMasks * kStages + 15) / 16 * 16;
    static constexpr int kShiftOff = kQueueOff + 32 * kQueue;
    static constexpr int kCtlBytes = kShiftOff + 16;
    static constexpr int kWarpBytes = kStages * kStageBytes + kCtlBytes;
    static constexpr int kSmemBytes = kWarps * kWarpBytes;
    static_assert(kTok == 32 || kTok == 64, "whole blocks of 16 or 32 tokens");
    static_assert(kStageBytes % 16 == 0 && kCtlBytes % 16 == 0, "bulk copies want 16-byte addresses");
    static_assert(kSmemBytes <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(pol)
        : "memory");
}
__device__ __forceinline__ void mma1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <int G>
__device__ __forceinline__ void lds_words(const unsigned char* p, uint32_t (&w)[G]) {
    if constexpr (G == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    }
}

// the weight 2^(x xs + mu) of a logit; absent tokens (x = -inf, also where xs is 0) weigh nothing
template <bool WHOLE>
__device__ __forceinline__ float weight(float x, float xs, float mu) {
    if constexpr (!WHOLE)
        if (x == -CUDART_INF_F) return 0.f;
    return fast_exp2(fmaf(x, xs, mu));
}

constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;   // codes at 2^-24 and at 2^-20
constexpr float kWeightLog2 = 12.f, kWeightInv = 1.f / 4096.f;   // what the weights carry

// 2^x, x in [-126, 127]
__device__ __forceinline__ float pow2(int x) { return __uint_as_float((uint32_t)(127 + x) << 23); }

template <int D, int BS, bool WIN>
__global__ void __launch_bounds__(KCfg<D>::kWarps * 32, 1)
    decode_kv4_kernel(const __grid_constant__ DecodeParams p, unsigned long long total_units,
                      unsigned long long region_a, int nsets) {
    using C = KCfg<D>;
    constexpr int G = C::G, kTok = C::kTok, kMT = C::kMT;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;     // fragment row / column pair of this lane
    unsigned char* ws = smem + warp * C::kWarpBytes;
    const uint32_t ws_addr = smem_addr(ws);
    unsigned char* ctl = ws + C::kStages * C::kStageBytes;
    const uint32_t ctl_addr = ws_addr + C::kStages * C::kStageBytes;
    uint32_t* masks = reinterpret_cast<uint32_t*>(ctl + 8 * C::kStages);
    Unit* queue = reinterpret_cast<Unit*>(ctl + C::kQueueOff);
    auto bar = [&](int i) { return ctl_addr + 8 * i; };

    pdl_trigger();
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(bar(i), 1);
        fence_barrier_init();
    }
    __syncwarp();
    pdl_wait();

    const uint64_t kv_pol = l2_policy_evict_first();       // streamed, as in the tensor-core decode
    const unsigned long long total_warps = (unsigned long long)gridDim.x * C::kWarps;
    unsigned long long static_next = (unsigned long long)blockIdx.x * C::kWarps + warp;
    constexpr int kHeadBytes = kv4_head_bytes(BS, D), kBlocks = kTok / BS;   // of one block; blocks per stage
    // byte offsets inside a stage's K (or V) part of each 16-token tile's codes, scales and zeros:
    // tile mt is tile (16 mt % BS) / 16 of block 16 mt / BS
    constexpr int kZeroOff = BS * G * 2;                   // from a block's scales to its zeros
    auto tile_codes = [](int mt) { return (16 * mt / BS) * kHeadBytes + (16 * mt % BS) * (D / 2); };
    auto tile_scales = [](int mt) { return (16 * mt / BS) * kHeadBytes + BS * (D / 2) + (16 * mt % BS) * (G * 2); };

    // ---- issue side: claims units, fills stages
    bool claiming = true, i_have = false, first_claim = true;
    Unit iu{};
    int i_stage = 0, i_nst = 0, i_first = 0;   // i_first: with a window, its first token (window_span's numbering)
    WindowSpan i_span{};
    unsigned g_issue = 0, q_tail = 0;
    uint4 qn[G];                          // the query of the oldest claimed unit that has not started
    int qn_for = -1;
    auto load_qn = [&](int s, int h0, int nh) {
        // head r, values 32 g + 8 c .. + 7 of every group; zero past the unit's heads
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.q) +
                                                        ((size_t)s * p.Hq + h0 + (r < nh ? r : 0)) * D * 2);
#pragma unroll
        for (int g = 0; g < G; ++g) qn[g] = r < nh ? __ldg(q + 4 * g + c) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto claim = [&](Unit& x) -> bool {
        for (;;) {
            unsigned long long v = 0;
            if (first_claim) {
                v = (unsigned long long)warp * gridDim.x + blockIdx.x;   // consecutive units on different SMs
                first_claim = false;
            } else if (lane == 0) {
                v = p.sched != nullptr ? atomicAdd(reinterpret_cast<unsigned long long*>(p.sched), 1ull) + total_warps
                                       : static_next;
            }
            v = __shfl_sync(0xffffffffu, v, 0);
            static_next += total_warps;
            if (v >= total_units) return false;
            if (!unit_of<WIN>(p, v, nsets, region_a, x)) continue;
            if (x.t1 <= x.t0) {
                // a sequence with no tokens: its output is zero
                for (int i = lane; i < x.nh * D; i += 32)
                    store_elem<BF16>(p.out, ((size_t)x.s * p.Hq + x.h0) * D + i, 0.f);
                continue;
            }
            return true;
        }
    };
    int tab = 0, tab_next = 0, tab_chunk = 0, tab_blocks = 0;
    auto load_chunk = [&](int chunk) -> int {
        const int rb = 32 * chunk + lane;
        if (rb >= tab_blocks) return 0;
        int lb = iu.t0 / BS + rb;
        if constexpr (WIN) lb = span_token(i_span, lb * BS) / BS;
        return __ldg(p.block_tables + (size_t)iu.s * p.MB + lb);
    };
    auto issue_one = [&]() -> bool {
        while (!i_have || i_stage == i_nst) {
            if (!claiming) return false;
            if (!claim(iu)) {
                claiming = false;
                return false;
            }
            if constexpr (WIN) {
                const int n = min(max(__ldg(p.context_lens + iu.s), 0), p.max_ctx);
                i_span = window_span(n - p.window, p.sinks, BS);
                i_first = n - p.window - i_span.gap;
            }
            if (lane == 0) {
                int4* e = reinterpret_cast<int4*>(queue + q_tail % C::kQueue);
                e[0] = make_int4(iu.s, iu.kvh, iu.h0, iu.nh);
                e[1] = make_int4(iu.part, iu.t0, iu.t1, iu.np);
            }
            if (qn_for < 0) {
                load_qn(iu.s, iu.h0, iu.nh);
                qn_for = (int)q_tail;
            }
            ++q_tail;
            i_have = true;
            i_stage = 0;
            i_nst = (iu.t1 - iu.t0 + kTok - 1) / kTok;
            tab_blocks = (iu.t1 - iu.t0 + BS - 1) / BS;
            tab_chunk = 0;
            tab = load_chunk(0);
            tab_next = load_chunk(1);
        }
        const int slot = g_issue % C::kStages;
        const int rs = i_stage * kTok, ts = iu.t0 + rs;
        const int tn = min(kTok, iu.t1 - ts);
        if (rs / (32 * BS) != tab_chunk) {                     // the stage's blocks start a new chunk
            ++tab_chunk;
            tab = tab_next;
            tab_next = load_chunk(tab_chunk + 1);
        }
        // lane 2 b + v copies block b of the stage, K (v 0) or V; a block with a bad id is left out
        const int b = lane >> 1, isv = lane & 1;
        const int pb = __shfl_sync(0xffffffffu, tab, (rs / BS + b) & 31);
        const bool here = b < kBlocks && b * BS < tn;
        const bool live = here && pb >= 0 && pb < p.NB;
        if (here && !live) report(p.err, PKV_DEVERR_BLOCK_ID);
        const uint32_t lives = __ballot_sync(0xffffffffu, live);
        // in the unit's numbering the unseen tokens are those from the sinks to the window's start
        const bool whole = lives == (1u << (2 * kBlocks)) - 1u && tn == kTok &&
                           (!WIN || p.sinks >= i_first || ts >= i_first || ts + kTok <= p.sinks);
        if (lane == 0) {
            // per token: inside the unit, seen, and in a loaded block
#pragma unroll
            for (int k = 0; k < C::kMasks; ++k) {
                uint32_t m = 0xffffffffu;
                if (!whole) {
                    m = bits_below(tn - 32 * k);
                    if constexpr (BS == 32) {
                        if (!((lives >> (2 * k)) & 1u)) m = 0;
                    } else {
                        if (!((lives >> (4 * k)) & 1u)) m &= 0xffff0000u;
                        if (!((lives >> (4 * k + 2)) & 1u)) m &= 0x0000ffffu;
                    }
                    if constexpr (WIN) m &= ~bits_between(ts + 32 * k, p.sinks, i_first);
                }
                masks[slot * C::kMasks + k] = m;
            }
            mbar_arrive_expect_tx(bar(slot), __popc(lives) * kHeadBytes);
        }
        __syncwarp();
        if (live)
            bulk_load_hint(ws_addr + slot * C::kStageBytes + isv * C::kPartBytes + b * kHeadBytes,
                           static_cast<const unsigned char*>(isv ? p.vc : p.kc) +
                               ((size_t)pb * p.Hkv + iu.kvh) * kHeadBytes,
                           kHeadBytes, bar(slot), kv_pol);
        ++g_issue;
        ++i_stage;
        return true;
    };

    // ---- consume side
    unsigned g_cons = 0, q_head = 0;
    bool have_unit = false, need_q = false, bail = false;
    Unit cu{};
    int c_stage = 0, c_nst = 0;
    uint32_t qf[G][4];                    // (d0, d0 + 4) * 4, (d0 + 1, d0 + 5) / 4, ... of head r; d0 = 32 g + 8 c
    uint32_t qs = 0;                      // the group sums' fragment of the zeros' product
    float o[2 * G][4], zo[4];             // V's codes' part; zeros' part: group r, heads 2c, 2c + 1
    float m_ref[2];                       // reference maximum of heads 2c, 2c + 1
    // byte g: group g's values are accumulated times 2^-j, j <= 16; bit 30: some j is not 0 (in shared memory: one
    // register more is a spill, 2% of the launch)
    uint32_t* shift_word = reinterpret_cast<uint32_t*>(ctl + C::kShiftOff);
    // Logits are kept in units of code * |q| sums: x = xs * x', xs >= 0 (the query carries the sign)
    // and the query is taken times 2^e, its largest finite value in the unit then in [512, 1024): it has fp16's
    // precision whatever its size, and a sum of 32 stays below 2^15
    const float xs_base = 4194304.f * fabsf(p.logit_scale_log2);
    const float q_sign = p.logit_scale_log2 < 0.f ? -1.f : 1.f;
    float xs = 0.f, slack = 0.f;

    for (int i = 0; i < C::kStages; ++i)
        if (!issue_one()) break;

    for (;;) {
        if (!have_unit) {
            if (q_head == q_tail) break;
            __syncwarp();
            const int4* e = reinterpret_cast<const int4*>(queue + q_head % C::kQueue);
            const int4 a = e[0], b2 = e[1];
            cu.s = a.x; cu.kvh = a.y; cu.h0 = a.z; cu.nh = a.w;
            cu.part = b2.x; cu.t0 = b2.y; cu.t1 = b2.z; cu.np = b2.w;
            ++q_head;
            c_stage = 0;
            c_nst = (cu.t1 - cu.t0 + kTok - 1) / kTok;
            have_unit = need_q = true;
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
            zo[0] = zo[1] = zo[2] = zo[3] = 0.f;
            m_ref[0] = m_ref[1] = -CUDART_INF_F;
            if (lane == 0) *shift_word = 0;
            __syncwarp();
        }
        const int slot = g_cons % C::kStages;
        const uint32_t parity = (g_cons / C::kStages) & 1u;
        if (!mbar_try_wait(bar(slot), parity)) {
            const long long t_start = clock64();
            while (!mbar_try_wait(bar(slot), parity)) {
                if (clock64() - t_start > kWaitLimitCycles) {
                    report(p.err, PKV_DEVERR_TIMEOUT);
                    bail = true;
                    break;
                }
            }
        }
        if (__any_sync(0xffffffffu, bail)) break;
        if (need_q) {
            need_q = false;
            float hi[G], lo[G];
            // largest exponent of a finite value, as bf16's bits
            uint32_t top = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t w[4] = {qn[g].x, qn[g].y, qn[g].z, qn[g].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a = w[k] & 0x7f800000u, b = (w[k] << 16) & 0x7f800000u;
                    if (a != 0x7f800000u) top = max(top, a);
                    if (b != 0x7f800000u) top = max(top, b);
                }
            }
            top = __reduce_max_sync(0xffffffffu, top) >> 23;
            const int e = top > 0 ? min(max(136 - (int)top, -90), 100) : 0;
            xs = xs_base * pow2(-e);
            slack = xs > 0.f ? 2.f / xs : CUDART_INF_F;
            const float q_by = q_sign * pow2(e);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t w[4] = {qn[g].x, qn[g].y, qn[g].z, qn[g].w};
                float f[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = __uint_as_float(w[k] << 16);
                    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float by = q_by * ((k & 1) ? 0.25f : 4.f);
                    qf[g][k] = pack2<true>(f[k] * by, f[k + 4] * by);
                }
                float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum *= q_by;
                hi[g] = __half2float(__float2half_rn(sum));
                lo[g] = sum - hi[g];
            }
            // k = 2c, 2c + 1 of the zeros' product: the groups' high parts, then their low parts
            if constexpr (G == 4)
                qs = c == 0 ? pack2<true>(hi[0], hi[1]) : c == 1 ? pack2<true>(hi[2], hi[3])
                   : c == 2 ? pack2<true>(lo[0], lo[1]) : pack2<true>(lo[2], lo[3]);
            else
                qs = c == 0 ? pack2<true>(hi[0], hi[1]) : c == 1 ? pack2<true>(lo[0], lo[1]) : 0u;
            qn_for = -1;
            if (q_tail > q_head) {
                const int4 a = reinterpret_cast<const int4*>(queue + q_head % C::kQueue)[0];
                load_qn(a.x, a.z, a.w);
                qn_for = (int)q_head;
            }
        }
        const unsigned char* kp = ws + slot * C::kStageBytes;
        const unsigned char* vp = kp + C::kPartBytes;
        uint32_t vm[C::kMasks];
        bool full = true;
#pragma unroll
        for (int k = 0; k < C::kMasks; ++k) {
            vm[k] = masks[slot * C::kMasks + k];
            full = full && vm[k] == 0xffffffffu;
        }

        // ---- logits of the stage: rows r and r + 8 of each 16-token tile
        float x[kMT][4];
        float cmax0 = -CUDART_INF_F, cmax1 = -CUDART_INF_F;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            const unsigned char* codes = kp + tile_codes(mt);
            const unsigned char* scales = kp + tile_scales(mt);
            uint32_t ka[G], kb[G], sa[G / 2], sb[G / 2];
            lds_words<G>(codes + r * (D / 2) + c * (D / 8), ka);
            lds_words<G>(codes + (r + 8) * (D / 2) + c * (D / 8), kb);
#pragma unroll
            for (int j = 0; j < G / 2; ++j) {
                sa[j] = reinterpret_cast<const uint32_t*>(scales + r * G * 2)[j];
                sb[j] = reinterpret_cast<const uint32_t*>(scales + (r + 8) * G * 2)[j];
            }
            const int zw = G == 4 ? 4 * (c & 1) : 0;
            float z[4] = {0.f, 0.f, 0.f, 0.f};
            mma1688(z, *reinterpret_cast<const uint32_t*>(scales + kZeroOff + r * G * 2 + zw),
                    *reinterpret_cast<const uint32_t*>(scales + kZeroOff + (r + 8) * G * 2 + zw), qs);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[mt][k] = z[k] * 2.384185791015625e-7f;     // 2^-22
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float a[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816<true>(a, ka[g] & kLo, kb[g] & kLo, ka[g] & kHi, kb[g] & kHi, qf[g][0], qf[g][1]);
                const uint32_t ua = ka[g] >> 8, ub = kb[g] >> 8;
                mma16816<true>(a, ua & kLo, ub & kLo, ua & kHi, ub & kHi, qf[g][2], qf[g][3]);
                const __half2 ha = *reinterpret_cast<const __half2*>(&sa[g / 2]);
                const __half2 hb = *reinterpret_cast<const __half2*>(&sb[g / 2]);
                const float fa = (g & 1) ? __high2float(ha) : __low2float(ha);
                const float fb = (g & 1) ? __high2float(hb) : __low2float(hb);
                x[mt][0] = fmaf(fa, a[0], x[mt][0]);
                x[mt][1] = fmaf(fa, a[1], x[mt][1]);
                x[mt][2] = fmaf(fb, a[2], x[mt][2]);
                x[mt][3] = fmaf(fb, a[3], x[mt][3]);
            }
        }
        if (!full) {
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
                const uint32_t v = vm[mt / 2] >> (16 * (mt & 1) + r);
                if (!(v & 1u)) x[mt][0] = x[mt][1] = -CUDART_INF_F;
                if (!(v & 0x100u)) x[mt][2] = x[mt][3] = -CUDART_INF_F;
            }
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            cmax0 = fmaxf(cmax0, fmaxf(x[mt][0], x[mt][2]));
            cmax1 = fmaxf(cmax1, fmaxf(x[mt][1], x[mt][3]));
        }

        // ---- online softmax: the reference maximum moves only when a logit exceeds it by a
        // factor of 4 in weight, so that most stages need no maximum over the warp
        if (__any_sync(0xffffffffu, cmax0 > m_ref[0] + slack || cmax1 > m_ref[1] + slack ||
                                        m_ref[0] == -CUDART_INF_F || m_ref[1] == -CUDART_INF_F)) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                cmax0 = fmaxf(cmax0, __shfl_xor_sync(0xffffffffu, cmax0, off));
                cmax1 = fmaxf(cmax1, __shfl_xor_sync(0xffffffffu, cmax1, off));
            }
            const float mn0 = fmaxf(m_ref[0], cmax0), mn1 = fmaxf(m_ref[1], cmax1);
            const float al0 = m_ref[0] == -CUDART_INF_F ? 0.f : fast_exp2((m_ref[0] - mn0) * xs);
            const float al1 = m_ref[1] == -CUDART_INF_F ? 0.f : fast_exp2((m_ref[1] - mn1) * xs);
            zo[0] *= al0;
            zo[1] *= al1;
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) {
                o[t][0] *= al0;
                o[t][1] *= al1;
                o[t][2] *= al0;
                o[t][3] *= al1;
            }
            m_ref[0] = mn0;
            m_ref[1] = mn1;
        }
        const float mu0 = m_ref[0] == -CUDART_INF_F ? 0.f : kWeightLog2 - m_ref[0] * xs;
        const float mu1 = m_ref[1] == -CUDART_INF_F ? 0.f : kWeightLog2 - m_ref[1] * xs;

        // V's scales of tokens 2 u and 2 u + 1 (u: the lane), in fp16; one of 2 or more has bit 14 set
        uint32_t sv[G], large = 0;
        lds_words<G>(vp + lane % (kTok / 2) / (BS / 2) * kHeadBytes + BS * (D / 2) + lane % (BS / 2) * (4 * G), sv);
#pragma unroll
        for (int g = 0; g < G; ++g) large |= sv[g];
        const bool shifted = __any_sync(0xffffffffu, (large | *shift_word) & 0x40004000u);
        uint32_t shifts = 0;
        if (shifted) {
            shifts = *shift_word;
            // each group's j for the largest scale of its present tokens so far, 2^j <= s < 2^(j + 1)
            const int u = lane % (kTok / 2);
            const uint32_t here = (u < 16 ? vm[0] : vm[C::kMasks - 1]) >> (2 * (u % 16));
            uint32_t next = 0;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint32_t lo = here & 1u ? sv[g] & 0x7fffu : 0u, hi = here & 2u ? (sv[g] >> 16) & 0x7fffu : 0u;
                const int e = (int)(__reduce_max_sync(0xffffffffu, max(lo, hi)) >> 10) - 15;
                const int was = (shifts >> (8 * g)) & 0x1fu, j = max(was, e);
                if (j > was) {
                    const float down = pow2(was - j);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        o[2 * g][k] *= down;
                        o[2 * g + 1][k] *= down;
                    }
                }
                next |= (uint32_t)j << (8 * g);
            }
            shifts = next;
            __syncwarp();
            if (lane == 0) *shift_word = next != 0 ? next | 0x40000000u : 0u;
            __syncwarp();
        }

        // ---- O^T += V^T . P^T, tile by tile
        auto product = [&](auto whole, auto shift) {
            constexpr bool kWhole = decltype(whole)::value, kShift = decltype(shift)::value;
#pragma unroll
            for (int kt = 0; kt < kMT; ++kt) {
                const float p0 = weight<kWhole>(x[kt][0], xs, mu0), p1 = weight<kWhole>(x[kt][1], xs, mu1);
                const float p2 = weight<kWhole>(x[kt][2], xs, mu0), p3 = weight<kWhole>(x[kt][3], xs, mu1);
                // tokens 2c, 2c + 1 and 2c + 8, 2c + 9 of head r
                const uint32_t pb0 = movmatrix_t(pack2<true>(p0, p1)), pb1 = movmatrix_t(pack2<true>(p2, p3));
                const unsigned char* codes = vp + tile_codes(kt);
                const unsigned char* scales = vp + tile_scales(kt);
                uint32_t w0[G], w1[G], s0[G], s1[G];
                lds_words<G>(codes + lane * (4 * G), w0);
                lds_words<G>(codes + (32 + lane) * (4 * G), w1);
                lds_words<G>(scales + c * (4 * G), s0);
                lds_words<G>(scales + (c + 4) * (4 * G), s1);
                // rows of the zeros' product: group r's zeros, and in row G ones, whose sum of weights is l
                uint32_t z0 = r == G ? 0x3c003c00u : 0u, z1 = z0;
                if (r < G) {
                    z0 = *reinterpret_cast<const uint32_t*>(scales + kZeroOff + c * (4 * G) + 4 * r);
                    z1 = *reinterpret_cast<const uint32_t*>(scales + kZeroOff + (c + 4) * (4 * G) + 4 * r);
                }
                if constexpr (!kWhole) {             // absent tokens: their scales and zeros may be NaN
                    const uint32_t v = vm[kt / 2] >> (16 * (kt & 1) + 2 * c);
                    const uint32_t mlo = (v & 1u ? 0x0000ffffu : 0u) | (v & 2u ? 0xffff0000u : 0u);
                    const uint32_t mhi = (v & 0x100u ? 0x0000ffffu : 0u) | (v & 0x200u ? 0xffff0000u : 0u);
                    z0 &= mlo;
                    z1 &= mhi;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        s0[g] &= mlo;
                        s1[g] &= mhi;
                    }
                }
                mma16816<true>(zo, z0, 0u, z1, 0u, pb0, pb1);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    uint32_t q0 = pb0, q1 = pb1;
                    if constexpr (kShift) {
                        const float down = pow2(-(int)((shifts >> (8 * g)) & 0x1fu));
                        q0 = hmul2u(q0, pack2<true>(down, down));
                        q1 = hmul2u(q1, pack2<true>(down, down));
                    }
                    const uint32_t b0 = hmul2u(q0, s0[g]), b1 = hmul2u(q1, s1[g]);
                    mma16816<true>(o[2 * g], w0[g] & kLo, w0[g] & kHi, w1[g] & kLo, w1[g] & kHi, b0, b1);
                    // the upper byte's two codes as one number n + 16 n', and n alone: one instruction
                    // less than taking them apart; the rows are parted when the unit is finished
                    const uint32_t u0 = __byte_perm(w0[g], 0u, 0x4341u), u1 = __byte_perm(w1[g], 0u, 0x4341u);
                    mma16816<true>(o[2 * g + 1], u0 & kLo, u0, u1 & kLo, u1, b0, b1);
                }
            }
        };
        if (shifted) product(std::false_type{}, std::true_type{});
        else if (full) product(std::true_type{}, std::false_type{});
        else product(std::false_type{}, std::false_type{});

        // the slot is free again: let the issue side refill it
        __syncwarp();
        fence_proxy_async();
        ++g_cons;
        ++c_stage;
        issue_one();

        if (c_stage == c_nst) {
            // ---- finish the unit
            const uint32_t shifts = *shift_word;
            const uint64_t keep = l2_policy_evict_last();   // partials: held in L2 until the merge reads them
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = 2 * c + j;
                const bool wr = h < cu.nh;
                const size_t row = (size_t)cu.s * p.Hq + cu.h0 + h, u = row * p.Pmax + cu.part;
                const float l = __shfl_sync(0xffffffffu, zo[j], 4 * G + c);
                const float f = cu.np > 1 ? kWeightInv : (l > 0.f ? p.out_scale / l : 0.f);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float zg = __shfl_sync(0xffffffffu, zo[j], 4 * g + c);
                    const int up = (shifts >> (8 * g)) & 0x1fu;
                    const float c0 = pow2(24 + up), c1 = pow2(20 + up);
                    // values 32 g + 4 r .. + 3 of head h; the last pair's second row holds both
                    const float v[4] = {fmaf(o[2 * g][j], c0, zg) * f, fmaf(o[2 * g][j + 2], c1, zg) * f,
                                        fmaf(o[2 * g + 1][j], c0, zg) * f,
                                        fmaf(o[2 * g + 1][j + 2] - o[2 * g + 1][j], c1, zg) * f};
                    if (!wr) continue;
                    if (cu.np == 1) {
                        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * D + 32 * g + 4 * r) =
                            make_uint2(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]));
                    } else {
                        asm volatile("st.global.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(
                                         p.part_acc + u * D + 32 * g + 4 * r),
                                     "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "l"(keep)
                                     : "memory");
                    }
                }
                if (wr && cu.np > 1 && r == 0) {
                    st_l2_hint(p.part_ml + 2 * u, m_ref[j] == -CUDART_INF_F ? m_ref[j] : m_ref[j] * xs, keep);
                    st_l2_hint(p.part_ml + 2 * u + 1, l * kWeightInv, keep);
                }
            }
            have_unit = false;
        }
    }

    wait_stages(bar, C::kStages, g_cons, g_issue, kWaitLimitCycles);   // none, unless it gave up

    if (p.local) merge_set<D, BF16>(p, nsets, C::kWarps);

    // ---- leave the scheduling counters at zero for the next launch
    if (p.sched != nullptr && lane == 0) {
        unsigned long long* ctr = reinterpret_cast<unsigned long long*>(p.sched);
        __threadfence();
        const unsigned long long done = atomicAdd(ctr + 1, 1ull);
        if (done == total_warps - 1) {
            atomicExch(ctr, 0ull);
            atomicExch(ctr + 1, 0ull);
        }
    }
}

template <int D, int BS, bool WIN>
cudaError_t launch_kv4_one(DecodeParams& p, int num_sms, cudaStream_t st) {
    using C = KCfg<D>;
    auto kern = decode_kv4_kernel<D, BS, WIN>;
    static SmemOptIn optin;
    const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(kern), C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const int nsets = (p.g + kHeadsPerUnit - 1) / kHeadsPerUnit;
    const unsigned long long per_part = (unsigned long long)p.S * p.Hkv * nsets;
    const unsigned long long region_a = (unsigned long long)(max_visible(p) / p.P) * per_part;   // full partitions
    const unsigned long long units = region_a + (unsigned long long)chunk_slots(p.P, p.Q, p.hold) * per_part;
    // a small launch puts its units on as many SMs as it has
    int grid = (int)(units < (unsigned long long)num_sms ? units : (unsigned long long)num_sms);
    if ((p.local = merges_itself(p, per_part, units, C::kWarps, num_sms))) {
        grid = (int)per_part;
        p.sched = nullptr;
    }
    return launch_pdl(kern, dim3(grid < 1 ? 1 : grid), dim3(C::kWarps * 32), C::kSmemBytes, st, p, units, region_a,
                      nsets);
}

template <int D, bool WIN>
cudaError_t launch_kv4_bs(DecodeParams& p, int num_sms, cudaStream_t st) {
    return p.bs == 16 ? launch_kv4_one<D, 16, WIN>(p, num_sms, st) : launch_kv4_one<D, 32, WIN>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_decode_kv4(DecodeParams& p, int num_sms, cudaStream_t st) {
    if (p.S == 0) return cudaSuccess;
    if (p.window > 0) return p.d == 64 ? launch_kv4_bs<64, true>(p, num_sms, st) : launch_kv4_bs<128, true>(p, num_sms, st);
    return p.d == 64 ? launch_kv4_bs<64, false>(p, num_sms, st) : launch_kv4_bs<128, false>(p, num_sms, st);
}

}  // namespace pkv
