// paged_attention_decode_window over an fp32 cache (sm_103a).
//
// "LLM推論の基礎とvLLMの内部", section 1: decode is bound by memory bandwidth;
// section 2: one read of a K/V head serves its query heads.  No matrix
// instruction takes fp32 operands at full precision, so the products are
// fused multiply-adds: 64 per lane and token for 8 heads of 128 values, half
// of what the issue slots allow at HBM's pace (a 16-token tile is 16 KB and
// ~1,500 warp instructions, and HBM delivers one per SM every ~700 cycles,
// 2,800 slots).
//
// Work units, their order, the numbering of the visible tokens and the ring
// of stages per warp are the tensor-core decode's (pkv_units.cuh); a stage is
// 16 tokens of K and V of one head, one tensor copy each (rows of 4 d bytes,
// no swizzle: a warp reads whole rows).  A lane holds four values of d: all
// 32 lanes a row of 128, the two halves of the warp two rows of 64.
//
// Logits: each lane's partial sums of 8 tokens x 8 heads are added over the
// lanes of a row by halving (a lane keeps half of what it holds and gives
// away the other half): 62 shuffles for 64 sums over 32 lanes.  A lane ends
// with the logits of one token and two (d 64: four) heads.  The weights go
// through 512 bytes of shared memory and come back as broadcasts.  The
// reference maximum is raised only when a logit exceeds it by 8 (a factor of
// 256 in weight); every sum is fp32.
//
// 32 sequences of 500..16,384 with a window of 1,024 (28 / 4 heads of 128,
// 135 MB): 46 us with the merge, 2.9 TB/s: its 1,100 partitions of 128 tokens
// go over 912 workers, so most of the launch is one or two units' pace (41% of
// HBM's rate, 46% of the issue slots in the kernel).  The CUDA-core kernel,
// which reads 4-byte elements and reduces each logit on its own, takes 124 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <mutex>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_tc_common.cuh"
#include "pkv_units.cuh"

namespace pkv {
namespace {

using namespace tc;

constexpr int kTok = 16, kStages = 2;                  // tokens per stage, stages per warp
constexpr long long kWaitLimitCycles = 4000000000LL;   // ~2 s: a stage that never lands

template <int D>
struct FCfg {
    static constexpr int kRowBytes = 4 * D, kPartBytes = kTok * kRowBytes, kStageBytes = 2 * kPartBytes;
    static constexpr int kWarps = D == 128 ? 6 : 8;      // 6 rings of rows of 128 fill shared memory
    // per worker: stages, a batch's weights [token][head], 8 head factors, barriers, masks, the unit queue
    static constexpr int kWeightOff = kStages * kStageBytes;
    static constexpr int kFactorOff = kWeightOff + kTok * kHeadsPerUnit * 4;
    static constexpr int kBarOff = kFactorOff + kHeadsPerUnit * 4;
    static constexpr int kMaskOff = kBarOff + 8 * kStages;
    static constexpr int kQueueOff = (kMaskOff + 4 * kStages + 15) / 16 * 16;
    static constexpr int kWarpBytes = (kQueueOff + 32 * kStages + 127) / 128 * 128;   // tensor copies want 128
    static constexpr int kSmemBytes = kWarps * kWarpBytes + 128;
    static_assert(kSmemBytes <= 232448, "shared memory per CTA");
};

// One halving step over the lane distance `mask`: of v[0 .. 2 N) a lane keeps
// one half (the upper where `upper`), summed with its partner's, in v[0 .. N).
template <int N>
__device__ __forceinline__ void halve_sum(float* v, int mask, bool upper) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float send = upper ? v[i] : v[i + N], keep = upper ? v[i + N] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
    }
}

template <int D, typename QF>
__global__ void __launch_bounds__(FCfg<D>::kWarps * 32, 1)
    decode_f32_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, unsigned long long total_units,
                      unsigned long long region_a, int nsets) {
    using C = FCfg<D>;
    constexpr int kRowLanes = D / 4;                       // lanes per row
    constexpr int kRows = 32 / kRowLanes;                  // rows a warp takes at once
    constexpr int kBatches = kTok / (8 * kRows);           // of 8 tokens per lane
    constexpr int kOwn = kRowLanes == 32 ? 2 : 4;          // heads a lane holds logits of
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t raw = smem_addr(smem_raw), base_addr = (raw + 127u) & ~127u;
    unsigned char* ws = smem_raw + (base_addr - raw) + warp * C::kWarpBytes;
    const uint32_t ws_addr = base_addr + warp * C::kWarpBytes;
    float* weights = reinterpret_cast<float*>(ws + C::kWeightOff);
    float* factors = reinterpret_cast<float*>(ws + C::kFactorOff);
    uint32_t* masks = reinterpret_cast<uint32_t*>(ws + C::kMaskOff);
    Unit* queue = reinterpret_cast<Unit*>(ws + C::kQueueOff);
    auto bar = [&](int i) { return ws_addr + C::kBarOff + 8 * i; };

    pdl_trigger();
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(bar(i), 1);
        fence_barrier_init();
    }
    __syncwarp();
    pdl_wait();

    const uint64_t kv_pol = l2_policy_evict_first();       // streamed, as in the tensor-core decode
    const unsigned long long total_warps = (unsigned long long)gridDim.x * C::kWarps;
    unsigned long long static_next = (unsigned long long)blockIdx.x * C::kWarps + warp;

    // ---- issue side: claims units, fills stages
    bool claiming = true, i_have = false, first_claim = true;
    Unit iu{};
    int i_stage = 0, i_nst = 0, i_first = 0;               // i_first: the window's first token (window_span's numbering)
    WindowSpan i_span{};
    unsigned g_issue = 0, q_tail = 0;
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
            if (!unit_of<true>(p, v, nsets, region_a, x)) continue;
            if (x.t1 <= x.t0) {
                // a sequence with no tokens: its output is zero
                for (int i = lane; i < x.nh * D; i += 32)
                    store_elem<QF>(p.out, ((size_t)x.s * p.Hq + x.h0) * D + i, 0.f);
                continue;
            }
            return true;
        }
    };
    int tab = 0, tab_next = 0, tab_chunk = 0, tab_blocks = 0;
    auto load_chunk = [&](int chunk) -> int {
        const int rb = 32 * chunk + lane;
        if (rb >= tab_blocks) return 0;
        const int t = span_token(i_span, iu.t0 + rb * p.bs);
        return __ldg(p.block_tables + (size_t)iu.s * p.MB + t / p.bs);
    };
    auto issue_one = [&]() -> bool {
        while (!i_have || i_stage == i_nst) {
            if (!claiming) return false;
            if (!claim(iu)) {
                claiming = false;
                return false;
            }
            const int n = min(max(__ldg(p.context_lens + iu.s), 0), p.max_ctx);
            i_span = window_span(n - p.window, p.sinks, p.bs);
            i_first = n - p.window - i_span.gap;
            if (lane == 0) {
                int4* e = reinterpret_cast<int4*>(queue + q_tail % kStages);
                e[0] = make_int4(iu.s, iu.kvh, iu.h0, iu.nh);
                e[1] = make_int4(iu.part, iu.t0, iu.t1, iu.np);
            }
            ++q_tail;
            i_have = true;
            i_stage = 0;
            i_nst = (iu.t1 - iu.t0 + kTok - 1) / kTok;
            tab_blocks = (iu.t1 - iu.t0 + p.bs - 1) / p.bs;
            tab_chunk = 0;
            tab = load_chunk(0);
            tab_next = load_chunk(1);
        }
        const int slot = g_issue % kStages, rs = i_stage * kTok, ts = iu.t0 + rs;
        const int blk = rs / p.bs;
        if (blk / 32 != tab_chunk) {                           // the stage's block starts a new chunk
            ++tab_chunk;
            tab = tab_next;
            tab_next = load_chunk(tab_chunk + 1);
        }
        const int pb = __shfl_sync(0xffffffffu, tab, blk & 31);
        const bool live = pb >= 0 && pb < p.NB;
        if (lane == 0) {
            if (!live) report(p.err, PKV_DEVERR_BLOCK_ID);
            // per token: inside the unit, seen, and in a valid block
            masks[slot] = live ? bits_below(min(kTok, iu.t1 - ts)) & ~bits_between(ts, p.sinks, i_first) : 0u;
            mbar_arrive_expect_tx(bar(slot), live ? C::kStageBytes : 0);
            if (live) {
                const uint32_t dst = ws_addr + slot * C::kStageBytes;
                const int row = pb * p.bs + ts % p.bs;
                tensor_load_2d_hint(dst, &kmap, iu.kvh * D, row, bar(slot), kv_pol);
                tensor_load_2d_hint(dst + C::kPartBytes, &vmap, iu.kvh * D, row, bar(slot), kv_pol);
            }
        }
        __syncwarp();
        ++g_issue;
        ++i_stage;
        return true;
    };

    // ---- consume side
    unsigned g_cons = 0, q_head = 0;
    bool have_unit = false, bail = false;
    Unit cu{};
    int c_stage = 0, c_nst = 0;
    const int rl = lane % kRowLanes, half = lane / kRowLanes;   // lane within its row, the row among kRows
    // the token (of a batch's 8 per row) and the first head this lane ends a halving with
    const int my_tok = kRowLanes == 32 ? lane >> 2 : rl >> 1, my_head = kOwn * (lane & (kRowLanes == 32 ? 3 : 1));
    float q[kHeadsPerUnit][4], acc[kHeadsPerUnit][4];
    float m_ref[kOwn], l_run[kOwn];
    const float scl = p.logit_scale_log2;

    for (int i = 0; i < kStages; ++i)
        if (!issue_one()) break;

    for (;;) {
        if (!have_unit) {
            if (q_head == q_tail) break;
            __syncwarp();
            const int4* e = reinterpret_cast<const int4*>(queue + q_head % kStages);
            const int4 a = e[0], b2 = e[1];
            cu.s = a.x; cu.kvh = a.y; cu.h0 = a.z; cu.nh = a.w;
            cu.part = b2.x; cu.t0 = b2.y; cu.t1 = b2.z; cu.np = b2.w;
            ++q_head;
            c_stage = 0;
            c_nst = (cu.t1 - cu.t0 + kTok - 1) / kTok;
            have_unit = true;
#pragma unroll
            for (int h = 0; h < kHeadsPerUnit; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[h][k] = 0.f;
                    q[h][k] = h < cu.nh ? load_elem<QF>(p.q, ((size_t)cu.s * p.Hq + cu.h0 + h) * D + 4 * rl + k) : 0.f;
                }
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                m_ref[k] = -CUDART_INF_F;
                l_run[k] = 0.f;
            }
        }
        const int slot = g_cons % kStages;
        const uint32_t parity = (g_cons / kStages) & 1u;
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
        const unsigned char* kp = ws + slot * C::kStageBytes + rl * 16;
        const unsigned char* vp = kp + C::kPartBytes;
        const uint32_t mask = masks[slot];

        // batches of 8 tokens per row: batch b's token i of this lane's row is kRows (8 b + i) + half.  One
        // copy of the code: a stage's, unrolled, is 24 KB of instructions
#pragma unroll 1
        for (int b = 0; b < kBatches; ++b, kp += 8 * kRows * C::kRowBytes, vp += 8 * kRows * C::kRowBytes) {
            const uint32_t bm = mask >> (8 * kRows * b);
            // ---- logits (log2 units)
            float s[8 * kHeadsPerUnit];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 k = *reinterpret_cast<const float4*>(kp + (kRows * i + half) * C::kRowBytes);
#pragma unroll
                for (int h = 0; h < kHeadsPerUnit; ++h)
                    s[8 * i + h] = fmaf(q[h][0], k.x, fmaf(q[h][1], k.y, fmaf(q[h][2], k.z, q[h][3] * k.w)));
            }
            if constexpr (kRowLanes == 32) {
                halve_sum<32>(s, 16, lane & 16);
                halve_sum<16>(s, 8, lane & 8);
                halve_sum<8>(s, 4, lane & 4);
                halve_sum<4>(s, 2, lane & 2);
                halve_sum<2>(s, 1, lane & 1);
            } else {
                halve_sum<32>(s, 8, lane & 8);
                halve_sum<16>(s, 4, lane & 4);
                halve_sum<8>(s, 2, lane & 2);
                halve_sum<4>(s, 1, lane & 1);
            }
            const bool seen = (bm >> (kRows * my_tok + half)) & 1u;
            bool above = false;
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                s[k] = seen ? s[k] * scl : -CUDART_INF_F;
                above = above || s[k] > m_ref[k] + 8.f;
            }
            if (__any_sync(0xffffffffu, above)) {
                // raise the reference maxima to the batch's; the factors of the 8 heads go to every lane
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    float m = fmaxf(m_ref[k], s[k]);
#pragma unroll
                    for (int off = kOwn == 2 ? 4 : 2; off < 32; off <<= 1)
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                    const float f = m_ref[k] == -CUDART_INF_F ? 0.f : fast_exp2(m_ref[k] - m);
                    l_run[k] *= f;
                    m_ref[k] = m;
                    if (lane < kHeadsPerUnit / kOwn) factors[my_head + k] = f;
                }
                __syncwarp();
#pragma unroll
                for (int h = 0; h < kHeadsPerUnit; ++h) {
                    const float f = factors[h];
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[h][k] *= f;
                }
            }
            float w[kOwn];
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                // an absent token (and a head that has seen none) weighs nothing
                w[k] = s[k] == -CUDART_INF_F ? 0.f : fast_exp2(s[k] - m_ref[k]);
                l_run[k] += w[k];
            }
            __syncwarp();                          // the previous batch's weights have been read
            float* to = weights + (kRows * my_tok + half) * kHeadsPerUnit + my_head;
            if constexpr (kOwn == 2) *reinterpret_cast<float2*>(to) = make_float2(w[0], w[1]);
            else *reinterpret_cast<float4*>(to) = make_float4(w[0], w[1], w[2], w[3]);
            __syncwarp();

            // ---- acc[h] += p[t][h] V[t]
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = kRows * i + half;
                float4 v = *reinterpret_cast<const float4*>(vp + t * C::kRowBytes);
                if (!((bm >> t) & 1u)) v = make_float4(0.f, 0.f, 0.f, 0.f);      // it may hold NaN
                const float4 w0 = reinterpret_cast<const float4*>(weights)[2 * t];
                const float4 w1 = reinterpret_cast<const float4*>(weights)[2 * t + 1];
                const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int h = 0; h < kHeadsPerUnit; ++h) {
                    acc[h][0] = fmaf(wt[h], v.x, acc[h][0]);
                    acc[h][1] = fmaf(wt[h], v.y, acc[h][1]);
                    acc[h][2] = fmaf(wt[h], v.z, acc[h][2]);
                    acc[h][3] = fmaf(wt[h], v.w, acc[h][3]);
                }
            }
        }

        // the slot is free again: let the issue side refill it
        __syncwarp();
        fence_proxy_async();
        ++g_cons;
        ++c_stage;
        issue_one();

        if (c_stage == c_nst) {
            // ---- finish the unit: l over the lanes that hold the same heads, then to every lane
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
#pragma unroll
                for (int off = kOwn == 2 ? 4 : 2; off < 32; off <<= 1)
                    l_run[k] += __shfl_xor_sync(0xffffffffu, l_run[k], off);
                if (lane < kHeadsPerUnit / kOwn) factors[my_head + k] = l_run[k];
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < kHeadsPerUnit; ++h) {
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = acc[h][k];
                    if constexpr (kRows == 2) v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
                }
                if (h >= cu.nh || half != 0) continue;
                const size_t row = (size_t)cu.s * p.Hq + cu.h0 + h;
                if (cu.np == 1) {
                    const float l = factors[h], f = l > 0.f ? p.out_scale / l : 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) store_elem<QF>(p.out, row * D + 4 * rl + k, v[k] * f);
                } else {
                    *reinterpret_cast<float4*>(p.part_acc + (row * p.Pmax + cu.part) * D + 4 * rl) =
                        make_float4(v[0], v[1], v[2], v[3]);
                }
            }
            if (cu.np > 1 && lane < kHeadsPerUnit / kOwn) {
#pragma unroll
                for (int k = 0; k < kOwn; ++k)
                    if (my_head + k < cu.nh) {
                        const size_t u = ((size_t)cu.s * p.Hq + cu.h0 + my_head + k) * p.Pmax + cu.part;
                        p.part_ml[2 * u] = m_ref[k];
                        p.part_ml[2 * u + 1] = l_run[k];
                    }
            }
            have_unit = false;
        }
    }

    wait_stages(bar, kStages, g_cons, g_issue, kWaitLimitCycles);      // none, unless it gave up

    if (p.local) merge_set<D, QF>(p, nsets, C::kWarps);

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

// The cache [NB, bs, Hkv, d] as rows of Hkv * d values, NB * bs of them; a box
// is one K/V head's row of 16 consecutive tokens of a block.
bool encode_map(CUtensorMap* map, const void* base, const DecodeParams& p) {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)p.Hkv * p.d, (cuuint64_t)p.NB * p.bs};
    const cuuint64_t strides[1] = {(cuuint64_t)p.Hkv * p.d * 4};
    const cuuint32_t box[2] = {(cuuint32_t)p.d, (cuuint32_t)kTok};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, typename QF>
cudaError_t launch_f32_one(DecodeParams& p, int num_sms, cudaStream_t st) {
    using C = FCfg<D>;
    auto kern = decode_f32_kernel<D, QF>;
    static SmemOptIn optin;
    const cudaError_t e = optin.ensure(reinterpret_cast<const void*>(kern), C::kSmemBytes);
    if (e != cudaSuccess) return e;
    CUtensorMap kmap, vmap;
    if (!encode_map(&kmap, p.kc, p) || !encode_map(&vmap, p.vc, p)) return cudaErrorInvalidValue;
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
    return launch_pdl(kern, dim3(grid < 1 ? 1 : grid), dim3(C::kWarps * 32), C::kSmemBytes, st, p, kmap, vmap, units,
                      region_a, nsets);
}

}  // namespace

bool decode_f32_supports(pkv_dtype c_dt, int bs, int NB) {
    return c_dt == PKV_F32 && (long long)NB * bs < (1LL << 31);      // TMA row coordinates are 32-bit
}

cudaError_t launch_decode_f32(DecodeParams& p, pkv_dtype q_dt, int num_sms, cudaStream_t st) {
    if (p.S == 0) return cudaSuccess;
    if (p.d == 64) return q_dt == PKV_F32 ? launch_f32_one<64, F32>(p, num_sms, st) : launch_f32_one<64, BF16>(p, num_sms, st);
    return q_dt == PKV_F32 ? launch_f32_one<128, F32>(p, num_sms, st) : launch_f32_one<128, BF16>(p, num_sms, st);
}

}  // namespace pkv
