// Decode of sequences in groups whose first blocks are the same ones.
//
// "vLLM 内部構造 (2) — PagedAttention", section "共有": requests with one
// system prompt point at the same physical blocks; "LLM推論の基礎とvLLMの
// 内部", section 4: blocks of a shared prefix carry a reference count.
//
// softmax(q k^T) v over a sequence's tokens is joined from two parts by their
// maxima and sums: the shared tokens, which the queries of all members of a
// group attend to in one matrix product (attend_kernel<SHARED>: the group's
// K and V are read once, not once per member), and the sequence's own tokens
// (the decode, begun behind the shared ones).  Every partition of either part
// leaves (m, l, O) in fp32; one warp per (sequence, head) joins them.  Bound by
// HBM for groups of few rows (members x heads per K/V head), by the tensor
// cores for large ones.
#include "pkv_attend_umma.cuh"
#include "pkv_merge.cuh"

namespace pkv {
namespace {

template <int D>
__global__ void __launch_bounds__(256) shared_merge_kernel(const __grid_constant__ PromptParams p,
                                                           const __grid_constant__ SharedParts x) {
    constexpr int E = D / 32, B = kMergeChunk;
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.own_max = 0;      // for the next call
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)p.Tq * p.Hq) return;
    const int s = (int)(row / p.Hq);
    const int begin = load_behind_wait(p.begin + s), n = min(max(load_behind_wait(p.lens + s), 0), x.max_ctx) - begin;
    int pre = 0, own = num_partitions(n, x.P, x.Q, 0);
    if (begin == 0) {
        if (own <= 1) return;                    // the decode has written it
    } else {
        const int stages = ceil_div(begin, kTok);
        pre = p.P > 0 && stages > p.P ? ceil_div(stages, p.P) : 1;
        if (n <= 0) own = 0;
    }
    const int np = pre + own;
    const float* ml = p.part_ml + 2 * (size_t)row * p.Pmax;
    const float* acc = p.part_acc + (size_t)row * p.Pmax * D;
    auto part = [&](int j) { return j < pre ? j : x.first_own + j - pre; };
    // as merge_partitions, over two runs of partial results
    const uint64_t once = l2_policy_evict_first();
    float M = -CUDART_INF_F, lpart = 0.f, o[E];
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = 0.f;
    for (int c0 = 0; c0 < np; c0 += B) {
        const int cn = min(B, np - c0);
        float m = -CUDART_INF_F, l = 0.f;
        if (lane < cn) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(ml) + part(c0 + lane));
            m = v.x;
            l = v.y;
        }
        float a[B][E];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (j < cn) {
                merge_load_row<E>(acc + (size_t)part(c0 + j) * D + lane * E, a[j], once);
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) a[j][k] = 0.f;
            }
        }
        float cm = m;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, off));
        const float Mn = fmaxf(M, cm);
        // a partition with no visible token has m = -inf and weighs nothing
        const float f = M == -CUDART_INF_F ? 0.f : exp2f(M - Mn);
        const float w = m == -CUDART_INF_F ? 0.f : exp2f(m - Mn);
        lpart = fmaf(w, l, lpart * f);
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] *= f;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = fmaf(wj, a[j][k], o[k]);
        }
        M = Mn;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lpart += __shfl_xor_sync(0xffffffffu, lpart, off);
    const float f = lpart > 0.f || lpart != lpart ? 1.f / lpart : 0.f;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (size_t)row * D + lane * E;
    uint32_t w[E / 2];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) w[k] = pack2<false>(o[2 * k] * f, o[2 * k + 1] * f);
    if constexpr (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(out) = w[0];
}

template <int D>
cudaError_t launch_d(const PromptParams& p, const DecodeParams& d, int num_sms, cudaStream_t st) {
    CUtensorMap kmap, vmap;
    if (!prefill_encode_kv_map(&kmap, p.k, d) || !prefill_encode_kv_map(&vmap, p.v, d)) return cudaErrorInvalidValue;
    const long long tiles = ((long long)p.max_q * p.g + kRows - 1) / kRows;
    const long long units = (long long)p.S * p.Hkv * ((tiles + 1) / 2) * ceil_div(ceil_div(p.max_k, kTok), p.P > 0 ? p.P : 1 << 24);
    return launch_attend<D, kShared>(p, kmap, kmap, vmap, kmap, units, num_sms, st);
}

}  // namespace

cudaError_t launch_shared_prefix(const PromptParams& p, const DecodeParams& d, int num_sms, cudaStream_t st) {
    return d.d == 64 ? launch_d<64>(p, d, num_sms, st) : launch_d<128>(p, d, num_sms, st);
}

cudaError_t launch_shared_merge(const PromptParams& p, const SharedParts& x, int d, cudaStream_t st) {
    const long long rows = (long long)p.Tq * p.Hq;
    const dim3 grid((unsigned)((rows + 7) / 8)), block(256);
    return d == 64 ? launch_pdl(shared_merge_kernel<64>, grid, block, 0, st, p, x)
                   : launch_pdl(shared_merge_kernel<128>, grid, block, 0, st, p, x);
}

}  // namespace pkv
