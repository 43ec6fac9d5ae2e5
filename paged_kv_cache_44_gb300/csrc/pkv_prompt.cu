// Attention over whole packed prompts (pkv_attend_umma.cuh): the merge of a
// split launch, and the launch.
#include "pkv_attend_umma.cuh"
#include "pkv_merge.cuh"

namespace pkv {
namespace {

// The merge of a launch's partitions, one warp per (query, head).
template <int D, int MODE>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const __grid_constant__ PromptParams p) {
    constexpr int E = D / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long gw = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (gw >= (long long)p.Tq * p.Hq) return;
    const int tq = (int)(gw / p.Hq);
    // the sequence that holds the query, past any that is empty (starts that do not rise are skipped below)
    int lo = 0, hi = p.S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (load_behind_wait(p.query_start + mid) <= tq) lo = mid; else hi = mid;
    }
    Seq x;
    Group g;
    if (!sequence<MODE>(p, lo, x) || tq < x.q0 || tq >= x.q0 + x.ql ||
        !group_of<MODE>(p, x, MODE == kPacked ? 0 : (tq - x.q0) / (p.group * kRows), g) || g.np <= 1)
        return;
    float acc[E];
    const size_t u0 = (size_t)gw * p.Pmax;
    const float L = merge_partitions<D>(p.part_ml + 2 * u0, p.part_acc + u0 * D, g.np, lane, acc);
    const float f = L > 0.f || L != L ? 1.f / L : 0.f;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (size_t)gw * D + lane * E;
    uint32_t w[E / 2];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) w[k] = pack2<false>(acc[2 * k] * f, acc[2 * k + 1] * f);
    if constexpr (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(out) = w[0];
}

template <int D, int MODE>
cudaError_t launch_mode(const PromptParams& p, int num_sms, cudaStream_t st) {
    CUtensorMap qmap, kmap, vmap, omap;
    // (no keys at all: nothing is loaded through the maps of K and V)
    if (!encode_rows_map(&kmap, p.Tk > 0 ? p.k : p.q, p.Tk, p.Hkv * D, p.k_stride, kTok) ||
        !encode_rows_map(&vmap, p.Tk > 0 ? p.v : p.q, p.Tk, p.Hkv * D, p.v_stride, kTok))
        return cudaErrorInvalidValue;
    if (MODE == kPacked) {
        qmap = omap = kmap;                      // (not used)
    } else if (!encode_rows_map(&qmap, p.q, p.Tq, p.Hq * D, p.q_stride, kRows) ||
               !encode_rows_map(&omap, p.out, p.Tq, p.Hq * D, (long long)p.Hq * D, 32)) {
        return cudaErrorInvalidValue;
    }
    const long long per_head = MODE == kPacked ? (ceil_div(p.max_q * p.g, kRows) + 1) / 2
                                               : (long long)ceil_div(p.max_q, p.group * kRows) * ((p.g * p.group + 1) / 2);
    const cudaError_t e = launch_attend<D, MODE>(p, qmap, kmap, vmap, omap, (long long)p.S * p.Hkv * per_head * p.Pmax, num_sms, st);
    if (e != cudaSuccess || p.Pmax <= 1) return e;
    const long long rows = (long long)p.Tq * p.Hq;
    return launch_pdl(prompt_merge_kernel<D, MODE>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, p);
}

template <int D>
cudaError_t launch_prompt_d(const PromptParams& p, int num_sms, cudaStream_t st) {
    return p.packed ? launch_mode<D, kPacked>(p, num_sms, st) : launch_mode<D, kHeads>(p, num_sms, st);
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, int d, int num_sms, cudaStream_t st) {
    return d == 64 ? launch_prompt_d<64>(p, num_sms, st) : launch_prompt_d<128>(p, num_sms, st);
}

}  // namespace pkv
