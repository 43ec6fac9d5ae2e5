// paged_kv4_write and paged_kv4_read: new tokens into the 4-bit cache, and
// the values of its slots back.
//
// "LLM推論の基礎とvLLMの内部", section 2: the bytes of a K/V element set how
// many tokens a cache holds; the format is in pkv_kv4.cuh.
//
// Per group of 32 scaled values y = x / k_scale (v_scale), clamped to fp16's
// range: zero = fp16(min y), scale = fp16(max(max y - zero, 0) / 15),
// code = clamp(rint((y - zero) / scale), 0, 15), or 0 where scale is 0; all
// in fp32 with IEEE rounding, so the bytes do not depend on the kernel.  A
// NaN makes its group's zero NaN.
#include <cuda_fp16.h>
#include <math_constants.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_kv4.cuh"

namespace pkv {
namespace {

// One thread per 8 consecutive values, four lanes per group.
template <int D, typename In>
__global__ void __launch_bounds__(256) kv4_write_kernel(Kv4Params p) {
    using F = Kv4<D>;
    pdl_trigger();
    pdl_wait();
    constexpr int CH = D / 8;
    const long long total = (long long)p.T * 2 * p.Hkv * CH;
    const long long slots = (long long)p.NB * p.bs;
    const int head_bytes = kv4_head_bytes(p.bs, D);
    const int lane = threadIdx.x & 31;
    // every lane of a warp takes the same number of turns: the groups' shuffles need all of them
    for (long long it0 = (long long)blockIdx.x * blockDim.x + (threadIdx.x & ~31); it0 < total;
         it0 += (long long)gridDim.x * blockDim.x) {
        const long long it = it0 + lane;
        bool live = it < total;
        const int c = (int)(it % CH);
        long long r = it / CH;
        const int h = (int)(r % p.Hkv);
        r /= p.Hkv;
        const int which = (int)(r & 1);       // 0 = K, 1 = V
        const long long i = r >> 1;           // token
        long long s = -1;
        if (live) {
            s = p.slots[i];
            if (s >= slots) {
                if (which == 0 && h == 0 && c == 0) report(p.err, PKV_DEVERR_SLOT);
                s = -1;
            }
            live = s >= 0;
        }
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = 0.f;
        if (live) load8<In>(which ? p.value : p.key, ((size_t)i * p.Hkv + h) * D + 8 * (size_t)c, y);
        const float by = which ? p.v_scale : p.k_scale;
        float mn = CUDART_INF_F, mx = -CUDART_INF_F;
        bool nan = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            y[k] = __fdiv_rn(y[k], by);
            nan = nan || y[k] != y[k];
            y[k] = fminf(fmaxf(y[k], -kKv4Max), kKv4Max);
            mn = fminf(mn, y[k]);
            mx = fmaxf(mx, y[k]);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        nan = (__ballot_sync(0xffffffffu, nan) >> (lane & ~3)) & 15u;
        if (!live) continue;
        const __half hz = nan ? __ushort_as_half(0x7e00) : __float2half_rn(mn);
        const float z = __half2float(hz);
        const __half hs = nan ? __ushort_as_half(0) : __float2half_rn(__fdiv_rn(fmaxf(__fsub_rn(mx, z), 0.f), 15.f));
        const float sc = __half2float(hs);
        uint32_t w = 0;
        if (sc > 0.f) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float q = rintf(__fdiv_rn(__fsub_rn(y[k], z), sc));
                w |= (uint32_t)fminf(fmaxf(q, 0.f), 15.f) << (4 * k);
            }
        }
        const int t = (int)(s % p.bs), e = 8 * c, g = e / 32;
        unsigned char* blk = static_cast<unsigned char*>(which ? p.value_cache : p.key_cache) +
                             ((size_t)(s / p.bs) * p.Hkv + h) * head_bytes;
        __half* par = reinterpret_cast<__half*>(blk + F::codes(p.bs));
        if (which == 0) {
            reinterpret_cast<uint32_t*>(blk)[F::k_word(t, e)] = w;
        } else {
            uint16_t* c16 = reinterpret_cast<uint16_t*>(blk);
            c16[2 * F::v_word(t, e) + t % 2] = (uint16_t)w;
            c16[2 * F::v_word(t, e + 4) + t % 2] = (uint16_t)(w >> 16);
        }
        if (c % 4 == 0) {
            const int a = which ? F::v_par(t, g) : F::k_par(t, g);
            par[a] = hs;
            par[p.bs * F::G + a] = hz;
        }
    }
}

template <int D, typename Out>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Params p) {
    using F = Kv4<D>;
    pdl_trigger();
    pdl_wait();
    constexpr int CH = D / 8;
    const long long total = (long long)p.T * 2 * p.Hkv * CH;
    const long long slots = (long long)p.NB * p.bs;
    const int head_bytes = kv4_head_bytes(p.bs, D);
    for (long long it = (long long)blockIdx.x * blockDim.x + threadIdx.x; it < total;
         it += (long long)gridDim.x * blockDim.x) {
        const int c = (int)(it % CH);
        long long r = it / CH;
        const int h = (int)(r % p.Hkv);
        r /= p.Hkv;
        const int which = (int)(r & 1);
        const long long i = r >> 1;
        const long long s = p.slots[i];
        if (s < 0) continue;
        if (s >= slots) {
            if (which == 0 && h == 0 && c == 0) report(p.err, PKV_DEVERR_SLOT);
            continue;
        }
        const int t = (int)(s % p.bs), e = 8 * c, g = e / 32;
        const unsigned char* blk = static_cast<const unsigned char*>(which ? p.value_cache : p.key_cache) +
                                   ((size_t)(s / p.bs) * p.Hkv + h) * head_bytes;
        const __half* par = reinterpret_cast<const __half*>(blk + F::codes(p.bs));
        const int a = which ? F::v_par(t, g) : F::k_par(t, g);
        const float sc = __half2float(par[a]), z = __half2float(par[p.bs * F::G + a]);
        uint32_t w;
        if (which == 0) {
            w = reinterpret_cast<const uint32_t*>(blk)[F::k_word(t, e)];
        } else {
            const uint16_t* c16 = reinterpret_cast<const uint16_t*>(blk);
            w = c16[2 * F::v_word(t, e) + t % 2] | ((uint32_t)c16[2 * F::v_word(t, e + 4) + t % 2] << 16);
        }
        const float by = which ? p.v_scale : p.k_scale;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fmaf(sc, (float)((w >> (4 * k)) & 15u), z) * by;
        store8<Out>(which ? p.value_out : p.key_out, ((size_t)i * p.Hkv + h) * D + 8 * (size_t)c, v, 1.f);
    }
}

}  // namespace

cudaError_t launch_kv4(const Kv4Params& p, pkv_dtype dt, bool read, cudaStream_t st) {
    if (p.T == 0) return cudaSuccess;
    const long long items = (long long)p.T * 2 * p.Hkv * (p.d / 8);
    const long long want = (items + 255) / 256;
    const dim3 g((unsigned)(want < 65536 ? want : 65536)), b(256);
    const bool f32 = dt == PKV_F32, d64 = p.d == 64;
    if (read) {
        if (d64) return f32 ? launch_pdl(kv4_read_kernel<64, F32>, g, b, 0, st, p) : launch_pdl(kv4_read_kernel<64, BF16>, g, b, 0, st, p);
        return f32 ? launch_pdl(kv4_read_kernel<128, F32>, g, b, 0, st, p) : launch_pdl(kv4_read_kernel<128, BF16>, g, b, 0, st, p);
    }
    if (d64) return f32 ? launch_pdl(kv4_write_kernel<64, F32>, g, b, 0, st, p) : launch_pdl(kv4_write_kernel<64, BF16>, g, b, 0, st, p);
    return f32 ? launch_pdl(kv4_write_kernel<128, F32>, g, b, 0, st, p) : launch_pdl(kv4_write_kernel<128, BF16>, g, b, 0, st, p);
}

}  // namespace pkv
