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
//
// A warp takes 8 consecutive tokens of one K or V head, in the shape of the
// format: of K a lane holds one token's word of every group (eight values
// each), of V a pair of tokens' word of every group (four values each), so
// its codes leave in one 16-byte store and a warp's in 512 consecutive
// bytes.  Two tokens of V that are not neighbours in a block (a decoding
// step's) take 2-byte stores instead.  The bound is the bytes (read and
// written once) and, as close, about 16 instructions per value.
#include <cuda_fp16.h>
#include <math_constants.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_kv4.cuh"

namespace pkv {
namespace {

// NaN if either is
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A group's scale and zero from its smallest and largest value (NaN if the group holds one).
__device__ __forceinline__ void kv4_params(float mn, float mx, __half& hs, __half& hz) {
    if (mn != mn) {
        hz = __ushort_as_half(0x7e00);
        hs = __ushort_as_half(0);
        return;
    }
    hz = __float2half_rn(fminf(fmaxf(mn, -kKv4Max), kKv4Max));
    const float top = fminf(fmaxf(mx, -kKv4Max), kKv4Max);
    hs = __float2half_rn(__fdiv_rn(fmaxf(__fsub_rn(top, __half2float(hz)), 0.f), 15.f));
}

// N codes of one group, code k in bits 4 k.  The quotient is taken as a
// product with the scale's reciprocal, which is within 2^-18 of the IEEE
// quotient where that is between 0 and 15 (two roundings of 2^-24 relative,
// against one), so both round to the same whole number unless the product
// is that near a half; there the division is done.  Values clamped to fp16's
// range need no clamp here: they end at code 0 or 15 either way.
template <int N>
__device__ __forceinline__ uint32_t kv4_codes(const float (&y)[N], float sc, float z) {
    if (!(sc > 0.f)) return 0u;
    const float inv = __fdiv_rn(1.f, sc);
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float d = __fsub_rn(y[k], z);
        float q = fminf(fmaxf(__fmul_rn(d, inv), 0.f), 15.f);
        const float near = __fadd_rn(q, 12582912.f);            // 1.5 * 2^23: the nearest whole number in the low bits
        uint32_t code = __float_as_uint(near) & 15u;
        if (fabsf(__fsub_rn(q, __fsub_rn(near, 12582912.f))) > 0.5f - 3.814697265625e-6f)
            code = (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(d, sc)), 0.f), 15.f);
        w |= code << (4 * k);
    }
    return w;
}

// What a warp works on: head h of K (v false) or V, tokens i0 .. i0 + 7, whose
// slots lane j < 8 holds (-1: skipped).
struct Octet {
    long long i0, slot;
    int h;
    bool v;
};
__device__ __forceinline__ bool octet_of(const Kv4Params& p, Octet& o) {
    const int lane = threadIdx.x & 31, row = blockIdx.y * (blockDim.x / 32) + threadIdx.x / 32;
    if (row >= 2 * p.Hkv) return false;
    o.v = row >= p.Hkv;
    o.h = o.v ? row - p.Hkv : row;
    o.i0 = 8LL * blockIdx.x;
    o.slot = -1;
    if (lane < 8 && o.i0 + lane < p.T) {
        o.slot = __ldg(p.slots + o.i0 + lane);
        if (o.slot >= (long long)p.NB * p.bs) {
            if (row == 0) report(p.err, PKV_DEVERR_SLOT);
            o.slot = -1;
        }
    }
    return true;
}

// G words at `dst` (16- or 8-byte aligned)
template <int G>
__device__ __forceinline__ void store_words(void* dst, const uint32_t (&w)[G]) {
    if constexpr (G == 4) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}
template <int G>
__device__ __forceinline__ void load_words(const void* src, uint32_t (&w)[G]) {
    if constexpr (G == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(src);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        w[0] = v.x; w[1] = v.y;
    }
}
__device__ __forceinline__ uint32_t pair_bits(__half lo, __half hi) {
    return (uint32_t)__half_as_ushort(lo) | ((uint32_t)__half_as_ushort(hi) << 16);
}

// four consecutive input elements as fp32
template <typename In>
__device__ __forceinline__ void load4(const void* base, size_t i, float (&v)[4]) {
    if constexpr (In::bytes == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + i));
        v[0] = __uint_as_float(a.x << 16);
        v[1] = __uint_as_float(a.x & 0xffff0000u);
        v[2] = __uint_as_float(a.y << 16);
        v[3] = __uint_as_float(a.y & 0xffff0000u);
    }
}
template <typename Out>
__device__ __forceinline__ void store4(void* base, size_t i, const float (&v)[4]) {
    if constexpr (Out::bytes == 4) {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}

template <int D, typename In>
__global__ void __launch_bounds__(256) kv4_write_kernel(Kv4Params p) {
    using F = Kv4<D>;
    constexpr int G = F::G;
    pdl_trigger();
    pdl_wait();
    Octet o;
    if (!octet_of(p, o)) return;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, sh = p.bs == 16 ? 4 : 5;
    const int head_bytes = kv4_head_bytes(p.bs, D), zeros = p.bs * G;
    const float by = o.v ? p.v_scale : p.k_scale;
    const bool scaled = by != 1.f;
    if (!o.v) {
        const long long s = __shfl_sync(0xffffffffu, o.slot, r);
        const size_t src = ((size_t)(o.i0 + r) * p.Hkv + o.h) * D + 8 * c;
        float y[G][8], mn[G], mx[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (s >= 0) {
                load8<In>(p.key, src + 32 * g, y[g]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) y[g][k] = 0.f;
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (scaled)
#pragma unroll
                for (int k = 0; k < 8; ++k) y[g][k] = __fdiv_rn(y[g][k], by);
            mn[g] = mx[g] = y[g][0];
#pragma unroll
            for (int k = 1; k < 8; ++k) {
                mn[g] = min_nan(mn[g], y[g][k]);
                mx[g] = fmaxf(mx[g], y[g][k]);
            }
#pragma unroll
            for (int q = 1; q < 4; q <<= 1) {
                mn[g] = min_nan(mn[g], __shfl_xor_sync(0xffffffffu, mn[g], q));
                mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], q));
            }
        }
        if (s < 0) return;
        const int t = (int)s & (p.bs - 1);
        unsigned char* blk = static_cast<unsigned char*>(p.key_cache) + ((size_t)(s >> sh) * p.Hkv + o.h) * head_bytes;
        __half hs[G], hz[G];
        uint32_t w[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            kv4_params(mn[g], mx[g], hs[g], hz[g]);
            w[g] = kv4_codes(y[g], __half2float(hs[g]), __half2float(hz[g]));
        }
        store_words<G>(blk + 4 * F::k_word(t, 8 * c), w);
        if (c < 2) {                              // lane 0 of a token's four: the scales, lane 1: the zeros
            __half* par = reinterpret_cast<__half*>(blk + F::codes(p.bs)) + (c ? zeros : 0) + F::k_par(t, 0);
#pragma unroll
            for (int g = 0; g < G; g += 2)
                reinterpret_cast<uint32_t*>(par)[g / 2] = c ? pair_bits(hz[g], hz[g + 1]) : pair_bits(hs[g], hs[g + 1]);
        }
        return;
    }
    // V: tokens 2c and 2c + 1, values 32 g + 4 r .. + 3
    long long s[2];
    uint32_t half[2][G];                          // 16 bits: four codes
    __half hs[2][G], hz[2][G];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        s[j] = __shfl_sync(0xffffffffu, o.slot, 2 * c + j);
        const size_t src = ((size_t)(o.i0 + 2 * c + j) * p.Hkv + o.h) * D + 4 * r;
        float y[G][4];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (s[j] >= 0) {
                load4<In>(p.value, src + 32 * g, y[g]);
            } else {
                y[g][0] = y[g][1] = y[g][2] = y[g][3] = 0.f;
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (scaled)
#pragma unroll
                for (int k = 0; k < 4; ++k) y[g][k] = __fdiv_rn(y[g][k], by);
            float mn = min_nan(min_nan(y[g][0], y[g][1]), min_nan(y[g][2], y[g][3]));
            float mx = fmaxf(fmaxf(y[g][0], y[g][1]), fmaxf(y[g][2], y[g][3]));
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) {
                mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, q));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
            }
            kv4_params(mn, mx, hs[j][g], hz[j][g]);
            half[j][g] = kv4_codes(y[g], __half2float(hs[j][g]), __half2float(hz[j][g]));
        }
    }
    auto block = [&](long long slot) {
        return static_cast<unsigned char*>(p.value_cache) + ((size_t)(slot >> sh) * p.Hkv + o.h) * head_bytes;
    };
    if (s[0] >= 0 && (s[0] & 1) == 0 && s[1] == s[0] + 1) {
        const int t = (int)s[0] & (p.bs - 1);
        unsigned char* blk = block(s[0]);
        uint32_t w[G];
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = half[0][g] | (half[1][g] << 16);
        store_words<G>(blk + 4 * F::v_word(t, 4 * r), w);
        if (r < 2) {
            uint32_t q[G];
#pragma unroll
            for (int g = 0; g < G; ++g) q[g] = r ? pair_bits(hz[0][g], hz[1][g]) : pair_bits(hs[0][g], hs[1][g]);
            store_words<G>(reinterpret_cast<__half*>(blk + F::codes(p.bs)) + (r ? zeros : 0) + F::v_par(t, 0), q);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (s[j] < 0) continue;
        const int t = (int)s[j] & (p.bs - 1);
        unsigned char* blk = block(s[j]);
        __half* par = reinterpret_cast<__half*>(blk + F::codes(p.bs)) + (r ? zeros : 0);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            reinterpret_cast<uint16_t*>(blk)[2 * F::v_word(t, 32 * g + 4 * r) + t % 2] = (uint16_t)half[j][g];
            if (r < 2) par[F::v_par(t, g)] = r ? hz[j][g] : hs[j][g];
        }
    }
}

// (zero + scale * code) * tensor scale: the product of 11 and 4 bits is exact
__device__ __forceinline__ float kv4_value(uint32_t w, int k, float sc, float z, float by) {
    return fmaf(sc, (float)((w >> (4 * k)) & 15u), z) * by;
}

template <int D, typename Out>
__global__ void __launch_bounds__(256) kv4_read_kernel(Kv4Params p) {
    using F = Kv4<D>;
    constexpr int G = F::G;
    pdl_trigger();
    pdl_wait();
    Octet o;
    if (!octet_of(p, o)) return;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, sh = p.bs == 16 ? 4 : 5;
    const int head_bytes = kv4_head_bytes(p.bs, D), zeros = p.bs * G;
    const float by = o.v ? p.v_scale : p.k_scale;
    const unsigned char* cache = static_cast<const unsigned char*>(o.v ? p.value_cache : p.key_cache);
    auto block = [&](long long slot) { return cache + ((size_t)(slot >> sh) * p.Hkv + o.h) * head_bytes; };
    if (!o.v) {
        const long long s = __shfl_sync(0xffffffffu, o.slot, r);
        if (s < 0) return;
        const int t = (int)s & (p.bs - 1);
        const unsigned char* blk = block(s);
        const __half* par = reinterpret_cast<const __half*>(blk + F::codes(p.bs)) + F::k_par(t, 0);
        uint32_t w[G];
        load_words<G>(blk + 4 * F::k_word(t, 8 * c), w);
        const size_t dst = ((size_t)(o.i0 + r) * p.Hkv + o.h) * D + 8 * c;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float sc = __half2float(par[g]), z = __half2float(par[zeros + g]);
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = kv4_value(w[g], k, sc, z, by);
            store8<Out>(p.key_out, dst + 32 * g, v, 1.f);
        }
        return;
    }
    const long long s0 = __shfl_sync(0xffffffffu, o.slot, 2 * c), s1 = __shfl_sync(0xffffffffu, o.slot, 2 * c + 1);
    const long long s[2] = {s0, s1};
    uint32_t w[2][G], ps[2][G], pz[2][G];         // each token's codes, scales and zeros in the low half
    if (s0 >= 0 && (s0 & 1) == 0 && s1 == s0 + 1) {
        const int t = (int)s0 & (p.bs - 1);
        const unsigned char* blk = block(s0);
        const __half* par = reinterpret_cast<const __half*>(blk + F::codes(p.bs)) + F::v_par(t, 0);
        load_words<G>(blk + 4 * F::v_word(t, 4 * r), w[0]);
        load_words<G>(par, ps[0]);
        load_words<G>(par + zeros, pz[0]);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            w[1][g] = w[0][g] >> 16;
            ps[1][g] = ps[0][g] >> 16;
            pz[1][g] = pz[0][g] >> 16;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (s[j] < 0) continue;
            const int t = (int)s[j] & (p.bs - 1);
            const unsigned char* blk = block(s[j]);
            const uint16_t* par = reinterpret_cast<const uint16_t*>(blk + F::codes(p.bs));
#pragma unroll
            for (int g = 0; g < G; ++g) {
                w[j][g] = reinterpret_cast<const uint16_t*>(blk)[2 * F::v_word(t, 32 * g + 4 * r) + t % 2];
                ps[j][g] = par[F::v_par(t, g)];
                pz[j][g] = par[zeros + F::v_par(t, g)];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (s[j] < 0) continue;
        const size_t dst = ((size_t)(o.i0 + 2 * c + j) * p.Hkv + o.h) * D + 4 * r;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float sc = __half2float(__ushort_as_half((unsigned short)ps[j][g]));
            const float z = __half2float(__ushort_as_half((unsigned short)pz[j][g]));
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = kv4_value(w[j][g], k, sc, z, by);
            store4<Out>(p.value_out, dst + 32 * g, v);
        }
    }
}

}  // namespace

cudaError_t launch_kv4(const Kv4Params& p, pkv_dtype dt, bool read, cudaStream_t st) {
    if (p.T == 0) return cudaSuccess;
    const int warps = 2 * p.Hkv < 8 ? 2 * p.Hkv : 8;
    const dim3 g((unsigned)((p.T + 7LL) / 8), (unsigned)((2 * p.Hkv + warps - 1) / warps)), b(32 * warps);
    const bool f32 = dt == PKV_F32, d64 = p.d == 64;
    if (read) {
        if (d64) return f32 ? launch_pdl(kv4_read_kernel<64, F32>, g, b, 0, st, p) : launch_pdl(kv4_read_kernel<64, BF16>, g, b, 0, st, p);
        return f32 ? launch_pdl(kv4_read_kernel<128, F32>, g, b, 0, st, p) : launch_pdl(kv4_read_kernel<128, BF16>, g, b, 0, st, p);
    }
    if (d64) return f32 ? launch_pdl(kv4_write_kernel<64, F32>, g, b, 0, st, p) : launch_pdl(kv4_write_kernel<64, BF16>, g, b, 0, st, p);
    return f32 ? launch_pdl(kv4_write_kernel<128, F32>, g, b, 0, st, p) : launch_pdl(kv4_write_kernel<128, BF16>, g, b, 0, st, p);
}

}  // namespace pkv
