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
// step's) take 2-byte stores instead.  The smallest and largest values of
// the groups a warp's lanes share are reduced together, each lane ending with
// one group (14 shuffles for 16 reductions over 8 lanes), whose scale and
// zero it alone computes and hands out.  The bound is the bytes, read and
// written once, and, as close, the instructions per value: 8,192 bf16 tokens
// of 8 heads of 128 (34 MB in, 10 MB out) take 19.5 us, 61% of the issue slots
// over its length; the floor at the copy rate is 6.5.  Reading them back as
// fp32 takes 16.2 us (10 MB in, 67 out, floor 11.4).
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

// A group's scale and zero, and what its codes are computed with: a value x
// has the quotient q = (x / by - zero) / scale = 15 (x A + B) up to rounding.
struct GroupScale {
    __half hs, hz;
    float A, B, slack;
};

// mn, mx: the smallest and largest x of the group (NaN if it holds one);
// rby = 1 / by.  x / by is monotonic in x, so the two divisions give the
// smallest and largest y.  In fp32 A is off by three roundings (2^-24
// relative each), B by two, their sum by one; y, y - zero and its division
// in the definition by one each: together at most 2^-24 (6 max|y| / scale +
// 45) of q, which `slack` bounds.
__device__ __forceinline__ GroupScale group_scale(float mn, float mx, float by, float rby) {
    GroupScale s;
    s.A = s.B = 0.f;
    s.slack = 0.f;
    if (mn != mn) {
        s.hz = __ushort_as_half(0x7e00);
        s.hs = __ushort_as_half(0);
        return s;
    }
    if (by != 1.f) {
        mn = __fdiv_rn(mn, by);
        mx = __fdiv_rn(mx, by);
    }
    mn = fminf(fmaxf(mn, -kKv4Max), kKv4Max);
    mx = fminf(fmaxf(mx, -kKv4Max), kKv4Max);
    s.hz = __float2half_rn(mn);
    const float z = __half2float(s.hz);
    s.hs = __float2half_rn(__fdiv_rn(fmaxf(__fsub_rn(mx, z), 0.f), 15.f));
    const float sc = __half2float(s.hs);
    if (sc > 0.f) {
        const float inv = __fdiv_rn(1.f, 15.f * sc);
        s.A = __fmul_rn(inv, rby);
        s.B = -__fmul_rn(z, inv);
        s.slack = 4.76837158203125e-7f * (fmaxf(fabsf(mn), fabsf(mx)) * inv * 15.f + 6.f);   // 2^-21
        if (!(s.A > 1e-30f && s.A < 1e30f)) s.slack = 1.f;                                    // extreme tensor scales
    }
    return s;
}

// Four codes of one group by the definition, code k in bits 4 k; par: the group's scale and zero.
__device__ __noinline__ uint32_t kv4_codes_exact(float x0, float x1, float x2, float x3, float by, uint32_t par) {
    const float sc = __half2float(__ushort_as_half((unsigned short)par));
    const float z = __half2float(__ushort_as_half((unsigned short)(par >> 16)));
    if (!(sc > 0.f)) return 0u;
    const float x[4] = {x0, x1, x2, x3};
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float y = fminf(fmaxf(__fdiv_rn(x[k], by), -kKv4Max), kKv4Max);
        w |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(y, z), sc)), 0.f), 15.f) << (4 * k);
    }
    return w;
}

// The same: q saturated to 0 .. 15 and rounded by one fused multiply-add
// (1.5 * 2^23 + 15 q / 15); values past fp16's range end at code 0 or 15
// without a clamp.  Where a quotient is within the slack of a half, so that it
// may round either way, this lane takes the definition's: of bf16 values about
// one in 2,500 is an exact half.
__device__ __forceinline__ uint32_t kv4_codes(const float* x, float A, float B, float thr, float by, uint32_t par) {
    constexpr float kWhole = 12582912.f;
    float packed = 0.f;                                   // below 2^16: exact
    bool close = false;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
        const float q = __saturatef(__fmaf_rn(x[k], A, B));
        const float f = __fsub_rn(__fmaf_rn(q, 15.f, kWhole), kWhole);
        close = close || !(fabsf(__fmaf_rn(q, 15.f, -f)) <= thr);
        packed = __fmaf_rn(packed, 16.f, f);
    }
    if (close) return kv4_codes_exact(x[0], x[1], x[2], x[3], by, par);
    return __float2uint_rn(packed);
}

// One step of a reduction that halves what a lane holds: of v[0 .. 2 N) it keeps the upper
// half (in v[0 .. N)) where `upper`, its partner in the lane distance `mask` the lower one.
template <int N, bool MIN>
__device__ __forceinline__ void halve(float* v, int mask, bool upper) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float send = upper ? v[i] : v[i + N], keep = upper ? v[i + N] : v[i];
        const float got = __shfl_xor_sync(0xffffffffu, send, mask);
        v[i] = MIN ? min_nan(keep, got) : fmaxf(keep, got);
    }
}
__device__ __forceinline__ float warp_max(float v) {      // v >= 0
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
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
        o.slot = load_behind_wait(p.slots + o.i0 + lane);
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
    const float by = o.v ? p.v_scale : p.k_scale, rby = __fdiv_rn(1.f, by);
    if (!o.v) {
        const long long s = __shfl_sync(0xffffffffu, o.slot, r);
        const size_t src = ((size_t)(o.i0 + r) * p.Hkv + o.h) * D + 8 * c;
        float x[G][8], mn[G], mx[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (s >= 0) {
                load8<In>(p.key, src + 32 * g, x[g]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[g][k] = 0.f;
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            mn[g] = mx[g] = x[g][0];
#pragma unroll
            for (int k = 1; k < 8; ++k) {
                mn[g] = min_nan(mn[g], x[g][k]);
                mx[g] = fmaxf(mx[g], x[g][k]);
            }
        }
        // over the token's four lanes: lane c ends with group c (d 64: lanes 2 g, 2 g + 1 with group g)
        halve<G / 2, true>(mn, 2, c & 2);
        halve<G / 2, false>(mx, 2, c & 2);
        if constexpr (G == 4) {
            halve<1, true>(mn, 1, c & 1);
            halve<1, false>(mx, 1, c & 1);
        } else {
            mn[0] = min_nan(mn[0], __shfl_xor_sync(0xffffffffu, mn[0], 1));
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], 1));
        }
        const GroupScale gs = group_scale(mn[0], mx[0], by, rby);
        const float thr = 0.5f - warp_max(gs.slack);
        auto holder = [&](int g) { return (lane & ~3) | (g * (4 / G)); };
        const uint32_t mine = pair_bits(gs.hs, gs.hz);
        uint32_t w[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float A = __shfl_sync(0xffffffffu, gs.A, holder(g)), B = __shfl_sync(0xffffffffu, gs.B, holder(g));
            const uint32_t par = __shfl_sync(0xffffffffu, mine, holder(g));
            w[g] = kv4_codes(x[g], A, B, thr, by, par);
            w[g] |= kv4_codes(x[g] + 4, A, B, thr, by, par) << 16;
        }
        if (s < 0) return;
        const int t = (int)s & (p.bs - 1);
        unsigned char* blk = static_cast<unsigned char*>(p.key_cache) + ((size_t)(s >> sh) * p.Hkv + o.h) * head_bytes;
        store_words<G>(blk + 4 * F::k_word(t, 8 * c), w);
        if (c % (4 / G) == 0) {
            __half* par = reinterpret_cast<__half*>(blk + F::codes(p.bs)) + F::k_par(t, c / (4 / G));
            par[0] = gs.hs;
            par[zeros] = gs.hz;
        }
        return;
    }
    // V: tokens 2c and 2c + 1, values 32 g + 4 r .. + 3; (token, group) number G j + g
    constexpr int Q = 2 * G;
    long long s[2];
    float x[Q][4], mn[Q], mx[Q];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        s[j] = __shfl_sync(0xffffffffu, o.slot, 2 * c + j);
        const size_t src = ((size_t)(o.i0 + 2 * c + j) * p.Hkv + o.h) * D + 4 * r;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float (&y)[4] = x[G * j + g];
            if (s[j] >= 0) load4<In>(p.value, src + 32 * g, y);
            else y[0] = y[1] = y[2] = y[3] = 0.f;
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        mn[q] = min_nan(min_nan(x[q][0], x[q][1]), min_nan(x[q][2], x[q][3]));
        mx[q] = fmaxf(fmaxf(x[q][0], x[q][1]), fmaxf(x[q][2], x[q][3]));
    }
    // over the pair's eight lanes: lane r ends with number r (d 64: r / 2)
    halve<Q / 2, true>(mn, 16, r & 4);
    halve<Q / 2, false>(mx, 16, r & 4);
    halve<Q / 4, true>(mn, 8, r & 2);
    halve<Q / 4, false>(mx, 8, r & 2);
    if constexpr (G == 4) {
        halve<1, true>(mn, 4, r & 1);
        halve<1, false>(mx, 4, r & 1);
    } else {
        mn[0] = min_nan(mn[0], __shfl_xor_sync(0xffffffffu, mn[0], 4));
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], 4));
    }
    const GroupScale gs = group_scale(mn[0], mx[0], by, rby);
    const float thr = 0.5f - warp_max(gs.slack);
    auto holder = [&](int q) { return 4 * (q * (8 / Q)) + c; };
    const uint32_t mine = pair_bits(gs.hs, gs.hz);
    uint32_t code[Q];                             // 16 bits
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const float A = __shfl_sync(0xffffffffu, gs.A, holder(q)), B = __shfl_sync(0xffffffffu, gs.B, holder(q));
        code[q] = kv4_codes(x[q], A, B, thr, by, __shfl_sync(0xffffffffu, mine, holder(q)));
    }
    // the same group's scale and zero of the pair's other token
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 16);
    auto block = [&](long long slot) {
        return static_cast<unsigned char*>(p.value_cache) + ((size_t)(slot >> sh) * p.Hkv + o.h) * head_bytes;
    };
    const int own = r / (8 / Q), oj = own / G, og = own % G;   // this lane's (token, group)
    const bool holds = r % (8 / Q) == 0;
    if (s[0] >= 0 && (s[0] & 1) == 0 && s[1] == s[0] + 1) {
        const int t = (int)s[0] & (p.bs - 1);
        unsigned char* blk = block(s[0]);
        uint32_t w[G];
#pragma unroll
        for (int g = 0; g < G; ++g) w[g] = code[g] | (code[G + g] << 16);
        store_words<G>(blk + 4 * F::v_word(t, 4 * r), w);
        if (holds) {                              // the first token's lanes store scales, the second's zeros
            uint32_t* par = reinterpret_cast<uint32_t*>(reinterpret_cast<__half*>(blk + F::codes(p.bs)) + F::v_par(t, og));
            if (oj == 0) par[0] = __byte_perm(mine, other, 0x5410u);
            else par[zeros / 2] = __byte_perm(other, mine, 0x7632u);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (s[j] < 0) continue;
        const int t = (int)s[j] & (p.bs - 1);
        unsigned char* blk = block(s[j]);
#pragma unroll
        for (int g = 0; g < G; ++g)
            reinterpret_cast<uint16_t*>(blk)[2 * F::v_word(t, 32 * g + 4 * r) + t % 2] = (uint16_t)code[G * j + g];
        if (holds && oj == j) {
            __half* par = reinterpret_cast<__half*>(blk + F::codes(p.bs)) + F::v_par(t, og);
            par[0] = gs.hs;
            par[zeros] = gs.hz;
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
