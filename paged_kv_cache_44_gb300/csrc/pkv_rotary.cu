// rotary_kv_write: what stands between a layer's projections and its
// attention, in one pass.  The first rot values of every query and key head
// are rotated by the token's position, Q and K go on to the attention, and K
// and V go to the token's slot in the cache's format.
//
// "LLM推論の基礎とvLLMの内部", section 4: a new token's K/V occupies one slot
// (block, offset) of the pool; section 2: an fp8 cache stores one byte per
// element.
//
// A pair (a, b) of a head becomes (a c - b s, b c + a s) with the table's
// c, s of (position, pair): two products and a sum, each rounded to fp32, so
// that the result does not depend on what the compiler fuses.  The fp32
// result is rounded once to each output's format.
//
// Bound by HBM: 3 flops per 4 bytes.  One block per token, one thread per 16
// values of a head: 8 pairs, whose sines and cosines stay in the thread's
// registers for all the rows it takes (every head uses the same ones).  A
// thread loads two rows before it stores the first.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kRotaryThreads = 128;

// 8 elements, read as data that this kernel may overwrite (q_out, k_out may be the inputs)
template <typename In>
__device__ __forceinline__ void load8_rw(const void* base, size_t i, float v[8]);
template <>
__device__ __forceinline__ void load8_rw<F32>(const void* base, size_t i, float v[8]) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8_rw<BF16>(const void* base, size_t i, float v[8]) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}

template <typename In, typename Cache>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    pdl_trigger();
    pdl_wait();
    const int chunks = p.d / 16, lanes = blockDim.x / chunks;       // rows at a time
    const int c = threadIdx.x % chunks, r0 = threadIdx.x / chunks;
    const int rows = p.Hq + p.Hk + p.Hv;
    const bool turn = 16 * c < p.rot;
    // the two groups of 8 values this thread takes of a row
    const int at = turn && !p.interleaved ? 8 * c : 16 * c;
    const int next = turn && !p.interleaved ? p.rot / 2 : 8;
    const long long t = blockIdx.x;
    const long long pos = load_behind_wait(p.positions + t);
    if (pos < 0 || pos >= p.max_position) {      // a padding token, or one past the table
        if (pos >= 0 && threadIdx.x == 0) report(p.err, PKV_DEVERR_POSITION);
        return;
    }
    long long slot = -1;
    if (p.key_cache != nullptr) {
        slot = load_behind_wait(p.slot_mapping + t);
        if (slot >= (long long)p.NB * p.bs) {
            if (threadIdx.x == 0) report(p.err, PKV_DEVERR_SLOT);
            slot = -1;
        }
    }
    float cs[8], sn[8];
    if (turn) {
        load8<F32>(p.cos_sin, (size_t)pos * p.rot + 8 * c, cs);
        load8<F32>(p.cos_sin, (size_t)pos * p.rot + p.rot / 2 + 8 * c, sn);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) cs[k] = 1.f, sn[k] = 0.f;
    }
    auto load = [&](int r, float (&x)[16]) {
        const void* base = p.q;
        size_t i = (size_t)t * p.q_stride + (size_t)r * p.d;
        if (r >= p.Hq + p.Hk) {
            base = p.v;
            i = (size_t)t * p.v_stride + (size_t)(r - p.Hq - p.Hk) * p.d;
        } else if (r >= p.Hq) {
            base = p.k;
            i = (size_t)t * p.k_stride + (size_t)(r - p.Hq) * p.d;
        }
        load8_rw<In>(base, i + (r >= p.Hq + p.Hk ? 16 * c : at), x);
        load8_rw<In>(base, i + (r >= p.Hq + p.Hk ? 16 * c + 8 : at + next), x + 8);
    };
    auto store = [&](int r, float (&x)[16]) {
        const bool is_v = r >= p.Hq + p.Hk;
        if (turn && !is_v) {
            if (p.interleaved) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = x[2 * k], b = x[2 * k + 1];
                    x[2 * k] = __fsub_rn(__fmul_rn(a, cs[k]), __fmul_rn(b, sn[k]));
                    x[2 * k + 1] = __fadd_rn(__fmul_rn(b, cs[k]), __fmul_rn(a, sn[k]));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = x[k], b = x[8 + k];
                    x[k] = __fsub_rn(__fmul_rn(a, cs[k]), __fmul_rn(b, sn[k]));
                    x[8 + k] = __fadd_rn(__fmul_rn(b, cs[k]), __fmul_rn(a, sn[k]));
                }
            }
        }
        const int e0 = is_v ? 16 * c : at, e1 = is_v ? 16 * c + 8 : at + next;
        if (r < p.Hq) {
            const size_t o = (size_t)t * p.q_out_stride + (size_t)r * p.d;
            store8<In>(p.q_out, o + e0, x, 1.f);
            store8<In>(p.q_out, o + e1, x + 8, 1.f);
            return;
        }
        const int h = is_v ? r - p.Hq - p.Hk : r - p.Hq;
        if (!is_v && p.k_out != nullptr) {
            const size_t o = (size_t)t * p.k_out_stride + (size_t)h * p.d;
            store8<In>(p.k_out, o + e0, x, 1.f);
            store8<In>(p.k_out, o + e1, x + 8, 1.f);
        }
        if (slot >= 0) {
            const size_t o = ((size_t)slot * p.Hkv + h) * p.d;
            void* pool = is_v ? p.value_cache : p.key_cache;
            const float by = is_v ? p.v_scale : p.k_scale;
            store8<Cache>(pool, o + e0, x, by);
            store8<Cache>(pool, o + e1, x + 8, by);
        }
    };
    for (int r = r0; r < rows; r += 2 * lanes) {
        float x[16], y[16];
        load(r, x);
        const bool two = r + lanes < rows;
        if (two) load(r + lanes, y);
        store(r, x);
        if (two) store(r + lanes, y);
    }
}

template <typename In>
cudaError_t launch_rotary_in(const RotaryParams& p, pkv_dtype cache_dt, dim3 g, dim3 b, cudaStream_t st) {
    switch (cache_dt) {
        case PKV_F32: return launch_pdl(rotary_kernel<In, F32>, g, b, 0, st, p);
        case PKV_BF16: return launch_pdl(rotary_kernel<In, BF16>, g, b, 0, st, p);
        case PKV_FP8_E4M3: return launch_pdl(rotary_kernel<In, E4M3>, g, b, 0, st, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, pkv_dtype in_dt, pkv_dtype cache_dt, cudaStream_t st) {
    const int rows = p.Hq + p.Hk + p.Hv;
    if (p.T == 0 || rows == 0) return cudaSuccess;
    // rows side by side: as many as leave no thread without one in the last round, e.g. 36 rows of 8 threads
    // in three rounds of 12
    const int chunks = p.d / 16, most = kRotaryThreads / chunks;
    const int rounds = (rows + most - 1) / most, lanes = (rows + rounds - 1) / rounds;
    const dim3 g(p.T), b(chunks * lanes);
    return in_dt == PKV_F32 ? launch_rotary_in<F32>(p, cache_dt, g, b, st) : launch_rotary_in<BF16>(p, cache_dt, g, b, st);
}

}  // namespace pkv
