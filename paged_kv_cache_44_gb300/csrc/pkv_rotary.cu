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
// registers for all the rows it takes (every head uses the same ones).  The
// first rows of V, K and Q are requested before any is stored, and each next
// row before the one before it: 16,384 tokens of 64 / 8 heads of 128 into an
// E4M3 cache, 642 MB, 102 us (6.3 TB/s, 94% of a copy); with one row after the
// other 133.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

// Threads (rows side by side) and registers by the blocks they leave on an SM.
// 8,240 tokens of 28 / 4 heads and 16,384 of 64 / 8 into E4M3: 64 threads of at
// most 64 registers 28.5 and 102 us, of all they ask for (110) 28.6 and 117, of
// 48 (spills) 35.7 and 132; 128 threads 29.6 and 134, 32 29.3 and 118.  fp32
// rows need twice the registers for what is on its way: 63.0 us for 8,240 tokens
// of 32 / 8 heads with all they ask for, 85.7 with 64.
constexpr int kRotaryThreads = 64;

// 8 elements as they lie in memory, read as data that this kernel may overwrite
// (q_out, k_out may be the inputs)
template <typename In>
struct Raw8;
template <>
struct Raw8<F32> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* base, size_t i) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        a = p[0];
        b = p[1];
    }
    __device__ __forceinline__ void get(float v[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <>
struct Raw8<BF16> {
    uint4 r;
    __device__ __forceinline__ void load(const void* base, size_t i) {
        r = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    }
    __device__ __forceinline__ void get(float v[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
};

template <typename In, typename Cache, bool PAIRS_APART>
__global__ void __launch_bounds__(kRotaryThreads, In::bytes == 2 ? 16 : 1) rotary_kernel(const __grid_constant__ RotaryParams p, int chunks) {
    pdl_trigger();
    pdl_wait();
    const int lanes = blockDim.x / chunks;                          // rows at a time
    const int r0 = threadIdx.x / chunks, c = threadIdx.x - r0 * chunks;
    const bool turn = 16 * c < p.rot;
    const long long t = blockIdx.x;
    const long long pos = load_behind_wait(p.positions + t);
    long long slot = -1;
    if (p.key_cache != nullptr) slot = load_behind_wait(p.slot_mapping + t);
    if (pos < 0 || pos >= p.max_position) {      // a padding token, or one past the table
        if (pos >= 0 && threadIdx.x == 0) report(p.err, PKV_DEVERR_POSITION);
        return;
    }
    if (slot >= (long long)p.NB * p.bs) {
        if (threadIdx.x == 0) report(p.err, PKV_DEVERR_SLOT);
        slot = -1;
    }
    // one kind of row after the other: the two groups of 8 values this thread takes of a head, in `n` rows from
    // `in` to `out` and, where there is one, the cache row `pool`
    float cs[8], sn[8];
    auto rows = [&](Raw8<In> lo, Raw8<In> hi, const void* in, int n, bool turned, void* out, void* pool, float by) {
        const int e0 = turned && PAIRS_APART ? 8 * c : 16 * c, e1 = turned && PAIRS_APART ? p.rot / 2 + 8 * c : 16 * c + 8;
        Raw8<In> lo2, hi2;
        for (int r = r0; r < n; r += lanes) {
            if (r + lanes < n) {                 // the next row is on its way while this one is stored
                lo2.load(in, (size_t)(r + lanes) * p.d + e0);
                hi2.load(in, (size_t)(r + lanes) * p.d + e1);
            }
            float x[16];
            lo.get(x);
            hi.get(x + 8);
            if (turned) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int ia = PAIRS_APART ? k : 2 * k, ib = PAIRS_APART ? 8 + k : 2 * k + 1;
                    const float a = x[ia], b = x[ib];
                    x[ia] = __fsub_rn(__fmul_rn(a, cs[k]), __fmul_rn(b, sn[k]));
                    x[ib] = __fadd_rn(__fmul_rn(b, cs[k]), __fmul_rn(a, sn[k]));
                }
            }
            if (out != nullptr) {
                store8<In>(out, (size_t)r * p.d + e0, x, 1.f);
                store8<In>(out, (size_t)r * p.d + e1, x + 8, 1.f);
            }
            if (pool != nullptr) {
                store8<Cache>(pool, (size_t)r * p.d + e0, x, by);
                store8<Cache>(pool, (size_t)r * p.d + e1, x + 8, by);
            }
            lo = lo2;
            hi = hi2;
        }
    };
    constexpr int eb = In::bytes, cb = Cache::bytes;
    auto at = [](const void* base, long long i, int bytes) { return static_cast<const char*>(base) + i * bytes; };
    // the first rows of all three are requested before the first is stored
    const char* v_in = at(p.v, t * p.v_stride, eb);
    const char* k_in = at(p.k, t * p.k_stride, eb);
    const char* q_in = at(p.q, t * p.q_stride, eb);
    const int e0 = turn && PAIRS_APART ? 8 * c : 16 * c, e1 = turn && PAIRS_APART ? p.rot / 2 + 8 * c : 16 * c + 8;
    const bool write_v = p.Hv > 0 && slot >= 0;
    Raw8<In> v_lo, v_hi, k_lo, k_hi, q_lo, q_hi;
    if (turn) {
        load8<F32>(p.cos_sin, (size_t)pos * p.rot + 8 * c, cs);
        load8<F32>(p.cos_sin, (size_t)pos * p.rot + p.rot / 2 + 8 * c, sn);
    }
    if (write_v && r0 < p.Hv) {
        v_lo.load(v_in, (size_t)r0 * p.d + 16 * c);
        v_hi.load(v_in, (size_t)r0 * p.d + 16 * c + 8);
    }
    if (r0 < p.Hk) {
        k_lo.load(k_in, (size_t)r0 * p.d + e0);
        k_hi.load(k_in, (size_t)r0 * p.d + e1);
    }
    if (r0 < p.Hq) {
        q_lo.load(q_in, (size_t)r0 * p.d + e0);
        q_hi.load(q_in, (size_t)r0 * p.d + e1);
    }
    const long long row = slot * p.Hkv * p.d;
    if (write_v)
        rows(v_lo, v_hi, v_in, p.Hv, false, nullptr, const_cast<char*>(at(p.value_cache, row, cb)), p.v_scale);
    if (p.Hk > 0)
        rows(k_lo, k_hi, k_in, p.Hk, turn, p.k_out ? const_cast<char*>(at(p.k_out, t * p.k_out_stride, eb)) : nullptr,
             slot >= 0 ? const_cast<char*>(at(p.key_cache, row, cb)) : nullptr, p.k_scale);
    if (p.Hq > 0)
        rows(q_lo, q_hi, q_in, p.Hq, turn, const_cast<char*>(at(p.q_out, t * p.q_out_stride, eb)), nullptr, 1.f);
}

template <typename In, typename Cache>
cudaError_t launch_rotary_pairs(const RotaryParams& p, int chunks, dim3 g, dim3 b, cudaStream_t st) {
    return p.interleaved ? launch_pdl(rotary_kernel<In, Cache, false>, g, b, 0, st, p, chunks)
                         : launch_pdl(rotary_kernel<In, Cache, true>, g, b, 0, st, p, chunks);
}

template <typename In>
cudaError_t launch_rotary_in(const RotaryParams& p, pkv_dtype cache_dt, int chunks, dim3 g, dim3 b, cudaStream_t st) {
    switch (cache_dt) {
        case PKV_F32: return launch_rotary_pairs<In, F32>(p, chunks, g, b, st);
        case PKV_BF16: return launch_rotary_pairs<In, BF16>(p, chunks, g, b, st);
        case PKV_FP8_E4M3: return launch_rotary_pairs<In, E4M3>(p, chunks, g, b, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, pkv_dtype in_dt, pkv_dtype cache_dt, cudaStream_t st) {
    const int rows = p.Hq + p.Hk + p.Hv;
    if (p.T == 0 || rows == 0) return cudaSuccess;
    const int chunks = p.d / 16, most = kRotaryThreads / chunks, widest = p.Hq > p.Hkv ? p.Hq : p.Hkv;
    const int lanes = widest < most ? widest : most;
    const dim3 g(p.T), b(chunks * lanes);
    return in_dt == PKV_F32 ? launch_rotary_in<F32>(p, cache_dt, chunks, g, b, st) : launch_rotary_in<BF16>(p, cache_dt, chunks, g, b, st);
}

}  // namespace pkv
