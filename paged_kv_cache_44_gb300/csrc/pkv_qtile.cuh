// Work units of paged attention over query chunks, shared by the kernels
// that compute it and by the merge of their partitions.
//
// A sequence s with n tokens computes its last q_len tokens as queries
// (a chunk of prefill, or the tokens a speculative decoder proposes).  For
// K/V head kvh its rows are the pairs (query i, head kvh * g + j), row
// r = i * g + j, cut into tiles of tile_rows rows; a tile needs the keys up to
// its last query's position n - q_len + i_last, cut into partitions of P
// tokens.  Unit ids run partition-major, then sequence, K/V head, row tile,
// so the tiles of one key range are claimed together and share the K/V
// reads in L2.  With a sliding window (WIN) the keys of a tile are numbered
// without the blocks none of its queries sees (window_span, from the window
// of its first query): key_end, the partitions and k0, k1 are of that
// numbering, in which the keys a query at position pos does not see are
// those from `sinks` to pos - window - gap and those past pos - gap.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_tc_common.cuh"

namespace pkv {

struct __align__(16) QTile {
    int s, kvh, rt, part;      // sequence, K/V head, row tile, key partition
    int k0, k1;                // key tokens [k0, k1)
    int n, ql;                 // sequence length, queries in the chunk
    int q0, np, rows;          // first query token, partitions of the tile, rows of the sequence
    int first;                 // WIN: the first token of the window of the tile's first query
    WindowSpan span;           // WIN: the tokens left out
};

// Keys of a row tile: how many its queries reach, in window_span's numbering with a window.
__device__ __forceinline__ int qtile_keys(const DecodeParams& p, int n, int ql, int first_row, int last_row,
                                          int& first, WindowSpan& span) {
    const int key_end = n - ql + last_row / p.g + 1;
    if (p.window <= 0) return key_end;
    first = n - ql + first_row / p.g - p.window + 1;
    span = window_span(first, p.sinks, p.bs);
    return key_end - span.gap;
}

// Unit id -> coordinates; false for ids that name no work.  A sequence whose
// length exceeds the host bound, whose query count is outside [0, n] or
// above the host's max_q, or whose queries leave [0, T) is skipped and
// reported once.  rt_max = ceil(max_q * g / tile_rows) tiles per (sequence, K/V
// head).
template <bool WIN>
__device__ __forceinline__ bool qtile_of(const DecodeParams& p, const int32_t* query_start, int T, int max_q,
                                         unsigned long long u, int rt_max, int tile_rows,
                                         QTile& x) {
    const unsigned long long per_part = (unsigned long long)p.S * p.Hkv * rt_max;
    x.part = (int)(u / per_part);
    const unsigned long long rem = u - (unsigned long long)x.part * per_part;
    x.s = (int)(rem / ((unsigned long long)p.Hkv * rt_max));
    const int r2 = (int)(rem - (unsigned long long)x.s * p.Hkv * rt_max);
    x.kvh = r2 / rt_max;
    x.rt = r2 - x.kvh * rt_max;
    const int n = __ldg(p.context_lens + x.s);
    x.q0 = __ldg(query_start + x.s);
    x.ql = __ldg(query_start + x.s + 1) - x.q0;
    if (n < 0 || n > p.max_ctx || x.ql < 0 || x.ql > n || x.ql > max_q || x.q0 < 0 || x.q0 + x.ql > T) {
        if (x.part == 0 && r2 == 0) report(p.err, PKV_DEVERR_QUERY_LEN);
        return false;
    }
    x.n = n;
    x.rows = x.ql * p.g;
    if (x.rt * tile_rows >= x.rows) return false;
    const int last_row = min(x.rt * tile_rows + tile_rows - 1, x.rows - 1);
    int key_end;
    if constexpr (WIN) key_end = qtile_keys(p, n, x.ql, x.rt * tile_rows, last_row, x.first, x.span);
    else key_end = n - x.ql + last_row / p.g + 1;
    x.np = (key_end + p.P - 1) / p.P;
    if (x.part >= x.np) return false;
    x.k0 = x.part * p.P;
    x.k1 = min(key_end, x.k0 + p.P);
    return true;
}

// One warp copies (query, head) rows of Q into a 128-byte-swizzled
// shared-memory tile (a region of ROWS rows per 64 values): rows [r0, r1) of
// the tile whose first row is `row` of the chunk that starts at query token
// q0; rows past `here` become zeros.  Every copy is issued before the first is
// waited for, and a lane steps from row to row (RPI rows on) without dividing:
// of the 16 x 512-query chunks under a window of 1,024 the divisions and four
// round trips per tile were 30% of the time (256.8 -> 180.3 us).  The caller
// waits (cp.async.wait_all), fences and signals.
template <int D, int ROWS>
__device__ __forceinline__ void load_q_rows(const DecodeParams& p, int q0, int kvh, int row, int r0, int r1, int here,
                                            uint32_t dst) {
    constexpr int CH = 2 * D / 16, RPI = 32 / CH;        // 16-byte chunks per row, rows per request
    const int lane = threadIdx.x & 31, c = lane % CH;
    int r = r0 + lane / CH;
    const int qi = (row + r) / p.g;
    int hh = row + r - qi * p.g;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                               ((size_t)(q0 + qi) * p.Hq + kvh * p.g + hh) * D + c * 8;
    const size_t next_query = (size_t)(p.Hq - p.g) * D;
    dst += (c >> 3) * (ROWS * 128);
#pragma unroll 4
    for (; r < r1; r += RPI) {
        const uint32_t to = dst + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        if (r < here) {
            tc::cp_async16(to, src);
        } else {
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to), "r"(0u) : "memory");
        }
        hh += RPI;
        src += RPI * D;
        while (hh >= p.g) {
            hh -= p.g;
            src += next_query;
        }
    }
}

// 32 values of one output row, times f, as bf16 at `dst`.  Every lane of a warp
// stores to a row of its own, so a store's cost is its sectors: 32-byte stores
// (wide: dst is 32-byte aligned) write whole ones, 16-byte ones halves.
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const uint32_t (&o)[32], float f, bool wide) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = tc::pack2<false>(__uint_as_float(o[16 * k + 2 * j]) * f, __uint_as_float(o[16 * k + 2 * j + 1]) * f);
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * k), "r"(w[0]),
                         "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        } else {
            reinterpret_cast<uint4*>(dst + 16 * k)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst + 16 * k)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

// The same 32 values as fp32, unscaled: a line of a partition's partial result.
__device__ __forceinline__ void store_part32(float* dst, const uint32_t (&o)[32], bool wide) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 8 * k), "r"(o[8 * k]),
                         "r"(o[8 * k + 1]), "r"(o[8 * k + 2]), "r"(o[8 * k + 3]), "r"(o[8 * k + 4]), "r"(o[8 * k + 5]),
                         "r"(o[8 * k + 6]), "r"(o[8 * k + 7])
                         : "memory");
        } else {
            reinterpret_cast<uint4*>(dst + 8 * k)[0] = make_uint4(o[8 * k], o[8 * k + 1], o[8 * k + 2], o[8 * k + 3]);
            reinterpret_cast<uint4*>(dst + 8 * k)[1] =
                make_uint4(o[8 * k + 4], o[8 * k + 5], o[8 * k + 6], o[8 * k + 7]);
        }
    }
}

}  // namespace pkv
