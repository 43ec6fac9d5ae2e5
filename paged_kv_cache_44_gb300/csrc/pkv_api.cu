// C ABI of libpkv.so: host-side validation, workspace planning, dispatch.
// Nothing here allocates, synchronises or reads device memory.
#include <math.h>
#include <string.h>

#include <cudaTypedefs.h>

#include <mutex>

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_kv4.cuh"
#include "pkv_units.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Units of work (sequence x K/V head x head-set x partition) the default
// partition size aims for, counted as if every sequence had the maximum
// length: about four per worker warp of a full GB300 (152 SMs x 8 warps),
// so that dynamic scheduling evens out ragged lengths and the last units to
// finish are short next to the whole launch.  It depends on no dtype, so the
// workspace size and the launch always agree.
constexpr long long kTargetUnits = 152LL * 8 * 4;
constexpr int kMinDefaultPartition = 512;
// A small launch: fewer than about 1.3 units per worker warp of a full
// GB300 (152 SMs x 7 bf16 workers) even if every sequence had the maximum
// length.
constexpr long long kSmallLaunchUnits = 152LL * 9;
constexpr int kMinSmallPartition = 256;
constexpr long long kPrefillTargetUnits = 152LL * 4;
constexpr int kPrefillTileRows = 128;       // (query, head) rows per tcgen05 tile
constexpr int kHeadSet = 8;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool finite_pos(float x) { return isfinite(x) && x > 0.f; }

bool decode_shape_ok(int S, int Hq, int Hkv, int d, int bs, int max_ctx) {
    return S >= 0 && S <= 65535 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && (d == 64 || d == 128) &&
           (bs == 16 || bs == 32) && max_ctx >= 0;
}

// Partition size in tokens (0 = no split) for a request; -1 if invalid.
int resolve_partition(int S, int Hq, int Hkv, int d, int bs, int max_ctx, int req) {
    if (!decode_shape_ok(S, Hq, Hkv, d, bs, max_ctx)) return -1;
    if (req > 0) return req % bs == 0 ? req : -1;
    if (req == -1) return 0;
    if (req != 0) return -1;
    const long long sets = (long long)S * Hkv * ((Hq / Hkv + kHeadSet - 1) / kHeadSet);
    if (sets == 0 || max_ctx <= kMinDefaultPartition) return 0;
    int P = 1 << 20;
    while (P > kMinDefaultPartition && sets * ((max_ctx + P - 1) / P) < kTargetUnits) P >>= 1;
    // A small launch gives each worker warp about one long unit, streamed at
    // a single warp's latency-bound rate, and the longest units set the
    // launch's length: take the largest partition, in steps of 128 tokens
    // down to 256, that gives that many units at the maximum length.
    // 64 sequences of 512..4096 tokens, 2 K/V heads: 384 instead of 512,
    // decode 35.3-35.4 vs 37.5-37.9 us (256: 38.1, 320: 35.6, 448: 36.0).
    while (P > kMinSmallPartition && sets * ((max_ctx + P - 1) / P) < kSmallLaunchUnits) P -= 128;
    if (P >= max_ctx) return 0;
    return P;
}

// The same for the windowed and the 4-bit decode (keys: the most tokens a
// sequence reads).  A launch too small to fill the GPU is split further, down
// to 64 tokens: one warp's pace (a 4-bit stage of 64 tokens alone takes about
// 2 us), not bandwidth, is then the launch's length.  In 64- / 128- /
// 256-token partitions and in one: a 4-bit sequence of 500 tokens 12.4 / 14.4
// / 16.5 / 20.7 us; a window of 1,000 bf16 tokens over 8 sequences of 4 K/V
// heads 14.6 / 17.0 / 20.6 / 55.5.  Beyond 48 partitions a row's merge costs
// what that saves (one 4-bit sequence of 32,768 tokens: 69 us in 64, 45 in
// 128, 28.7 in 256; a window of 4,100 bf16 tokens: 18.5 and 18.7).
// The windowed fp32 decode, 1.8 us per 16-token stage, goes down to 32 while
// every unit has a worker (152 SMs x 6): one sequence of 400 tokens, 4 K/V
// heads, in 32 / 64 / 128: 11.8 / 15.4 / 22.4 us; eight of 1,000 (1,024
// units) 20.8 / 17.2 / 23.7.
//
// A bf16 or E4M3 launch of up to three units per worker is a few rounds of
// whole partitions, so it takes a partition that fills whole rounds: under a
// window (most sequences fill it) as many equal ones per sequence as all
// workers take at once; without one sets * keys / (1.6 workers) tokens
// (lengths then reach down from the longest; at half of it on average one
// round is four fifths full).  The plain rule's partition and this one: 32
// E4M3 sequences of 256..16,384 tokens, scored, 78 us (512) and 67 (800); 16
// bf16 ones 68 and 58 (640); 64 E4M3 ones under a window of 4,096: 54 and 50
// (704); 32 bf16 ones 49 (384) and 42 (544); 256 of 1,056 tokens 93 (512) and
// 88 (whole), in E4M3 73 and 56.  Lengths of 2,000..6,000, two thirds of the
// longest on average, lose: 48 E4M3 sequences 53 and 56.5.  In 4 bits it gains
// 12% on the first and loses 15% on 64 sequences of 512..4,096, so it is not
// taken there.
constexpr int kMaxSmallSplits = 48, kMinWavePartition = 384, kMaxWavePartition = 1024;
struct SplitRule {
    int smallest;
    long long units;
    int workers;                          // of a full GB300; 0: no partition by rounds
};
constexpr SplitRule kSplitBf16{64, kSmallLaunchUnits, 152 * 7}, kSplitE4m3{64, kSmallLaunchUnits, 152 * 11},
    kSplitKv4{64, kSmallLaunchUnits, 0}, kSplitF32{32, 152LL * 6, 0};
int resolve_split(int S, int Hq, int Hkv, int d, int bs, int max_ctx, int keys, int req, SplitRule rule) {
    const int P = resolve_partition(S, Hq, Hkv, d, bs, keys, req);
    if (P < 0 || req != 0 || keys <= rule.smallest) return P;
    const long long sets = (long long)S * Hkv * ((Hq / Hkv + kHeadSet - 1) / kHeadSet);
    if (P >= kMinWavePartition && sets * ((keys + P - 1) / P) < 3LL * rule.workers) {
        const long long parts = rule.workers / sets;
        const long long wave = keys < max_ctx ? (parts > 0 ? keys / parts : 0) : sets * keys * 10 / (rule.workers * 16LL);
        const int p = (int)((min(wave, 2LL * kMaxWavePartition) + 31) / 32 * 32);
        if (p >= keys) return 0;
        if (p >= kMinWavePartition && p <= kMaxWavePartition) return p;
    }
    int p = P > 0 ? P : keys;
    while (p > rule.smallest) {
        const int half = max(rule.smallest, (p / 2 + 31) / 32 * 32);
        const int n = (keys + half - 1) / half;
        if (half >= p || sets * n > rule.units || n > kMaxSmallSplits) break;
        p = half;
    }
    return p < keys ? p : 0;
}

// The last, partial partition of a sequence is cut into chunks of Q tokens
// (a quarter partition, a multiple of 32 tokens and so of the block size):
// those chunks are the last units a launch hands out, so the launch ends on
// small units instead of on whichever partial partitions happened to be large.
int tail_chunk(int P) { return P >= 128 ? (P / 4) / 32 * 32 : P; }

// Full partitions held back into chunks at a long sequence's end
// (num_partitions), for E4M3 caches on the tensor-core kernel: a worker
// streams E4M3 at the pace of its own arithmetic (about 17 tokens/us, a
// full 1024-token unit lasts ~60 us), so the units claimed last decide when
// the launch ends, and small ones end it sooner.  On bf16 caches the same
// layout was slower (more units and partial results for the same tail).
constexpr int kTailHold = 1;
int tail_hold(pkv_dtype cache_dtype, bool tensor_cores) {
    return cache_dtype == PKV_FP8_E4M3 && tensor_cores ? kTailHold : 0;
}

// The 4-bit decode: partitions held back where the launch has fewer than
// three units per worker (152 SMs x 11), so that its last round is made of
// chunks.  128 sequences (28 / 4 heads of 128) under a window of 2,048 and 4
// sinks: 53.3 us held, 56.6 not (floor 24.0); 64 (12 / 2 heads) of 512..4,096
// tokens: 26.8 and 27.9; with five rounds (256 sequences, 28 / 4 heads, of
// 1..4,096) the small units cost more than they even out: 86.5 and 81.9.
int kv4_hold(int S, int Hq, int Hkv, int keys, int P) {
    const long long sets = (long long)S * Hkv * ((Hq / Hkv + kHeadSet - 1) / kHeadSet);
    return P > 0 && sets * ((keys + P - 1) / P) < 3LL * 152 * 11 ? kTailHold : 0;
}

// Partial results per row for lengths up to max_ctx with `hold` held-back
// partitions: the count (num_partitions) grows with n between multiples of
// P, so its largest value is at max_ctx, just below the last multiple of P,
// or just below the length from which partitions are held back.
int max_partitions(int max_ctx, int P, int Q, int hold) {
    int m = num_partitions(max_ctx, P, Q, hold);
    const int F = max_ctx / P;
    if (F >= 1) m = max(m, num_partitions(F * P - 1, P, Q, hold));
    m = max(m, num_partitions(min(max_ctx, kTailHoldMin * P - 1), P, Q, hold));
    return m > 1 ? m : 1;
}

DecodePlan make_plan(int S, int Hq, int d, int max_ctx, int P) {
    DecodePlan pl{};
    pl.P = P;
    pl.Q = P;
    pl.Pmax = P > 0 ? (max_ctx > 0 ? (max_ctx + P - 1) / P : 1) : 1;
    pl.Pmax_plain = pl.Pmax;
    pl.split = P > 0 && pl.Pmax > 1;
    pl.bytes = kWorkspaceHeaderBytes;
    if (!pl.split) return pl;
    pl.Q = tail_chunk(P);
    // the workspace fits both layouts; each launch uses its own row stride
    pl.Pmax_plain = max_partitions(max_ctx, P, pl.Q, 0);
    pl.Pmax = max(pl.Pmax_plain, max_partitions(max_ctx, P, pl.Q, kTailHold));
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t units = (size_t)S * Hq * pl.Pmax;
    pl.ml_offset = kWorkspaceHeaderBytes;
    pl.acc_offset = up(pl.ml_offset + units * 2 * sizeof(float));
    pl.bytes = up(pl.acc_offset + units * d * sizeof(float));
    return pl;
}

// Partition a launch uses.  With the library's choice (request 0), an E4M3
// cache on the tensor-core kernel takes twice the planned partition where
// that still leaves half of kTargetUnits units: an E4M3 worker streams at
// the pace of its own arithmetic and every unit has a fixed cost (its
// claim, its first stage in flight, its partial result and merge row), so
// fewer, longer units end the launch sooner.  Measured on the fp8 workloads
// (128 sequences of 256..16384 tokens, bs 16 and 32): 2048-token partitions
// 1.1-1.5% faster than 1024, 3072 and 4096 slower.  The workspace is planned
// for the dtype-independent partition; a partition twice as large never
// needs more partial results per row, and the larger one is taken only when
// the plan's row stride holds them.
int launch_partition(const DecodePlan& pl, int S, int Hq, int Hkv, int max_ctx, int req, bool e4m3_tc) {
    if (req != 0 || !pl.split || !e4m3_tc) return pl.P;
    const int P2 = 2 * pl.P;
    const long long sets = (long long)S * Hkv * ((Hq / Hkv + kHeadSet - 1) / kHeadSet);
    if (P2 >= max_ctx || sets * ((max_ctx + P2 - 1) / P2) < kTargetUnits / 2) return pl.P;
    return max_partitions(max_ctx, P2, tail_chunk(P2), kTailHold) <= pl.Pmax ? P2 : pl.P;
}

// Fills the partition fields of a launch: P, its chunk Q, the row stride.
void set_partitions(DecodeParams& p, const DecodePlan& pl, int Pl, int no_split_P, int hold) {
    p.P = Pl > 0 ? Pl : no_split_P;      // no split: one partition covers every token
    p.Q = Pl <= 0 ? p.P : (Pl == pl.P ? pl.Q : tail_chunk(Pl));
    p.hold = hold;
    p.Pmax = hold ? pl.Pmax : pl.Pmax_plain;
}

// The bytes of a workspace that a call may lay its partial results out in.
// One that holds no header is none: then the size is the caller's mistake.
size_t workspace_room(const void* workspace, size_t workspace_bytes) {
    return workspace && workspace_bytes >= kWorkspaceHeaderBytes ? workspace_bytes : SIZE_MAX;
}

// The library's partition P where `room` bytes hold its plan, else the next
// larger one of which they do (0: no split).  The plan's size does not grow
// with the lengths, sequences or queries alone (few of them are split
// further), so a workspace made for the largest call of a loop may be short
// of a smaller one's choice by a few partitions.  bytes(P): the plan's size.
template <typename Bytes>
int fit_partition(int P, int keys, int req, size_t room, Bytes bytes) {
    if (req != 0) return P;
    while (P > 0 && bytes(P) > room) {
        const long long next = (P + (P / 8 > 32 ? P / 8 : 32) + 31LL) / 32 * 32;
        P = next < keys ? (int)next : 0;
    }
    return P;
}

// A window or sinks beyond the longest sequence are as good as its length
// (kept small so that the kernels' sums of them stay in 32 bits).
void clamp_window(int max_ctx, int& window, int& sinks) {
    if (window > max_ctx) window = max_ctx > 0 ? max_ctx : 1;
    if (sinks > max_ctx) sinks = max_ctx;
}

// Tokens of the longest sequence a decode reads (max_ctx when window is 0).
int decode_keys(int bs, int max_ctx, int window, int sinks) {
    return window > 0 ? window_bound(max_ctx, window, sinks, bs, 1) : max_ctx;
}

// The partial results' place in the workspace and its scheduling counters.
void set_workspace(DecodeParams& p, const DecodePlan& pl, void* workspace, size_t workspace_bytes) {
    char* ws = static_cast<char*>(workspace);
    if (pl.split) {
        p.sched = reinterpret_cast<unsigned*>(ws);
        p.part_ml = reinterpret_cast<float*>(ws + pl.ml_offset);
        p.part_acc = reinterpret_cast<float*>(ws + pl.acc_offset);
    } else if (workspace && workspace_bytes >= kWorkspaceHeaderBytes && aligned16(workspace)) {
        p.sched = reinterpret_cast<unsigned*>(workspace);
    }
}

// Workspace of a scored decode: its (max, sum) pairs are always there, and
// the logits of every token behind the partial results.
struct ScoredPlan {
    DecodePlan pl;
    size_t ml_offset, logits_offset, bytes;
};
ScoredPlan make_scored_plan(int S, int Hq, int Hkv, int d, int max_tokens, int P) {
    ScoredPlan sp{};
    sp.pl = make_plan(S, Hq, d, max_tokens, P);
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const int g = Hq / Hkv;
    const size_t sets = (size_t)S * Hkv * ((g + kHeadSet - 1) / kHeadSet);
    sp.ml_offset = sp.pl.split ? sp.pl.ml_offset : kWorkspaceHeaderBytes;
    sp.logits_offset = sp.pl.split ? sp.pl.bytes : up(sp.ml_offset + (size_t)S * Hq * 2 * sizeof(float));
    sp.bytes = up(sp.logits_offset + sets * max_tokens * score_width(g) * sizeof(float));
    return sp;
}

bool overlap(const void* a, const void* b, size_t na, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

pkv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

int num_sms_current() {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
    std::lock_guard<std::mutex> g(mu);
    if (cache[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
        cache[dev] = n;
    }
    return cache[dev];
}

}  // namespace

CUcontext current_context() {
    static std::once_flag once;
    static PFN_cuCtxGetCurrent_v4000 fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 4000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(f);
    });
    CUcontext ctx = nullptr;
    if (fn == nullptr || fn(&ctx) != CUDA_SUCCESS) return nullptr;
    return ctx;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

const char* pkv_status_string(pkv_status st) {
    switch (st) {
        case PKV_OK: return "ok";
        case PKV_ERR_INVALID_ARG: return "invalid argument";
        case PKV_ERR_UNSUPPORTED: return "unsupported dtype or shape";
        case PKV_ERR_WORKSPACE: return "workspace missing or too small";
        case PKV_ERR_CUDA: return "CUDA launch failed";
    }
    return "unknown status";
}

const char* pkv_version(void) { return "pkv 0.1.0 sm_103a"; }

pkv_status pkv_paged_kv_write(const void* key, const void* value, pkv_dtype in_dtype, void* key_cache,
                              void* value_cache, pkv_dtype cache_dtype, const int64_t* slot_mapping, int T,
                              int NB, int bs, int Hkv, int d, float k_scale, float v_scale, int32_t* err_word,
                              pkv_stream_t stream) {
    if (T < 0 || NB < 1 || bs < 1 || Hkv < 1 || d < 8) return PKV_ERR_INVALID_ARG;
    if (in_dtype != PKV_F32 && in_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (cache_dtype != PKV_F32 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3)
        return PKV_ERR_UNSUPPORTED;
    if (d % 8 != 0 || d > 512) return PKV_ERR_UNSUPPORTED;
    if (cache_dtype == PKV_FP8_E4M3 && (!finite_pos(k_scale) || !finite_pos(v_scale))) return PKV_ERR_INVALID_ARG;
    if ((long long)NB * bs > (1LL << 40)) return PKV_ERR_INVALID_ARG;
    if (T == 0) return PKV_OK;
    if (!key || !value || !key_cache || !value_cache || !slot_mapping) return PKV_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_INVALID_ARG;
    WriteParams p{};
    p.key = key; p.value = value; p.key_cache = key_cache; p.value_cache = value_cache;
    p.slot_mapping = slot_mapping; p.err = err_word;
    p.T = T; p.NB = NB; p.bs = bs; p.Hkv = Hkv; p.d = d; p.k_scale = k_scale; p.v_scale = v_scale;
    return from_cuda(launch_write(p, in_dtype, cache_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int pkv_decode_partition_size(int S, int Hq, int Hkv, int d, int bs, int max_context_len, int partition_size) {
    return resolve_partition(S, Hq, Hkv, d, bs, max_context_len, partition_size);
}

int pkv_decode_launch_partition_size(int S, int Hq, int Hkv, int d, int bs, int NB, int max_context_len,
                                     int partition_size, pkv_dtype q_dtype, pkv_dtype cache_dtype, int kernel) {
    if (kernel < PKV_DECODE_AUTO || kernel > PKV_DECODE_TENSOR_CORES || NB < 1) return -1;
    if (q_dtype != PKV_F32 && q_dtype != PKV_BF16) return -1;
    if (cache_dtype != PKV_F32 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3) return -1;
    const int P = resolve_partition(S, Hq, Hkv, d, bs, max_context_len, partition_size);
    if (P < 0) return -1;
    const bool tc_ok = decode_tc_supports(q_dtype, cache_dtype, d, bs, NB);
    if (kernel == PKV_DECODE_TENSOR_CORES && !tc_ok) return -1;      // the decode would refuse it
    const bool use_tc = kernel != PKV_DECODE_CUDA_CORES && tc_ok;
    const DecodePlan pl = make_plan(S, Hq, d, max_context_len, P);
    return launch_partition(pl, S, Hq, Hkv, max_context_len, partition_size, use_tc && cache_dtype == PKV_FP8_E4M3);
}

size_t pkv_decode_workspace_size(int S, int Hq, int Hkv, int d, int bs, int max_context_len, int partition_size) {
    const int P = resolve_partition(S, Hq, Hkv, d, bs, max_context_len, partition_size);
    if (P < 0) return 0;
    return make_plan(S, Hq, d, max_context_len, P).bytes;
}

}  // extern "C"

namespace pkv {

pkv_status check_decode_args(const void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                             const void* value_cache, pkv_dtype cache_dtype, const int32_t* block_tables, int MB,
                             const int32_t* context_lens, int S, int max_context_len, int Hq, int Hkv, int d,
                             int bs, int NB, float scale, float k_scale, float v_scale, int partition_size,
                             int kernel) {
    if (S < 0 || MB < 1 || NB < 1 || Hkv < 1 || Hq < 1 || max_context_len < 0) return PKV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_F32 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (cache_dtype != PKV_F32 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3)
        return PKV_ERR_UNSUPPORTED;
    if (!(d == 64 || d == 128) || !(bs == 16 || bs == 32)) return PKV_ERR_UNSUPPORTED;
    if (S > 65535) return PKV_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)MB * bs) return PKV_ERR_INVALID_ARG;
    if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if (cache_dtype == PKV_FP8_E4M3 && (!finite_pos(k_scale) || !finite_pos(v_scale))) return PKV_ERR_INVALID_ARG;
    if (partition_size < -1 || (partition_size > 0 && partition_size % bs != 0)) return PKV_ERR_INVALID_ARG;
    if (kernel < 0 || kernel > 2) return PKV_ERR_INVALID_ARG;
    if (S == 0) return PKV_OK;
    if (!out || !query || !key_cache || !value_cache || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u))
        return PKV_ERR_INVALID_ARG;
    if (resolve_partition(S, Hq, Hkv, d, bs, max_context_len, partition_size) < 0) return PKV_ERR_INVALID_ARG;
    if (kernel == PKV_DECODE_TENSOR_CORES && !decode_tc_supports(q_dtype, cache_dtype, d, bs, NB))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace pkv

extern "C" {

pkv_status pkv_paged_attention_decode_ex(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                         const void* value_cache, pkv_dtype cache_dtype,
                                         const int32_t* block_tables, int MB, const int32_t* context_lens, int S,
                                         int max_context_len, int Hq, int Hkv, int d, int bs, int NB, float scale,
                                         float k_scale, float v_scale, int partition_size, void* workspace,
                                         size_t workspace_bytes, int32_t* err_word, pkv_stream_t stream,
                                         int kernel) {
    const pkv_status chk = check_decode_args(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables,
                                             MB, context_lens, S, max_context_len, Hq, Hkv, d, bs, NB, scale,
                                             k_scale, v_scale, partition_size, kernel);
    if (chk != PKV_OK || S == 0) return chk;

    const int P = resolve_partition(S, Hq, Hkv, d, bs, max_context_len, partition_size);
    const bool use_tc = kernel != PKV_DECODE_CUDA_CORES && decode_tc_supports(q_dtype, cache_dtype, d, bs, NB);
    const DecodePlan pl = make_plan(S, Hq, d, max_context_len, P);
    if (pl.split) {
        if (!workspace || workspace_bytes < pl.bytes) return PKV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    }

    DecodeParams p{};
    p.out = out; p.q = query; p.kc = key_cache; p.vc = value_cache;
    p.block_tables = block_tables; p.context_lens = context_lens; p.err = err_word;
    p.S = S; p.MB = MB; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.bs = bs; p.NB = NB;
    set_partitions(p, pl,
                   launch_partition(pl, S, Hq, Hkv, max_context_len, partition_size,
                                    use_tc && cache_dtype == PKV_FP8_E4M3),
                   MB * bs, tail_hold(cache_dtype, use_tc));
    p.max_ctx = max_context_len;
    const float ks = cache_dtype == PKV_FP8_E4M3 ? k_scale : 1.f;
    p.logit_scale_log2 = scale * ks * kLog2e;
    p.out_scale = cache_dtype == PKV_FP8_E4M3 ? v_scale : 1.f;
    if (pl.split) {
        char* ws = static_cast<char*>(workspace);
        p.sched = reinterpret_cast<unsigned*>(ws);
        p.part_ml = reinterpret_cast<float*>(ws + pl.ml_offset);
        p.part_acc = reinterpret_cast<float*>(ws + pl.acc_offset);
    } else if (workspace && workspace_bytes >= kWorkspaceHeaderBytes && aligned16(workspace)) {
        p.sched = reinterpret_cast<unsigned*>(workspace);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = use_tc ? launch_decode_tc(p, q_dtype, cache_dtype, num_sms_current(), st)
                           : launch_decode_simt(p, q_dtype, cache_dtype, st);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    if (pl.split) e = launch_decode_reduce(p, q_dtype, st);
    return from_cuda(e);
}

pkv_status pkv_paged_kv_write_decode(void* out, const void* query, pkv_dtype q_dtype, const void* key,
                                     const void* value, pkv_dtype in_dtype, void* key_cache, void* value_cache,
                                     pkv_dtype cache_dtype, const int64_t* slot_mapping, const int32_t* block_tables,
                                     int MB, const int32_t* context_lens, int S, int max_context_len, int Hq, int Hkv,
                                     int d, int bs, int NB, float scale, float k_scale, float v_scale,
                                     int partition_size, void* workspace, size_t workspace_bytes, int32_t* err_word,
                                     pkv_stream_t stream) {
    if (S < 0 || MB < 1 || NB < 1 || Hkv < 1 || Hq < 1 || max_context_len < 0) return PKV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_F32 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (in_dtype != PKV_F32 && in_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (cache_dtype != PKV_F32 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3)
        return PKV_ERR_UNSUPPORTED;
    if (!decode_tc_supports(q_dtype, cache_dtype, d, bs, NB)) return PKV_ERR_UNSUPPORTED;
    if (S > 65535) return PKV_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)MB * bs) return PKV_ERR_INVALID_ARG;
    if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if (cache_dtype == PKV_FP8_E4M3 && (!finite_pos(k_scale) || !finite_pos(v_scale))) return PKV_ERR_INVALID_ARG;
    if (partition_size < -1 || (partition_size > 0 && partition_size % bs != 0)) return PKV_ERR_INVALID_ARG;
    if (S == 0) return PKV_OK;
    if (!out || !query || !key || !value || !key_cache || !value_cache || !slot_mapping || !block_tables ||
        !context_lens)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key) || !aligned16(value) || !aligned16(key_cache) ||
        !aligned16(value_cache) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u))
        return PKV_ERR_INVALID_ARG;
    const int P = resolve_partition(S, Hq, Hkv, d, bs, max_context_len, partition_size);
    if (P < 0) return PKV_ERR_INVALID_ARG;
    const DecodePlan pl = make_plan(S, Hq, d, max_context_len, P);
    if (pl.split) {
        if (!workspace || workspace_bytes < pl.bytes) return PKV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    }
    DecodeParams p{};
    p.out = out; p.q = query; p.kc = key_cache; p.vc = value_cache;
    p.block_tables = block_tables; p.context_lens = context_lens; p.err = err_word;
    p.S = S; p.MB = MB; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.bs = bs; p.NB = NB;
    set_partitions(p, pl,
                   launch_partition(pl, S, Hq, Hkv, max_context_len, partition_size, cache_dtype == PKV_FP8_E4M3),
                   MB * bs, tail_hold(cache_dtype, true));
    p.max_ctx = max_context_len;
    const float ks = cache_dtype == PKV_FP8_E4M3 ? k_scale : 1.f;
    p.logit_scale_log2 = scale * ks * kLog2e;
    p.out_scale = cache_dtype == PKV_FP8_E4M3 ? v_scale : 1.f;
    p.new_k = key; p.new_v = value; p.slot_mapping = slot_mapping; p.new_dt = in_dtype;
    p.k_scale = k_scale; p.v_scale = v_scale;
    if (pl.split) {
        char* ws = static_cast<char*>(workspace);
        p.sched = reinterpret_cast<unsigned*>(ws);
        p.part_ml = reinterpret_cast<float*>(ws + pl.ml_offset);
        p.part_acc = reinterpret_cast<float*>(ws + pl.acc_offset);
    } else if (workspace && workspace_bytes >= kWorkspaceHeaderBytes && aligned16(workspace)) {
        p.sched = reinterpret_cast<unsigned*>(workspace);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_decode_tc(p, q_dtype, cache_dtype, num_sms_current(), st);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    if (pl.split) e = launch_decode_reduce(p, q_dtype, st);
    return from_cuda(e);
}

pkv_status pkv_token_attention_decode(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                      const void* value_cache, pkv_dtype cache_dtype, const int32_t* token_slots,
                                      int MT, const int32_t* num_tokens, int S, int max_tokens, int Hq, int Hkv,
                                      int d, int bs, int NB, float scale, float k_scale, float v_scale,
                                      int partition_size, void* workspace, size_t workspace_bytes,
                                      int32_t* err_word, pkv_stream_t stream) {
    if (S < 0 || MT < 1 || NB < 1 || Hkv < 1 || Hq < 1 || max_tokens < 0 || max_tokens > MT)
        return PKV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_F32 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (cache_dtype != PKV_F32 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3)
        return PKV_ERR_UNSUPPORTED;
    if (!decode_tc_supports(q_dtype, cache_dtype, d, bs, NB)) return PKV_ERR_UNSUPPORTED;
    if (S > 65535) return PKV_ERR_UNSUPPORTED;
    if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if (cache_dtype == PKV_FP8_E4M3 && (!finite_pos(k_scale) || !finite_pos(v_scale))) return PKV_ERR_INVALID_ARG;
    if (partition_size < -1 || (partition_size > 0 && partition_size % bs != 0)) return PKV_ERR_INVALID_ARG;
    if (S == 0) return PKV_OK;
    if (!out || !query || !key_cache || !value_cache || !token_slots || !num_tokens) return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(token_slots) & 3u) || (reinterpret_cast<uintptr_t>(num_tokens) & 3u))
        return PKV_ERR_INVALID_ARG;
    const int P = resolve_partition(S, Hq, Hkv, d, bs, max_tokens, partition_size);
    if (P < 0) return PKV_ERR_INVALID_ARG;
    const DecodePlan pl = make_plan(S, Hq, d, max_tokens, P);
    if (pl.split) {
        if (!workspace || workspace_bytes < pl.bytes) return PKV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    }
    DecodeParams p{};
    p.out = out; p.q = query; p.kc = key_cache; p.vc = value_cache;
    p.token_slots = token_slots; p.MT = MT; p.context_lens = num_tokens; p.err = err_word;
    p.S = S; p.MB = 1; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.bs = bs; p.NB = NB;
    set_partitions(p, pl,
                   launch_partition(pl, S, Hq, Hkv, max_tokens, partition_size, cache_dtype == PKV_FP8_E4M3),
                   max_tokens > 0 ? max_tokens : 1, tail_hold(cache_dtype, true));
    p.max_ctx = max_tokens;
    const float ks = cache_dtype == PKV_FP8_E4M3 ? k_scale : 1.f;
    p.logit_scale_log2 = scale * ks * kLog2e;
    p.out_scale = cache_dtype == PKV_FP8_E4M3 ? v_scale : 1.f;
    if (pl.split) {
        char* ws = static_cast<char*>(workspace);
        p.sched = reinterpret_cast<unsigned*>(ws);
        p.part_ml = reinterpret_cast<float*>(ws + pl.ml_offset);
        p.part_acc = reinterpret_cast<float*>(ws + pl.acc_offset);
    } else if (workspace && workspace_bytes >= kWorkspaceHeaderBytes && aligned16(workspace)) {
        p.sched = reinterpret_cast<unsigned*>(workspace);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_decode_tc(p, q_dtype, cache_dtype, num_sms_current(), st, DecodeMode::kTokenTable);
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    if (pl.split) e = launch_decode_reduce(p, q_dtype, st);
    return from_cuda(e);
}

pkv_status pkv_repack_tokens(void* const* key_caches, void* const* value_caches, int num_layers,
                             int32_t* token_slots, int MT, int S, const int64_t* moves, int M, int NB, int bs,
                             size_t token_bytes, int32_t* err_word, pkv_stream_t stream) {
    if (num_layers < 0 || num_layers > kMaxCopyLayers || M < 0 || MT < 1 || S < 0 || NB < 1 || bs < 1)
        return PKV_ERR_INVALID_ARG;
    if (token_bytes == 0 || token_bytes % 16 != 0) return PKV_ERR_INVALID_ARG;
    if (M == 0 || num_layers == 0) return PKV_OK;
    if (!key_caches || !value_caches || !moves || !token_slots) return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(moves) & 7u) || (reinterpret_cast<uintptr_t>(token_slots) & 3u))
        return PKV_ERR_INVALID_ARG;
    RepackParams p{};
    for (int l = 0; l < num_layers; ++l) {
        if (!key_caches[l] || !value_caches[l] || !aligned16(key_caches[l]) || !aligned16(value_caches[l]))
            return PKV_ERR_INVALID_ARG;
        p.k[l] = key_caches[l];
        p.v[l] = value_caches[l];
    }
    p.moves = moves; p.token_slots = token_slots; p.err = err_word;
    p.M = M; p.L = num_layers; p.S = S; p.MT = MT; p.NB = NB; p.bs = bs; p.token_bytes = token_bytes;
    return from_cuda(launch_repack(p, reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status pkv_paged_attention_decode(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                      const void* value_cache, pkv_dtype cache_dtype, const int32_t* block_tables,
                                      int MB, const int32_t* context_lens, int S, int max_context_len, int Hq,
                                      int Hkv, int d, int bs, int NB, float scale, float k_scale, float v_scale,
                                      int partition_size, void* workspace, size_t workspace_bytes,
                                      int32_t* err_word, pkv_stream_t stream) {
    return pkv_paged_attention_decode_ex(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables, MB,
                                         context_lens, S, max_context_len, Hq, Hkv, d, bs, NB, scale, k_scale,
                                         v_scale, partition_size, workspace, workspace_bytes, err_word, stream,
                                         PKV_DECODE_AUTO);
}

}  // extern "C"

namespace pkv {
namespace {

bool prefill_two_tiles(int S, int T, int g) {
    // two query tiles per unit pay when a (sequence, K/V head) has 256 or
    // more (query, head) rows on average: prompt chunks, not speculative tokens
    return (long long)T * g >= 2LL * kPrefillTileRows * S;
}

// Prefill partition size (0 = no split; -1 = invalid): tiles of 16 (query,
// head) rows already give parallelism, so split only when there are few.
// keys: the most a tile's queries reach (max_ctx without a window).
int resolve_prefill_partition(int S, int max_q_len, int Hq, int Hkv, int d, int bs, int max_ctx, int keys, int req) {
    if (!decode_shape_ok(S, Hq, Hkv, d, bs, max_ctx) || max_q_len < 0 || max_q_len > max_ctx) return -1;
    if (req > 0) return req % bs == 0 ? req : -1;
    if (req == -1) return 0;
    if (req != 0) return -1;
    // counted in tiles of 128 rows (the tcgen05 kernel's unit); about four
    // units per SM keep the persistent CTAs busy to the end
    const long long tiles = (long long)S * Hkv * ((max_q_len * (long long)(Hq / Hkv) + 127) / 128);
    if (tiles == 0 || tiles >= kPrefillTargetUnits || keys <= kMinDefaultPartition) return 0;
    int P = 1 << 20;
    while (P > kMinDefaultPartition && tiles * ((keys + P - 1) / P) < kPrefillTargetUnits) P >>= 1;
    return P >= keys ? 0 : P;
}

struct PrefillPlan {
    int P, Pmax;
    bool split;
    size_t ml_offset, acc_offset, bytes;
};

PrefillPlan plan_prefill(int T, int Hq, int d, int max_ctx, int P) {
    PrefillPlan pl{};
    pl.P = P;
    pl.Pmax = P > 0 ? (max_ctx > 0 ? (max_ctx + P - 1) / P : 1) : 1;
    pl.split = P > 0 && pl.Pmax > 1;
    pl.bytes = kWorkspaceHeaderBytes;
    if (!pl.split) return pl;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t units = (size_t)T * Hq * pl.Pmax;
    pl.ml_offset = kWorkspaceHeaderBytes;
    pl.acc_offset = up(pl.ml_offset + units * 2 * sizeof(float));
    pl.bytes = up(pl.acc_offset + units * d * sizeof(float));
    return pl;
}

// The same under a window, whose keys are few and a little more than a power
// of two: the number of equal partitions (of whole 128-key stages) with the
// least estimated time, in tenths of a microsecond.  A unit is a tile of 256
// rows (128 in the one-tile kernel); its time was fitted to 16 shapes, a
// stage 1.8 us (1.0), the rest 7.4 (6), and 6.6 (2) more to store a partial
// result; the merge takes 3 and reads 512 bytes per row and partition.  512
// queries, 64 / 8 heads, window 1,024: 26.8 us in one partition, 68 in the
// three that the plain rule takes; 4 x 512 queries, 28 / 4 heads, window
// 4,096: 136 and 170 (two); 128 queries: 69.8 in one, 25.2 in the nine of 512.
// Only partitions whose partial results `room` bytes hold are considered.
int resolve_prefill_window_partition(int S, int T, int max_q_len, int Hq, int Hkv, int d, int bs, int max_ctx, int keys,
                                     int req, size_t room) {
    const int P = resolve_prefill_partition(S, max_q_len, Hq, Hkv, d, bs, max_ctx, keys, req);
    if (P < 0 || req != 0 || T < 1 || S < 1 || max_q_len < 1) return P;
    const int g = Hq / Hkv;
    const bool two = prefill_two_tiles(S, T, g);
    const long long rows = two ? 2 * kPrefillTileRows : kPrefillTileRows;
    const long long dense = S * (((long long)max_q_len * g + rows - 1) / rows), ragged = (long long)T * g / rows + S;
    const long long tiles = (dense < ragged ? dense : ragged) * Hkv;
    long long best = 0;
    int best_P = 0;
    for (int np = 1; np <= 16; ++np) {
        const int part = ((keys + np - 1) / np + 127) / 128 * 128;
        if (part >= keys && np > 1) break;
        const int n = np > 1 ? (keys + part - 1) / part : 1;
        if (n > 1 && plan_prefill(T, Hq, d, keys, part).bytes > room) break;
        const long long stages = ((n > 1 ? part : keys) + 127) / 128;
        const long long unit = stages * (two ? 18 : 10) + (two ? 74 : 60) + (n > 1 ? (two ? 66 : 20) : 0);
        const long long cost =
            (tiles * n + 151) / 152 * unit + (n > 1 ? 30 + (long long)T * Hq * n * 512 / 650000 : 0);
        if (np == 1 || cost < best) {
            best = cost;
            best_P = n > 1 ? part : 0;
        }
    }
    return best_P;
}

// Keys of the longest tile under a window: a tile of either kernel (up to
// 256 rows) holds at most 255 / g + 2 queries.
int prefill_keys(int max_q_len, int Hq, int Hkv, int bs, int max_ctx, int window, int sinks) {
    if (window <= 0) return max_ctx;
    const int queries = (2 * kPrefillTileRows - 1) / (Hq / Hkv) + 2;
    return window_bound(max_ctx, window, sinks, bs, max_q_len < queries ? max_q_len : queries);
}

}  // namespace
}  // namespace pkv

namespace pkv {
namespace {

// Query chunks; window 0: every key up to the query.
pkv_status prefill_call(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache, const void* value_cache,
                        pkv_dtype cache_dtype, const int32_t* block_tables, int MB, const int32_t* context_lens,
                        const int32_t* query_start, int S, int num_query_tokens, int max_query_len,
                        int max_context_len, int Hq, int Hkv, int d, int bs, int NB, float scale, int partition_size,
                        void* workspace, size_t workspace_bytes, int32_t* err_word, pkv_stream_t stream, int kernel,
                        int window, int sinks) {
    if (kernel < PKV_PREFILL_AUTO || kernel > PKV_PREFILL_TCGEN05_2TILE) return PKV_ERR_INVALID_ARG;
    if (S < 0 || MB < 1 || NB < 1 || Hkv < 1 || Hq < 1 || max_context_len < 0 || num_query_tokens < 0 ||
        max_query_len < 0 || max_query_len > max_context_len)
        return PKV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_BF16 || cache_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (!(d == 64 || d == 128) || !(bs == 16 || bs == 32)) return PKV_ERR_UNSUPPORTED;
    if (S > 65535 || (long long)NB * bs >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)MB * bs) return PKV_ERR_INVALID_ARG;
    if (!isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if (partition_size < -1 || (partition_size > 0 && partition_size % bs != 0)) return PKV_ERR_INVALID_ARG;
    if (S == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !query || !key_cache || !value_cache || !block_tables || !context_lens || !query_start)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(query_start) & 3u))
        return PKV_ERR_INVALID_ARG;
    clamp_window(max_context_len, window, sinks);
    const int keys = prefill_keys(max_query_len, Hq, Hkv, bs, max_context_len, window, sinks);
    const int P = window > 0 ? resolve_prefill_window_partition(S, num_query_tokens, max_query_len, Hq, Hkv, d, bs,
                                                                max_context_len, keys, partition_size,
                                                                workspace_room(workspace, workspace_bytes))
                             : resolve_prefill_partition(S, max_query_len, Hq, Hkv, d, bs, max_context_len, keys,
                                                         partition_size);
    if (P < 0) return PKV_ERR_INVALID_ARG;
    const PrefillPlan pl = plan_prefill(num_query_tokens, Hq, d, keys, P);
    if (pl.split && (!workspace || workspace_bytes < pl.bytes)) return PKV_ERR_WORKSPACE;
    if (workspace && !aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    DecodeParams p{};
    p.out = out; p.q = query; p.kc = key_cache; p.vc = value_cache;
    p.block_tables = block_tables; p.context_lens = context_lens; p.err = err_word;
    p.S = S; p.MB = MB; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.bs = bs; p.NB = NB;
    p.P = pl.P > 0 ? pl.P : MB * bs;
    p.Q = p.P;                            // query chunks: whole partitions only
    p.Pmax = pl.Pmax;
    p.max_ctx = max_context_len;
    p.window = window;
    p.sinks = sinks;
    p.logit_scale_log2 = scale * kLog2e;
    p.out_scale = 1.f;
    if (workspace && workspace_bytes >= kWorkspaceHeaderBytes) p.sched = reinterpret_cast<unsigned*>(workspace);
    if (pl.split) {
        char* ws = static_cast<char*>(workspace);
        p.part_ml = reinterpret_cast<float*>(ws + pl.ml_offset);
        p.part_acc = reinterpret_cast<float*>(ws + pl.acc_offset);
    }
    auto st = reinterpret_cast<cudaStream_t>(stream);
    if (kernel == PKV_PREFILL_MMA_SYNC)
        return from_cuda(launch_prefill_tc(p, query_start, num_query_tokens, max_query_len, num_sms_current(),
                                           pl.split, st));
    const bool two_tiles = kernel == PKV_PREFILL_TCGEN05_2TILE ||
                           (kernel == PKV_PREFILL_AUTO && prefill_two_tiles(S, num_query_tokens, Hq / Hkv));
    if (two_tiles)
        return from_cuda(launch_prefill_umma2(p, query_start, num_query_tokens, max_query_len, num_sms_current(),
                                              pl.split, st));
    return from_cuda(launch_prefill_umma(p, query_start, num_query_tokens, max_query_len, num_sms_current(),
                                         pl.split, st));
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t pkv_prefill_workspace_size(int S, int num_query_tokens, int max_query_len, int Hq, int Hkv, int d, int bs,
                                  int max_context_len, int partition_size) {
    if (num_query_tokens < 0) return 0;
    const int P =
        resolve_prefill_partition(S, max_query_len, Hq, Hkv, d, bs, max_context_len, max_context_len, partition_size);
    if (P < 0) return 0;
    return plan_prefill(num_query_tokens, Hq, d, max_context_len, P).bytes;
}

size_t pkv_prefill_window_workspace_size(int S, int num_query_tokens, int max_query_len, int Hq, int Hkv, int d, int bs,
                                         int max_context_len, int window, int num_sinks, int partition_size) {
    if (num_query_tokens < 0 || window < 1 || num_sinks < 0) return 0;
    if (!decode_shape_ok(S, Hq, Hkv, d, bs, max_context_len)) return 0;
    clamp_window(max_context_len, window, num_sinks);
    const int keys = prefill_keys(max_query_len, Hq, Hkv, bs, max_context_len, window, num_sinks);
    const int P = resolve_prefill_window_partition(S, num_query_tokens, max_query_len, Hq, Hkv, d, bs, max_context_len,
                                                   keys, partition_size, SIZE_MAX);
    if (P < 0) return 0;
    return plan_prefill(num_query_tokens, Hq, d, keys, P).bytes;
}

pkv_status pkv_paged_attention_prefill_window(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                              const void* value_cache, pkv_dtype cache_dtype,
                                              const int32_t* block_tables, int MB, const int32_t* context_lens,
                                              const int32_t* query_start, int S, int num_query_tokens,
                                              int max_query_len, int max_context_len, int Hq, int Hkv, int d, int bs,
                                              int NB, float scale, int window, int num_sinks, int partition_size,
                                              void* workspace, size_t workspace_bytes, int32_t* err_word,
                                              pkv_stream_t stream) {
    if (window < 1 || num_sinks < 0) return PKV_ERR_INVALID_ARG;
    return prefill_call(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables, MB, context_lens,
                        query_start, S, num_query_tokens, max_query_len, max_context_len, Hq, Hkv, d, bs, NB, scale,
                        partition_size, workspace, workspace_bytes, err_word, stream, PKV_PREFILL_AUTO, window,
                        num_sinks);
}

pkv_status pkv_paged_attention_prefill(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                       const void* value_cache, pkv_dtype cache_dtype, const int32_t* block_tables,
                                       int MB, const int32_t* context_lens, const int32_t* query_start, int S,
                                       int num_query_tokens, int max_query_len, int max_context_len, int Hq,
                                       int Hkv, int d, int bs, int NB, float scale, int partition_size,
                                       void* workspace, size_t workspace_bytes, int32_t* err_word,
                                       pkv_stream_t stream) {
    return pkv_paged_attention_prefill_ex(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables, MB,
                                          context_lens, query_start, S, num_query_tokens, max_query_len,
                                          max_context_len, Hq, Hkv, d, bs, NB, scale, partition_size, workspace,
                                          workspace_bytes, err_word, stream, PKV_PREFILL_AUTO);
}

pkv_status pkv_paged_attention_prefill_ex(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                          const void* value_cache, pkv_dtype cache_dtype,
                                          const int32_t* block_tables, int MB, const int32_t* context_lens,
                                          const int32_t* query_start, int S, int num_query_tokens,
                                          int max_query_len, int max_context_len, int Hq, int Hkv, int d, int bs,
                                          int NB, float scale, int partition_size, void* workspace,
                                          size_t workspace_bytes, int32_t* err_word, pkv_stream_t stream,
                                          int kernel) {
    return prefill_call(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables, MB, context_lens,
                        query_start, S, num_query_tokens, max_query_len, max_context_len, Hq, Hkv, d, bs, NB, scale,
                        partition_size, workspace, workspace_bytes, err_word, stream, kernel, 0, 0);
}

pkv_status pkv_copy_blocks(void* const* key_caches, void* const* value_caches, int num_layers,
                           const int64_t* block_mapping, int P, int NB, size_t block_bytes, int32_t* err_word,
                           pkv_stream_t stream) {
    if (num_layers < 0 || num_layers > kMaxCopyLayers || P < 0 || NB < 1) return PKV_ERR_INVALID_ARG;
    if (block_bytes == 0 || block_bytes % 16 != 0) return PKV_ERR_INVALID_ARG;
    if (P == 0 || num_layers == 0) return PKV_OK;
    if (!key_caches || !value_caches || !block_mapping) return PKV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(block_mapping) & 7u) return PKV_ERR_INVALID_ARG;
    CopyParams p{};
    for (int l = 0; l < num_layers; ++l) {
        if (!key_caches[l] || !value_caches[l] || !aligned16(key_caches[l]) || !aligned16(value_caches[l]))
            return PKV_ERR_INVALID_ARG;
        p.k[l] = key_caches[l];
        p.v[l] = value_caches[l];
    }
    p.mapping = block_mapping; p.err = err_word; p.P = P; p.NB = NB; p.L = num_layers;
    p.block_bytes = block_bytes;
    return from_cuda(launch_copy(p, reinterpret_cast<cudaStream_t>(stream)));
}

// ---- sliding window with sinks

size_t pkv_decode_window_workspace_size(int S, int Hq, int Hkv, int d, int bs, int max_context_len, int window,
                                        int num_sinks, int partition_size) {
    if (window < 0 || num_sinks < 0 || !decode_shape_ok(S, Hq, Hkv, d, bs, max_context_len)) return 0;
    if (window > 0) clamp_window(max_context_len, window, num_sinks);
    const int keys = decode_keys(bs, max_context_len, window, num_sinks);
    size_t bytes = 0;                     // whatever the cache's dtype
    for (const SplitRule rule : {kSplitBf16, kSplitE4m3, kSplitKv4, kSplitF32}) {
        const int P = resolve_split(S, Hq, Hkv, d, bs, max_context_len, keys, partition_size, rule);
        if (P < 0) return 0;
        bytes = max(bytes, make_plan(S, Hq, d, keys, P).bytes);
    }
    return bytes;
}

pkv_status pkv_paged_attention_decode_window(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                             const void* value_cache, pkv_dtype cache_dtype,
                                             const int32_t* block_tables, int MB, const int32_t* context_lens, int S,
                                             int max_context_len, int Hq, int Hkv, int d, int bs, int NB, float scale,
                                             float k_scale, float v_scale, int window, int num_sinks,
                                             int partition_size, void* workspace, size_t workspace_bytes,
                                             int32_t* err_word, pkv_stream_t stream, int kernel) {
    if (window < 1 || num_sinks < 0) return PKV_ERR_INVALID_ARG;
    const pkv_status chk = check_decode_args(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables,
                                             MB, context_lens, S, max_context_len, Hq, Hkv, d, bs, NB, scale,
                                             k_scale, v_scale, partition_size, kernel);
    if (chk != PKV_OK || S == 0) return chk;
    clamp_window(max_context_len, window, num_sinks);
    const int keys = decode_keys(bs, max_context_len, window, num_sinks);
    const bool use_tc = kernel != PKV_DECODE_CUDA_CORES && decode_tc_supports(q_dtype, cache_dtype, d, bs, NB);
    const bool use_f32 = kernel == PKV_DECODE_AUTO && decode_f32_supports(cache_dtype, bs, NB);
    const SplitRule rule = use_f32 ? kSplitF32 : cache_dtype == PKV_FP8_E4M3 ? kSplitE4m3 : kSplitBf16;
    const int P = fit_partition(resolve_split(S, Hq, Hkv, d, bs, max_context_len, keys, partition_size, rule), keys,
                                partition_size, workspace_room(workspace, workspace_bytes),
                                [&](int n) { return make_plan(S, Hq, d, keys, n).bytes; });
    const bool e4m3 = cache_dtype == PKV_FP8_E4M3;
    const DecodePlan pl = make_plan(S, Hq, d, keys, P);
    if (pl.split && (!workspace || workspace_bytes < pl.bytes)) return PKV_ERR_WORKSPACE;
    if (pl.split && !aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    DecodeParams p{};
    p.out = out; p.q = query; p.kc = key_cache; p.vc = value_cache;
    p.block_tables = block_tables; p.context_lens = context_lens; p.err = err_word;
    p.S = S; p.MB = MB; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.bs = bs; p.NB = NB;
    p.window = window; p.sinks = num_sinks;
    set_partitions(p, pl, launch_partition(pl, S, Hq, Hkv, keys, partition_size, use_tc && e4m3), MB * bs,
                   tail_hold(cache_dtype, use_tc));
    p.max_ctx = max_context_len;
    p.logit_scale_log2 = scale * (e4m3 ? k_scale : 1.f) * kLog2e;
    p.out_scale = e4m3 ? v_scale : 1.f;
    set_workspace(p, pl, workspace, workspace_bytes);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = use_tc    ? launch_decode_tc(p, q_dtype, cache_dtype, num_sms_current(), st, DecodeMode::kWindow)
                    : use_f32 ? launch_decode_f32(p, q_dtype, num_sms_current(), st)
                              : launch_decode_simt(p, q_dtype, cache_dtype, st);
    if (e == cudaSuccess && pl.split && !p.local) e = launch_decode_reduce(p, q_dtype, st);
    return from_cuda(e);
}

// ---- 4-bit cache

size_t pkv_kv4_block_bytes(int bs, int Hkv, int d) {
    if (!(d == 64 || d == 128) || !(bs == 16 || bs == 32) || Hkv < 1) return 0;
    return (size_t)Hkv * kv4_head_bytes(bs, d);
}

static pkv_status kv4_rows(const void* key, const void* value, void* key_out, void* value_out, pkv_dtype dt,
                           const void* key_cache, const void* value_cache, const int64_t* slots, int T, int NB, int bs,
                           int Hkv, int d, float k_scale, float v_scale, int32_t* err_word, pkv_stream_t stream,
                           bool read) {
    if (T < 0 || NB < 1 || bs < 1 || Hkv < 1 || d < 1) return PKV_ERR_INVALID_ARG;
    if (dt != PKV_F32 && dt != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (pkv_kv4_block_bytes(bs, Hkv, d) == 0) return PKV_ERR_UNSUPPORTED;
    if (!finite_pos(k_scale) || !finite_pos(v_scale)) return PKV_ERR_INVALID_ARG;
    if (T == 0) return PKV_OK;
    const void* a = read ? key_out : key;
    const void* b = read ? value_out : value;
    if (!a || !b || !key_cache || !value_cache || !slots) return PKV_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(b) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (reinterpret_cast<uintptr_t>(slots) & 7u))
        return PKV_ERR_INVALID_ARG;
    Kv4Params p{};
    p.key = key; p.value = value; p.key_out = key_out; p.value_out = value_out;
    p.key_cache = const_cast<void*>(key_cache); p.value_cache = const_cast<void*>(value_cache);
    p.slots = slots; p.err = err_word;
    p.T = T; p.NB = NB; p.bs = bs; p.Hkv = Hkv; p.d = d; p.k_scale = k_scale; p.v_scale = v_scale;
    return from_cuda(launch_kv4(p, dt, read, reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status pkv_paged_kv4_write(const void* key, const void* value, pkv_dtype in_dtype, void* key_cache,
                               void* value_cache, const int64_t* slot_mapping, int T, int NB, int bs, int Hkv, int d,
                               float k_scale, float v_scale, int32_t* err_word, pkv_stream_t stream) {
    return kv4_rows(key, value, nullptr, nullptr, in_dtype, key_cache, value_cache, slot_mapping, T, NB, bs, Hkv, d,
                    k_scale, v_scale, err_word, stream, false);
}

pkv_status pkv_paged_kv4_read(void* key, void* value, pkv_dtype out_dtype, const void* key_cache,
                              const void* value_cache, const int64_t* slots, int T, int NB, int bs, int Hkv, int d,
                              float k_scale, float v_scale, int32_t* err_word, pkv_stream_t stream) {
    return kv4_rows(nullptr, nullptr, key, value, out_dtype, key_cache, value_cache, slots, T, NB, bs, Hkv, d, k_scale,
                    v_scale, err_word, stream, true);
}

pkv_status pkv_paged_attention_decode_kv4(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                          const void* value_cache, const int32_t* block_tables, int MB,
                                          const int32_t* context_lens, int S, int max_context_len, int Hq, int Hkv,
                                          int d, int bs, int NB, float scale, float k_scale, float v_scale, int window,
                                          int num_sinks, int partition_size, void* workspace, size_t workspace_bytes,
                                          int32_t* err_word, pkv_stream_t stream) {
    if (window < 0 || num_sinks < 0) return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    // the checks of a decode over a cache with tensor scales
    const pkv_status chk = check_decode_args(out, query, q_dtype, key_cache, value_cache, PKV_FP8_E4M3, block_tables,
                                             MB, context_lens, S, max_context_len, Hq, Hkv, d, bs, NB, scale,
                                             k_scale, v_scale, partition_size, PKV_DECODE_AUTO);
    if (chk != PKV_OK || S == 0) return chk;
    if (window > 0) clamp_window(max_context_len, window, num_sinks);
    const int keys = decode_keys(bs, max_context_len, window, num_sinks);
    const int P = fit_partition(resolve_split(S, Hq, Hkv, d, bs, max_context_len, keys, partition_size, kSplitKv4), keys,
                                partition_size, workspace_room(workspace, workspace_bytes),
                                [&](int n) { return make_plan(S, Hq, d, keys, n).bytes; });
    const DecodePlan pl = make_plan(S, Hq, d, keys, P);
    if (pl.split && (!workspace || workspace_bytes < pl.bytes)) return PKV_ERR_WORKSPACE;
    if (pl.split && !aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    DecodeParams p{};
    p.out = out; p.q = query; p.kc = key_cache; p.vc = value_cache;
    p.block_tables = block_tables; p.context_lens = context_lens; p.err = err_word;
    p.S = S; p.MB = MB; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.bs = bs; p.NB = NB;
    p.window = window; p.sinks = window > 0 ? num_sinks : 0;
    set_partitions(p, pl, pl.P, MB * bs, kv4_hold(S, Hq, Hkv, keys, pl.P));
    p.max_ctx = max_context_len;
    p.logit_scale_log2 = scale * k_scale * kLog2e;
    p.out_scale = v_scale;
    set_workspace(p, pl, workspace, workspace_bytes);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_decode_kv4(p, num_sms_current(), st);
    if (e == cudaSuccess && pl.split && !p.local) e = launch_decode_reduce(p, q_dtype, st);
    return from_cuda(e);
}

// ---- eviction by accumulated attention weight

size_t pkv_token_attention_scored_workspace_size(int S, int Hq, int Hkv, int d, int bs, int max_tokens,
                                                 int partition_size) {
    size_t bytes = 0;                     // whatever the cache's dtype
    for (const SplitRule rule : {kSplitBf16, kSplitE4m3}) {
        const int P = resolve_split(S, Hq, Hkv, d, bs, max_tokens, max_tokens, partition_size, rule);
        if (P < 0) return 0;
        bytes = max(bytes, make_scored_plan(S, Hq, Hkv, d, max_tokens, P).bytes);
    }
    return bytes;
}

pkv_status pkv_token_attention_decode_scored(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                             const void* value_cache, pkv_dtype cache_dtype,
                                             const int32_t* token_slots, int MT, const int32_t* num_tokens,
                                             float* scores, int S, int max_tokens, int Hq, int Hkv, int d, int bs,
                                             int NB, float scale, float k_scale, float v_scale, int partition_size,
                                             void* workspace, size_t workspace_bytes, int32_t* err_word,
                                             pkv_stream_t stream) {
    if (max_tokens < 0 || max_tokens > MT) return PKV_ERR_INVALID_ARG;
    // the checks of a decode whose table holds every token: one table entry per token, none per block
    const pkv_status chk = check_decode_args(out, query, q_dtype, key_cache, value_cache, cache_dtype, token_slots,
                                             MT, num_tokens, S, max_tokens, Hq, Hkv, d, bs, NB, scale, k_scale,
                                             v_scale, partition_size, PKV_DECODE_TENSOR_CORES);
    if (chk != PKV_OK || S == 0) return chk;
    if (!scores || (reinterpret_cast<uintptr_t>(scores) & 3u)) return PKV_ERR_INVALID_ARG;
    const int P = fit_partition(resolve_split(S, Hq, Hkv, d, bs, max_tokens, max_tokens, partition_size,
                                              cache_dtype == PKV_FP8_E4M3 ? kSplitE4m3 : kSplitBf16),
                                max_tokens, partition_size, workspace_room(workspace, workspace_bytes),
                                [&](int n) { return make_scored_plan(S, Hq, Hkv, d, max_tokens, n).bytes; });
    const ScoredPlan sp = make_scored_plan(S, Hq, Hkv, d, max_tokens, P);
    if (!workspace || workspace_bytes < sp.bytes) return PKV_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    const bool e4m3 = cache_dtype == PKV_FP8_E4M3;
    DecodeParams p{};
    p.out = out; p.q = query; p.kc = key_cache; p.vc = value_cache;
    p.token_slots = token_slots; p.MT = MT; p.context_lens = num_tokens; p.err = err_word;
    p.S = S; p.MB = 1; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.d = d; p.bs = bs; p.NB = NB;
    set_partitions(p, sp.pl, launch_partition(sp.pl, S, Hq, Hkv, max_tokens, partition_size, e4m3),
                   max_tokens > 0 ? max_tokens : 1, tail_hold(cache_dtype, true));
    p.max_ctx = max_tokens;
    p.logit_scale_log2 = scale * (e4m3 ? k_scale : 1.f) * kLog2e;
    p.out_scale = e4m3 ? v_scale : 1.f;
    set_workspace(p, sp.pl, workspace, workspace_bytes);
    char* ws = static_cast<char*>(workspace);
    p.part_ml = reinterpret_cast<float*>(ws + sp.ml_offset);
    p.logits = reinterpret_cast<float*>(ws + sp.logits_offset);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_decode_tc(p, q_dtype, cache_dtype, num_sms_current(), st, DecodeMode::kScored);
    if (e == cudaSuccess) e = launch_score(p, q_dtype, sp.pl.split, scores, MT, num_sms_current(), st);
    return from_cuda(e);
}

pkv_status pkv_evict_tokens(const int32_t* token_slots, const float* scores, const int32_t* num_tokens, int S, int MT,
                            int budget, int num_first, int num_recent, int32_t* new_slots, float* new_scores,
                            int32_t* new_num, int32_t* evicted, int32_t* err_word, pkv_stream_t stream) {
    if (S < 0 || MT < 1 || budget < 0 || num_first < 0 || num_recent < 0) return PKV_ERR_INVALID_ARG;
    if ((long long)num_first + num_recent > budget) return PKV_ERR_INVALID_ARG;
    if (S > 65535 || MT > (1 << 30)) return PKV_ERR_UNSUPPORTED;
    if (S == 0) return PKV_OK;
    if (!token_slots || !scores || !num_tokens || !new_slots || !new_scores || !new_num) return PKV_ERR_INVALID_ARG;
    const size_t rows = (size_t)S * MT * 4, nums = (size_t)S * 4;
    const void* in[3] = {token_slots, scores, num_tokens};
    const size_t in_bytes[3] = {rows, rows, nums};
    const void* to[4] = {new_slots, new_scores, new_num, evicted};
    const size_t to_bytes[4] = {rows, rows, nums, rows};
    for (int i = 0; i < 4; ++i) {
        if (to[i] == nullptr) continue;
        if (reinterpret_cast<uintptr_t>(to[i]) & 3u) return PKV_ERR_INVALID_ARG;
        for (int j = 0; j < 3; ++j)
            if (overlap(to[i], in[j], to_bytes[i], in_bytes[j])) return PKV_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(to[i], to[j], to_bytes[i], to_bytes[j])) return PKV_ERR_INVALID_ARG;
    }
    for (const void* q : in)
        if (reinterpret_cast<uintptr_t>(q) & 3u) return PKV_ERR_INVALID_ARG;
    EvictParams p{};
    p.token_slots = token_slots; p.scores = scores; p.num_tokens = num_tokens;
    p.new_slots = new_slots; p.new_scores = new_scores; p.new_num = new_num; p.evicted = evicted; p.err = err_word;
    p.S = S; p.MT = MT; p.budget = budget; p.first = num_first; p.recent = num_recent;
    return from_cuda(launch_evict(p, num_sms_current(), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
