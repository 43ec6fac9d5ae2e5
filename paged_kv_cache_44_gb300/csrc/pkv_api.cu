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

}  // extern "C"

namespace pkv {
namespace {

// Key stages of the longest tile of a prompt: those of the sinks and of what
// the windows of one group of query blocks span.
int prompt_stages(int max_k, int g, int window, int sinks) {
    const int all = (int)((max_k - 1LL + kPromptStage) / kPromptStage);      // (a bound may be as large as an int)
    if (window <= 0) return all;
    const long long span = (long long)window - 1 + prompt_group(g) * kPromptStage + kPromptStage - 1;
    const long long n = (span + kPromptStage - 1) / kPromptStage + (sinks - 1LL + kPromptStage) / kPromptStage;
    return n < all ? (int)n : all;
}

// (stages and P in stages, not tokens)
PrefillPlan plan_prompt(int Tq, int Hq, int d, int stages, int P) { return plan_prefill(Tq, Hq, d, stages, P); }

bool prompt_shape_ok(int S, int Tq, int max_q, int max_k, int Hq, int Hkv, int d, int req) {
    return S >= 0 && S <= 65535 && Tq >= 0 && max_q >= 0 && max_k >= 0 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
           (d == 64 || d == 128) && req >= -1 && (req <= 0 || req % kPromptStage == 0);
}

// Few queries: tiles of (query, head) rows, so that the heads of a K/V head
// share them.  (Rows are stepped through by heads.)
constexpr int kPackedQueries = 64;
bool prompt_packed(int max_q, int64_t q_stride, int d) { return max_q <= kPackedQueries && q_stride % d == 0; }

// Stages per partition (0: no split).
int resolve_prompt_partition(int S, int Tq, int max_q, int Hq, int Hkv, int d, int stages, int req, size_t room) {
    if (req != 0) return req > 0 ? req / kPromptStage : 0;
    const int g = Hq / Hkv, group = prompt_group(g);
    const long long rows = (long long)group * kPromptStage;
    const long long dense = S * ((max_q + rows - 1) / rows), ragged = Tq / rows + S;
    long long units = (dense < ragged ? dense : ragged) * Hkv * ((g * group + 1) / 2);
    if (max_q <= kPackedQueries) {
        const long long tiles = ((long long)max_q * g + kPromptStage - 1) / kPromptStage;
        units = (long long)S * Hkv * ((tiles + 1) / 2);
        if (tiles == 1) units = (units + 1) / 2;           // paired partitions
    }
    if (units == 0 || units > 76) return 0;
    const long long parts = 152 / units;
    int P = (int)((stages + parts - 1) / parts);
    if (P < 4) P = 4;
    // A stage takes 1.65 us; a split launch 7 more, and 1 KB written and read per row and partition (at 4 TB/s).  1,024
    // queries, 12 / 2 heads, 20.0 us (causal) and 21.3 in one partition, 25.2 and 30.0 in two; 2,048 of them 33.4 and
    // 35.6, in two 39 and 61; but 5 and 9 queries over 16,384 and 32,768 keys 329 and 26.4.
    const long long np = (stages + P - 1) / P;
    if ((stages - P) * 165LL < 700 + (long long)Tq * Hq * np / 40) return 0;
    while (P < stages && plan_prompt(Tq, Hq, d, stages, P).bytes > room) P += P / 8 > 1 ? P / 8 : 1;
    return P < stages ? P : 0;
}

}  // namespace
}  // namespace pkv

extern "C" {

// ---- a prompt's way into the cache

size_t pkv_prompt_workspace_size(int S, int num_query_tokens, int max_query_len, int max_key_len, int Hq, int Hkv, int d,
                                 int window, int num_sinks, int partition_size) {
    if (!prompt_shape_ok(S, num_query_tokens, max_query_len, max_key_len, Hq, Hkv, d, partition_size) || window < 0 ||
        num_sinks < 0)
        return 0;
    max_query_len = min(max_query_len, num_query_tokens);
    clamp_window(max_key_len, window, num_sinks);
    const int stages = prompt_stages(max_key_len, Hq / Hkv, window, num_sinks);
    const int P = resolve_prompt_partition(S, num_query_tokens, max_query_len, Hq, Hkv, d, stages, partition_size, SIZE_MAX);
    return plan_prompt(num_query_tokens, Hq, d, stages, P).bytes;
}

pkv_status pkv_prompt_attention(void* out, const void* query, const void* key, const void* value, pkv_dtype dtype,
                                int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* query_start,
                                const int32_t* key_start, int S, int num_query_tokens, int num_key_tokens,
                                int max_query_len, int max_key_len, int Hq, int Hkv, int d, float scale, int causal,
                                int window, int num_sinks, int partition_size, void* workspace,
                                size_t workspace_bytes, int32_t* err_word, pkv_stream_t stream) {
    if (S < 0 || Hkv < 1 || Hq < 1 || num_query_tokens < 0 || num_key_tokens < 0 || max_query_len < 0 || max_key_len < 0)
        return PKV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_BF16 || !(d == 64 || d == 128) || S > 65535) return PKV_ERR_UNSUPPORTED;
    if ((long long)Hq * d > (1 << 24) || num_query_tokens > (1 << 30) || num_key_tokens > (1 << 30))
        return PKV_ERR_UNSUPPORTED;
    if (!isfinite(scale) || window < 0 || num_sinks < 0 || (window > 0 && !causal)) return PKV_ERR_INVALID_ARG;
    if (partition_size < -1 || (partition_size > 0 && partition_size % kPromptStage != 0)) return PKV_ERR_INVALID_ARG;
    if (S == 0 || num_query_tokens == 0) return PKV_OK;
    if (!out || !query || !query_start || !key_start || (num_key_tokens > 0 && (!key || !value))) return PKV_ERR_INVALID_ARG;
    struct Rows {
        const void* at;
        int64_t stride;
        int heads, n;
    };
    const size_t out_bytes = (size_t)num_query_tokens * Hq * d * 2;
    for (const Rows& r : {Rows{query, q_stride, Hq, num_query_tokens}, Rows{key, k_stride, Hkv, num_key_tokens},
                          Rows{value, v_stride, Hkv, num_key_tokens}}) {
        if (r.n == 0) continue;
        if (!aligned16(r.at) || r.stride < (int64_t)r.heads * d || r.stride >= (1LL << 38) || r.stride % 8 != 0 ||
            r.stride > (1LL << 46) / r.n)
            return PKV_ERR_INVALID_ARG;
        if (overlap(out, r.at, out_bytes, (size_t)((r.n - 1) * r.stride + (int64_t)r.heads * d) * 2)) return PKV_ERR_INVALID_ARG;
    }
    if (!aligned16(out) || (reinterpret_cast<uintptr_t>(query_start) & 3u) || (reinterpret_cast<uintptr_t>(key_start) & 3u))
        return PKV_ERR_INVALID_ARG;
    // bounds may be loose: no sequence has more queries or keys than there are (but partitions that the caller asks
    // for take the workspace that it was told for its bound)
    max_query_len = min(max_query_len, num_query_tokens);
    if (partition_size == 0) max_key_len = min(max_key_len, num_key_tokens);
    clamp_window(max_key_len, window, num_sinks);
    const int stages = prompt_stages(max_key_len, Hq / Hkv, window, num_sinks);
    const int P = resolve_prompt_partition(S, num_query_tokens, max_query_len, Hq, Hkv, d, stages, partition_size,
                                           workspace_room(workspace, workspace_bytes));
    const PrefillPlan pl = plan_prompt(num_query_tokens, Hq, d, stages, P);
    if (pl.split && (!workspace || workspace_bytes < pl.bytes)) return PKV_ERR_WORKSPACE;
    if (workspace && !aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    PromptParams p{};
    p.out = out; p.q = query; p.k = key; p.v = value; p.query_start = query_start; p.key_start = key_start;
    p.err = err_word; p.q_stride = q_stride; p.k_stride = num_key_tokens > 0 ? k_stride : (int64_t)Hkv * d;
    p.v_stride = num_key_tokens > 0 ? v_stride : (int64_t)Hkv * d;
    p.S = S; p.Tq = num_query_tokens; p.Tk = num_key_tokens; p.max_q = max_query_len; p.max_k = max_key_len;
    p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv; p.group = prompt_group(p.g);
    p.packed = prompt_packed(max_query_len, q_stride, d);
    p.causal = causal != 0; p.window = window; p.sinks = num_sinks;
    p.P = pl.split ? P : 0;
    p.Pmax = pl.Pmax;
    p.scale_log2 = scale * kLog2e;
    if (workspace && workspace_bytes >= kWorkspaceHeaderBytes) p.sched = reinterpret_cast<unsigned*>(workspace);
    if (pl.split) {
        char* ws = static_cast<char*>(workspace);
        p.part_ml = reinterpret_cast<float*>(ws + pl.ml_offset);
        p.part_acc = reinterpret_cast<float*>(ws + pl.acc_offset);
    }
    return from_cuda(launch_prompt(p, d, num_sms_current(), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace pkv {
namespace {

// Partitions of a shared decode: of the shared tokens Pre (stages of 128; 0:
// not split), of a sequence's own tokens P, and where each row's partial
// results and the sequences' shared lengths lie.
struct SharedPlan {
    int pre, first_own;                   // partial results of the shared tokens come first
    DecodePlan own;
    int Pmax;
    size_t ml_offset, acc_offset, begin_offset, bytes;
};
SharedPlan plan_shared(int S, int Hq, int d, int max_ctx, int max_shared, int pre, int P) {
    SharedPlan sp{};
    const int stages = (int)((max_shared - 1LL + kPromptStage) / kPromptStage);
    sp.pre = pre;
    sp.first_own = pre > 0 ? (stages + pre - 1) / pre : 1;
    sp.own = make_plan(S, Hq, d, max_ctx, P);
    sp.Pmax = sp.first_own + sp.own.Pmax_plain;
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t units = (size_t)S * Hq * sp.Pmax;
    sp.ml_offset = kWorkspaceHeaderBytes;
    sp.acc_offset = up(sp.ml_offset + units * 2 * sizeof(float));
    sp.begin_offset = up(sp.acc_offset + units * d * sizeof(float));
    sp.bytes = up(sp.begin_offset + (size_t)S * sizeof(int32_t));
    return sp;
}

// Stages per partition of the shared tokens: the number of equal partitions
// with the least rounds of units, a unit's fixed cost counted as 3 stages.
int resolve_shared_prefix(int G, int max_group, int g, int Hkv, int max_shared, int req) {
    const int stages = (int)((max_shared - 1LL + kPromptStage) / kPromptStage);
    if (req == -1) return 0;
    if (req > 0) {
        const int p = (int)((req - 1LL + kPromptStage) / kPromptStage);
        return p < stages ? p : 0;
    }
    // a group of one tile pairs its partitions: two of them are a unit
    const long long tiles = ((long long)max_group * g + kPromptStage - 1) / kPromptStage, units = G * Hkv * ((tiles + 1) / 2);
    const int per = tiles == 1 ? 2 : 1;
    long long best = 0;
    int best_p = 0;
    for (int np = 1; np <= 64 && np <= stages; ++np) {
        const int p = (stages + np - 1) / np, n = (stages + p - 1) / p;
        const long long cost = (units * ((n + per - 1) / per) + 151) / 152 * ((n > 1 ? per : 1) * p + 4) * 16 + n;
        if (np == 1 || cost < best) {
            best = cost;
            best_p = n > 1 ? p : 0;
        }
    }
    return best_p;
}

bool shared_shape_ok(int S, int G, int Hq, int Hkv, int d, int bs, int max_ctx, int max_shared, int max_group, int req) {
    return decode_shape_ok(S, Hq, Hkv, d, bs, max_ctx) && G >= 0 && max_shared >= 0 && max_shared <= max_ctx && max_group >= 0 &&
           max_group <= 65535 && req >= -1 && (req <= 0 || req % bs == 0);
}

constexpr int kMaxOwnParts = 96;

// Whether the shared tokens get a launch of their own: where sequences on
// their own would read them from 256 MB on again.  By the bounds, which is all
// that the host has: G groups of max_group members, but no more members than
// sequences.  A group that shares nothing counts as the others do.  Two more
// launches take 15-20 us, about what HBM and L2 take for that: 64 sequences
// sharing 2,048 tokens of 4 heads of 128 (264 MB) 42 us and 45 on their own,
// 128 of them 48 and 64; 256 sharing 512 (267 MB) 64.5 and 61.4; 100 of 256
// sharing 1,024 (207 MB, read from L2 while HBM is the bound) 353 and 332 (by
// the bounds 207 MB where they are the only group, 415 with the others as a
// second one).
constexpr long long kShareBytes = 256LL << 20;
bool shares(int S, int G, int max_shared, int max_group, int Hkv, int d, int bs, int sharing) {
    if (G < 1 || max_shared < bs || max_group < 1) return false;
    const long long again = min((long long)G * (max_group - 1), (long long)S - 1);
    return sharing == PKV_SHARE_ALWAYS || again * max_shared * Hkv * d * 4 >= kShareBytes;
}

// Sequences on their own, as the windowed decode with everything in its window:
// it splits a small launch further and merges within it.  Eight sequences of
// 305..344 tokens, 2 K/V heads, 12.3 us and 22.5 by the plain decode; two of
// 1,088, 4 heads, 14.3 and 20.5; 64 of 129..384, 4 heads, 18.4 and 22.5; but 64
// of 513..640, 4 heads, 24.6 and 22.5, and two of 32,832, 2 heads, 32.8 and 28.7.
bool as_window(int S, int Hq, int Hkv, int d, int bs, int max_ctx, int req) {
    const long long sets = (long long)S * Hkv * ((Hq / Hkv + kHeadSet - 1) / kHeadSet);
    return req == 0 && max_ctx > 0 &&
           (resolve_partition(S, Hq, Hkv, d, bs, max_ctx, 0) == 0 || (max_ctx <= 1280 && sets < 152));
}

SharedPlan choose_shared(int S, int G, int Hq, int Hkv, int d, int bs, int max_ctx, int max_shared, int max_group, int req,
                         size_t room) {
    // what a sequence has of its own: taken to be what the longest one would have beside the longest shared part
    // (longer ones are more partitions, up to kMaxOwnParts)
    int P = resolve_partition(S, Hq, Hkv, d, bs, max_ctx > max_shared ? max_ctx - max_shared : max_ctx, req);
    if (req == 0) {
        if (P == 0) P = max_ctx > max_shared ? (max_ctx - max_shared + bs - 1) / bs * bs : max_ctx;
        P = max(P, (max_ctx / kMaxOwnParts + bs) / bs * bs);
        if (P >= max_ctx) P = 0;
    }
    int pre = resolve_shared_prefix(G, max_group, Hq / Hkv, Hkv, max_shared, req);
    SharedPlan sp = plan_shared(S, Hq, d, max_ctx, max_shared, pre, P);
    // a smaller workspace: fewer partitions
    while (req == 0 && sp.bytes > room && (P > 0 || pre > 0)) {
        P = P > 0 && 2 * P < max_ctx ? 2 * P : 0;
        pre = pre > 0 && 2 * pre * kPromptStage < max_shared ? 2 * pre : 0;
        sp = plan_shared(S, Hq, d, max_ctx, max_shared, pre, P);
    }
    return sp;
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t pkv_decode_shared_workspace_size(int S, int G, int Hq, int Hkv, int d, int bs, int max_context_len,
                                        int max_shared_len, int max_group_size, int partition_size, int sharing) {
    if (!shared_shape_ok(S, G, Hq, Hkv, d, bs, max_context_len, max_shared_len, max_group_size, partition_size) ||
        sharing < PKV_SHARE_AUTO || sharing > PKV_SHARE_ALWAYS)
        return 0;
    const size_t plain = as_window(S, Hq, Hkv, d, bs, max_context_len, partition_size)
                             ? pkv_decode_window_workspace_size(S, Hq, Hkv, d, bs, max_context_len, max_context_len, 0, 0)
                             : pkv_decode_workspace_size(S, Hq, Hkv, d, bs, max_context_len, partition_size);
    if (!shares(S, G, max_shared_len, max_group_size, Hkv, d, bs, sharing)) return plain;
    return max(plain, choose_shared(S, G, Hq, Hkv, d, bs, max_context_len, max_shared_len, max_group_size, partition_size,
                                    SIZE_MAX).bytes);
}

pkv_status pkv_paged_attention_decode_shared(void* out, const void* query, pkv_dtype q_dtype, const void* key_cache,
                                             const void* value_cache, pkv_dtype cache_dtype, const int32_t* block_tables,
                                             int MB, const int32_t* context_lens, const int32_t* group_start,
                                             const int32_t* shared_lens, int S, int G, int max_context_len,
                                             int max_shared_len, int max_group_size, int Hq, int Hkv, int d, int bs,
                                             int NB, float scale, int partition_size, void* workspace,
                                             size_t workspace_bytes, int32_t* err_word, pkv_stream_t stream, int sharing) {
    if (sharing < PKV_SHARE_AUTO || sharing > PKV_SHARE_ALWAYS) return PKV_ERR_INVALID_ARG;
    if (G < 0 || max_shared_len < 0 || max_shared_len > max_context_len || max_group_size < 0) return PKV_ERR_INVALID_ARG;
    if (q_dtype != PKV_BF16 || cache_dtype != PKV_BF16 || max_group_size > 65535 || G > 65535) return PKV_ERR_UNSUPPORTED;
    const pkv_status chk = check_decode_args(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables, MB,
                                             context_lens, S, max_context_len, Hq, Hkv, d, bs, NB, scale, 1.f, 1.f,
                                             partition_size, PKV_DECODE_TENSOR_CORES);
    if (chk != PKV_OK || S == 0) return chk;
    if (G > 0 && (!group_start || !shared_lens)) return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(group_start) & 3u) || (reinterpret_cast<uintptr_t>(shared_lens) & 3u))
        return PKV_ERR_INVALID_ARG;
    const size_t room = workspace_room(workspace, workspace_bytes);
    const bool share = shares(S, G, max_shared_len, max_group_size, Hkv, d, bs, sharing);
    SharedPlan sp{};
    if (share)
        sp = choose_shared(S, G, Hq, Hkv, d, bs, max_context_len, max_shared_len, max_group_size, partition_size, room);
    if (!share || (partition_size == 0 && sp.bytes > room)) {
        // not enough to share, or no room to: every sequence on its own
        if (as_window(S, Hq, Hkv, d, bs, max_context_len, partition_size))
            return pkv_paged_attention_decode_window(out, query, q_dtype, key_cache, value_cache, cache_dtype,
                                                     block_tables, MB, context_lens, S, max_context_len, Hq, Hkv, d, bs,
                                                     NB, scale, 1.f, 1.f, max_context_len, 0, 0, workspace,
                                                     workspace_bytes, err_word, stream, PKV_DECODE_AUTO);
        int P = resolve_partition(S, Hq, Hkv, d, bs, max_context_len, partition_size);
        P = fit_partition(P, max_context_len, partition_size, room, [&](int n) { return make_plan(S, Hq, d, max_context_len, n).bytes; });
        return pkv_paged_attention_decode_ex(out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables, MB,
                                             context_lens, S, max_context_len, Hq, Hkv, d, bs, NB, scale, 1.f, 1.f,
                                             P > 0 ? P : -1, workspace, workspace_bytes, err_word, stream,
                                             PKV_DECODE_TENSOR_CORES);
    }
    if (!workspace || workspace_bytes < sp.bytes) return PKV_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    DecodeParams d_p{};
    d_p.out = out; d_p.q = query; d_p.kc = key_cache; d_p.vc = value_cache;
    d_p.block_tables = block_tables; d_p.context_lens = context_lens; d_p.err = err_word;
    d_p.S = S; d_p.MB = MB; d_p.Hq = Hq; d_p.Hkv = Hkv; d_p.g = Hq / Hkv; d_p.d = d; d_p.bs = bs; d_p.NB = NB;
    set_partitions(d_p, sp.own, sp.own.P, MB * bs, 0);
    d_p.Pmax = sp.Pmax;
    d_p.max_ctx = max_context_len;
    d_p.logit_scale_log2 = scale * kLog2e;
    d_p.out_scale = 1.f;
    d_p.sched = reinterpret_cast<unsigned*>(ws);
    // a row's own partial results lie behind those of its shared tokens
    float* ml = reinterpret_cast<float*>(ws + sp.ml_offset);
    float* acc = reinterpret_cast<float*>(ws + sp.acc_offset);
    d_p.part_ml = ml + 2 * sp.first_own;
    d_p.part_acc = acc + (size_t)sp.first_own * d;
    d_p.begin = reinterpret_cast<int32_t*>(ws + sp.begin_offset);
    d_p.own_max = reinterpret_cast<int*>(ws + 128);       // behind the counters, in the header
    PromptParams p{};
    p.out = out; p.q = query; p.k = key_cache; p.v = value_cache;
    p.query_start = group_start; p.key_start = shared_lens; p.part_ml = ml; p.part_acc = acc;
    p.sched = d_p.sched; p.err = err_word;
    p.S = G; p.Tq = S; p.max_q = max_group_size; p.max_k = max_shared_len; p.Hq = Hq; p.Hkv = Hkv; p.g = Hq / Hkv;
    p.group = 1; p.q_stride = (int64_t)Hq * d; p.P = sp.pre; p.Pmax = sp.Pmax;
    p.scale_log2 = scale * kLog2e;
    p.tables = block_tables; p.lens = context_lens; p.begin = reinterpret_cast<int32_t*>(ws + sp.begin_offset);
    p.own_max = reinterpret_cast<int*>(ws + 128);
    p.MB = MB; p.bs = bs; p.NB = NB; p.max_ctx = max_context_len;
    const SharedParts parts{sp.first_own, d_p.P, d_p.Q, max_context_len};
    auto st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_shared_prefix(p, d_p, num_sms_current(), st);
    if (e == cudaSuccess) e = launch_decode_tc_suffix(d_p, q_dtype, cache_dtype, num_sms_current(), st);
    if (e == cudaSuccess) e = launch_shared_merge(p, parts, d, st);
    return from_cuda(e);
}

pkv_status pkv_rotary_kv_write(const void* query, const void* key, const void* value, pkv_dtype in_dtype,
                               int64_t q_stride, int64_t k_stride, int64_t v_stride, const int64_t* positions,
                               const float* cos_sin, int max_position, int rotary_dim, int interleaved, void* q_out,
                               int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* key_cache,
                               void* value_cache, pkv_dtype cache_dtype, const int64_t* slot_mapping, int T, int NB,
                               int bs, int Hq, int Hkv, int d, float k_scale, float v_scale, int32_t* err_word,
                               pkv_stream_t stream) {
    if (T < 0 || Hq < 0 || Hkv < 0 || d < 1 || max_position < 1 || rotary_dim < 0) return PKV_ERR_INVALID_ARG;
    if (in_dtype != PKV_F32 && in_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (d % 16 != 0 || d > 512 || rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (rotary_dim > d) return PKV_ERR_INVALID_ARG;
    if (Hq > 65535 || Hkv > 65535) return PKV_ERR_UNSUPPORTED;
    const bool cached = key_cache != nullptr;
    if (cached != (value_cache != nullptr) || cached != (slot_mapping != nullptr)) return PKV_ERR_INVALID_ARG;
    if (cached) {
        if (cache_dtype != PKV_F32 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3)
            return PKV_ERR_UNSUPPORTED;
        if (NB < 1 || bs < 1 || (long long)NB * bs > (1LL << 40)) return PKV_ERR_INVALID_ARG;
        if (cache_dtype == PKV_FP8_E4M3 && (!finite_pos(k_scale) || !finite_pos(v_scale))) return PKV_ERR_INVALID_ARG;
    } else {
        cache_dtype = PKV_BF16;
    }
    if (T == 0) return PKV_OK;
    // which of Q, K and V there are; what comes in has to go out
    const bool has_q = query != nullptr, has_k = key != nullptr;
    if (has_q != (q_out != nullptr) || has_q != (Hq > 0)) return PKV_ERR_INVALID_ARG;
    if ((has_k || cached) != (Hkv > 0) || has_k != (cached || k_out != nullptr) || cached != (value != nullptr))
        return PKV_ERR_INVALID_ARG;
    if (!has_q && !has_k) return PKV_ERR_INVALID_ARG;
    if (!positions || (!cos_sin && rotary_dim > 0)) return PKV_ERR_INVALID_ARG;
    const int eb = in_dtype == PKV_F32 ? 4 : 2;
    struct Rows {
        const void* at;
        int64_t stride;
        int heads;
    };
    const int64_t far = 1LL << 46;                   // (sums of sizes below stay in 64 bits)
    if (cached && ((int64_t)NB * bs > far / d || (int64_t)NB * bs * d > far / Hkv)) return PKV_ERR_INVALID_ARG;
    const Rows rows[5] = {{query, q_stride, Hq}, {key, k_stride, Hkv}, {value, v_stride, Hkv},
                          {q_out, q_out_stride, Hq}, {k_out, k_out_stride, Hkv}};
    for (const Rows& r : rows) {
        if (r.at == nullptr) continue;
        if (!aligned16(r.at) || r.stride < (int64_t)r.heads * d || r.stride > far / T || r.stride * eb % 16 != 0)
            return PKV_ERR_INVALID_ARG;
    }
    // an output lies on its own input, row for row, or on nothing that is read or written here
    auto apart = [&](const Rows& a, const Rows& b) {
        const int64_t wa = (int64_t)a.heads * d * eb, wb = (int64_t)b.heads * d * eb;
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
        if (!overlap(a.at, b.at, (size_t)(T - 1) * a.stride * eb + wa, (size_t)(T - 1) * b.stride * eb + wb)) return true;
        if (a.stride != b.stride) return false;
        const int64_t s = a.stride * eb, off = (int64_t)((x > y ? x - y : y - x) % (uintptr_t)s);
        const int64_t ab = x > y ? (s - off) % s : off;          // from a row of a to the next row of b
        return ab >= wa && s - ab >= wb;
    };
    for (int o = 3; o < 5; ++o) {
        if (rows[o].at == nullptr) continue;
        for (int i = 0; i < o; ++i) {
            if (rows[i].at == nullptr) continue;
            if (i == o - 3 && rows[i].at == rows[o].at && (rows[i].stride == rows[o].stride || T == 1)) continue;
            if (!apart(rows[o], rows[i])) return PKV_ERR_INVALID_ARG;
        }
    }
    if (cached) {
        const size_t pool = (size_t)NB * bs * Hkv * d *
                            (cache_dtype == PKV_F32 ? 4 : (cache_dtype == PKV_BF16 ? 2 : 1));
        if (overlap(key_cache, value_cache, pool, pool)) return PKV_ERR_INVALID_ARG;
        for (const Rows& r : rows)
            for (const void* c : {(const void*)key_cache, (const void*)value_cache})
                if (r.at && overlap(r.at, c, (size_t)((T - 1) * r.stride + (int64_t)r.heads * d) * eb, pool))
                    return PKV_ERR_INVALID_ARG;
    }
    if (!aligned16(cos_sin) || (reinterpret_cast<uintptr_t>(positions) & 7u) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) || !aligned16(key_cache) || !aligned16(value_cache))
        return PKV_ERR_INVALID_ARG;
    RotaryParams p{};
    p.q = query; p.k = key; p.v = value; p.q_out = q_out; p.k_out = k_out;
    p.positions = positions; p.cos_sin = cos_sin; p.key_cache = key_cache; p.value_cache = value_cache;
    p.slot_mapping = slot_mapping; p.err = err_word;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
    p.T = T; p.Hq = has_q ? Hq : 0; p.Hk = has_k ? Hkv : 0; p.Hv = cached ? Hkv : 0; p.Hkv = Hkv;
    p.d = d; p.rot = rotary_dim; p.max_position = max_position; p.interleaved = interleaved != 0;
    p.NB = NB; p.bs = bs; p.k_scale = k_scale; p.v_scale = v_scale;
    return from_cuda(launch_rotary(p, in_dtype, cache_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

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
