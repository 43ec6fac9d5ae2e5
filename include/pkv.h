/*
 * pkv -- paged KV-cache decode attention for GB300 (sm_103a).
 *
 * C ABI of libpkv.so.  Every pointer argument is a DEVICE pointer unless its
 * comment says "host".  Every call is asynchronous on `stream`: it validates
 * its arguments on the host, enqueues kernels, and returns without waiting
 * for the GPU.  No call allocates memory or synchronises the host, so the
 * write, decode and copy calls can be recorded into a CUDA graph (tested);
 * pkv_paged_attention_decode_static is described on its own below.  The
 * caller owns every buffer, including the decode workspace.
 *
 * Layouts (all row-major, contiguous, 16-byte aligned base pointers):
 *   new tokens  key / value        [T,  Hkv, d]
 *   query / out                    [S,  Hq,  d]
 *   caches      key / value_cache  [NB, bs,  Hkv, d]   (one layer)
 *   block_tables                   int32 [S, MB]
 *   context_lens                   int32 [S]
 *   slot_mapping                   int64 [T]
 *   block_mapping                  int64 [P, 2]  (src, dst)
 * Sizes: Hq = query heads, Hkv = K/V heads (Hq % Hkv == 0; query head h
 * reads K/V head h / (Hq / Hkv)), d = head dimension, bs = tokens per
 * physical block, NB = physical blocks in the pool, MB = table entries per
 * sequence.
 *
 * Error behaviour.  Problems visible on the host (null pointers, bad sizes,
 * unsupported dtypes or shapes, a workspace that is too small) return a
 * status other than PKV_OK before anything is enqueued.  Problems visible
 * only on the device (a block id outside [0, NB), a context length above
 * max_context_len, a slot outside [0, NB * bs), a copy pair out of range) never
 * fault: the offending block, token or pair is skipped and, when `err_word`
 * is not NULL, the first such problem's code (PKV_DEVERR_*) is stored there
 * with an atomic compare-and-swap from 0.  A launch failure returns
 * PKV_ERR_CUDA.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* pkv_stream_t;   /* same handle as cudaStream_t; NULL = legacy stream */

typedef enum {
    PKV_OK = 0,
    PKV_ERR_INVALID_ARG = 1,
    PKV_ERR_UNSUPPORTED = 2,
    PKV_ERR_WORKSPACE = 3,
    PKV_ERR_CUDA = 4
} pkv_status;

typedef enum {
    PKV_F32 = 0,       /* IEEE binary32 */
    PKV_BF16 = 1,      /* bfloat16 */
    PKV_FP8_E4M3 = 2   /* OCP fp8 E4M3 ("fn": max 448, no infinities); value = code * scale */
} pkv_dtype;

/* Device-side error codes stored into *err_word. */
enum {
    PKV_DEVERR_NONE = 0,
    PKV_DEVERR_BLOCK_ID = 1,      /* a block table entry outside [0, NB) */
    PKV_DEVERR_CONTEXT_LEN = 2,   /* context_lens[s] < 0 or > max_context_len (clamped) */
    PKV_DEVERR_SLOT = 3,          /* slot_mapping[i] >= NB * bs, or a token-table slot outside [0, NB * bs) */
    PKV_DEVERR_COPY_PAIR = 4,     /* a copy pair with an id outside [0, NB), or whose destination another
                                     pair also writes or any pair reads (see pkv_copy_blocks) */
    PKV_DEVERR_TIMEOUT = 5,       /* a staged copy did not land within ~2 s; the kernel gave up */
    PKV_DEVERR_QUERY_LEN = 6,     /* prefill: a sequence's queries are < 0, more than its length or
                                     than max_query_len, or outside [0, T) (the sequence is skipped) */
    PKV_DEVERR_MOVE = 7,          /* repack: a move out of range, or whose source is not the slot the
                                     token table holds (the move is skipped) */
    PKV_DEVERR_POSITION = 8       /* rotary: a position past the table (the token is skipped) */
};

/*
 * paged_kv_write -- store each new token's K and V into its slot
 * (vLLM's reshape_and_cache).
 *
 * Source: "LLM推論の基礎とvLLMの内部", section 4 "PagedAttentionとブロック
 * 管理": the KV cache is cut into fixed-size blocks that are handed to a
 * request one at a time as its tokens arrive, so each new token lands in one
 * slot of one physical block; section 2 of the same page: an fp8 KV cache
 * (--kv-cache-dtype fp8) stores one byte per element.
 *
 * For token i with s = slot_mapping[i]: s < 0 skips the token; otherwise
 * key_cache[s / bs][s % bs][h][:] = convert(key[i][h][:]) for every K/V head
 * h, and the same for value.  Conversions: f32->f32, bf16->bf16, bf16->f32
 * exact; f32->bf16 round to nearest even; (f32|bf16)->E4M3 stores
 * e4m3(float(x) / k_scale) (v_scale for V) with one IEEE fp32 divide,
 * round-to-nearest-even and saturation to +-448.
 * Supported: in_dtype in {F32, BF16}; cache_dtype in {F32, BF16, FP8_E4M3};
 * d a multiple of 8, at most 512.  T == 0 is a no-op.  Duplicate slots in
 * one call race (which token wins is unspecified).
 */
PKV_API pkv_status pkv_paged_kv_write(const void* key, const void* value, pkv_dtype in_dtype,
                              void* key_cache, void* value_cache, pkv_dtype cache_dtype,
                              const int64_t* slot_mapping, int T,
                              int NB, int bs, int Hkv, int d,
                              float k_scale, float v_scale,
                              int32_t* err_word, pkv_stream_t stream);

/*
 * Bytes of workspace pkv_paged_attention_decode needs for these sizes and
 * this partition request (see below); 0 for invalid arguments.  The
 * workspace holds a 256-byte scheduling header and, when a sequence may span
 * several partitions, one (max, sum, weighted sum) triple per (sequence,
 * query head, partition or chunk; see below).  The header must be zero before a workspace is
 * first used (every decode leaves it zero when it completes, so zero-filling
 * once at allocation is enough).  One workspace must not be used by two
 * decodes that may run at the same time.
 */
PKV_API size_t pkv_decode_workspace_size(int S, int Hq, int Hkv, int d, int bs,
                                 int max_context_len, int partition_size);

/*
 * Partition size (tokens) that a decode with these arguments will use:
 * the request itself when it is > 0, no split (returns 0) when it is -1,
 * and the library's choice when it is 0 (an E4M3 cache on the tensor-core
 * kernel may then take twice this size, in the same workspace; see
 * pkv_paged_attention_decode).  Returns -1 for invalid arguments.
 */
PKV_API int pkv_decode_partition_size(int S, int Hq, int Hkv, int d, int bs,
                              int max_context_len, int partition_size);

/*
 * paged_attention_decode -- one query token per sequence attends to every
 * cached token of that sequence, read through its block table.
 *
 * Source: "LLM推論の基礎とvLLMの内部", section 4: each request keeps a table
 * from logical blocks to physical blocks and the attention kernel reads K/V
 * through it; section 12 of the same page: PagedAttention changes where K/V
 * live, not what attention computes; section 2: GQA lets several query
 * heads share one K/V head.  "vLLM 内部構造 (2) — PagedAttention", section
 * "ブロックテーブル": logically contiguous, physically scattered blocks.
 *
 * For sequence s with n = context_lens[s] and query head h (K/V head
 * kvh = h / (Hq / Hkv)):
 *   k_t, v_t = key/value_cache[block_tables[s][t / bs]][t % bs][kvh], t < n
 *   x_t = scale * <query[s][h], k_t>,  p = softmax(x),  out[s][h] = sum p_t v_t
 * (for E4M3 caches k_t and v_t are code * k_scale and code * v_scale).  A
 * sequence with n == 0 gets zeros.  Arithmetic is fp32 with fp32
 * accumulation; out has the dtype of query.
 *
 * Long contexts are split into partitions of `partition_size` tokens
 * (a multiple of bs): each partition keeps its own running max and sum, and
 * a second pass merges them (M = max m_p, L = sum e^(m_p - M) l_p,
 * O = sum e^(m_p - M) acc_p / L).  When a decode is split, each sequence's
 * last, partial partition is processed in chunks of a quarter partition
 * (rounded down to a multiple of 32 tokens; partitions under 128 tokens are
 * not cut), which are merged like partitions: the launch then ends on small
 * pieces of work.  With an E4M3 cache on the tensor-core kernel, a sequence
 * of four or more full partitions has its last full partition cut into
 * chunks too.  partition_size: 0 = library choice,
 * -1 = never split, > 0 = that size.  The library's choice depends on the
 * sizes alone (so does the workspace size); an E4M3 cache on the
 * tensor-core kernel then takes twice that partition where the launch keeps
 * at least half as many units and the same workspace holds its partial
 * results (its units are bound by their own arithmetic, and fewer, longer
 * ones end the launch sooner).  When any sequence may span more than
 * one partition, `workspace` must hold pkv_decode_workspace_size(...) bytes,
 * else PKV_ERR_WORKSPACE is returned.
 *
 * max_context_len (host) must be >= every context_lens[s] and <= MB * bs; it
 * sizes the launch without reading device memory.  Supported: q_dtype in
 * {F32, BF16}; cache_dtype in {F32, BF16, FP8_E4M3}; d in {64, 128};
 * bs in {16, 32}; any group size Hq / Hkv >= 1 (a K/V head's query heads
 * are processed up to 8 at a time, each such set reading the head's K/V).
 * For E4M3 caches the query is rounded to fp16 for the tensor-core
 * products, so |query| must stay below 65504.
 */
PKV_API pkv_status pkv_paged_attention_decode(void* out, const void* query, pkv_dtype q_dtype,
                                      const void* key_cache, const void* value_cache,
                                      pkv_dtype cache_dtype,
                                      const int32_t* block_tables, int MB,
                                      const int32_t* context_lens, int S, int max_context_len,
                                      int Hq, int Hkv, int d, int bs, int NB,
                                      float scale, float k_scale, float v_scale,
                                      int partition_size,
                                      void* workspace, size_t workspace_bytes,
                                      int32_t* err_word, pkv_stream_t stream);

/*
 * paged_kv_write_decode -- pkv_paged_kv_write of one new token per sequence
 * followed by pkv_paged_attention_decode, in one launch (plus the merge
 * when split).  key/value [S, Hkv, d] (in_dtype f32 or bf16) are the new
 * tokens, slot_mapping [S] int64 their slots, which must be the slots of
 * the sequences' last positions (context_lens[s] - 1, through
 * block_tables); a negative slot skips that sequence's write, as in
 * paged_kv_write.  The caches end up as after the two calls and the output
 * equals theirs bit for bit.  The decode unit that holds a sequence's last
 * token puts the converted new K/V into its staged rows and stores them to
 * the slot.  Supported: the tensor-core decode's dtypes (see
 * pkv_paged_attention_decode_ex); anything else returns PKV_ERR_UNSUPPORTED.
 * Source: the two calls' passages; one launch per step instead of two.
 */
PKV_API pkv_status pkv_paged_kv_write_decode(void* out, const void* query, pkv_dtype q_dtype,
                                             const void* key, const void* value, pkv_dtype in_dtype,
                                             void* key_cache, void* value_cache, pkv_dtype cache_dtype,
                                             const int64_t* slot_mapping,
                                             const int32_t* block_tables, int MB,
                                             const int32_t* context_lens, int S, int max_context_len,
                                             int Hq, int Hkv, int d, int bs, int NB,
                                             float scale, float k_scale, float v_scale,
                                             int partition_size,
                                             void* workspace, size_t workspace_bytes,
                                             int32_t* err_word, pkv_stream_t stream);

/* Kernel choice for pkv_paged_attention_decode_ex. */
typedef enum {
    PKV_DECODE_AUTO = 0,          /* tensor cores where supported, else CUDA cores */
    PKV_DECODE_CUDA_CORES = 1,    /* the CUDA-core kernel (every dtype) */
    PKV_DECODE_TENSOR_CORES = 2   /* the tensor-core kernel; PKV_ERR_UNSUPPORTED where it does not apply
                                     (it needs a bf16 query with a bf16 cache, or an E4M3 cache) */
} pkv_decode_kernel;

/*
 * Same as pkv_paged_attention_decode, with an explicit kernel choice
 * (`kernel` is a pkv_decode_kernel).  Both kernels compute the same
 * function; the choice exists so the two can be measured against each
 * other.
 */
PKV_API pkv_status pkv_paged_attention_decode_ex(void* out, const void* query, pkv_dtype q_dtype,
                                         const void* key_cache, const void* value_cache,
                                         pkv_dtype cache_dtype,
                                         const int32_t* block_tables, int MB,
                                         const int32_t* context_lens, int S, int max_context_len,
                                         int Hq, int Hkv, int d, int bs, int NB,
                                         float scale, float k_scale, float v_scale,
                                         int partition_size,
                                         void* workspace, size_t workspace_bytes,
                                         int32_t* err_word, pkv_stream_t stream, int kernel);

/*
 * Partition size (tokens) a decode launch with these arguments uses:
 * pkv_decode_partition_size's answer, except that with the library's choice
 * (partition_size 0) an E4M3 cache on the tensor-core kernel may take twice
 * it (see pkv_paged_attention_decode; the workspace size is the same).
 * `kernel` is a pkv_decode_kernel; NB is the number of cache blocks.  The
 * paged decode, the fused write + decode and the token-table decode follow
 * the same rule.  Returns 0 for no split, -1 for invalid arguments (and
 * for PKV_DECODE_TENSOR_CORES where that kernel does not apply).  Touches
 * no device memory.
 */
PKV_API int pkv_decode_launch_partition_size(int S, int Hq, int Hkv, int d, int bs, int NB,
                                             int max_context_len, int partition_size,
                                             pkv_dtype q_dtype, pkv_dtype cache_dtype, int kernel);

/*
 * copy_blocks -- copy-on-write duplication of physical blocks.
 *
 * Source: "LLM推論の基礎とvLLMの内部", section 4: blocks of a shared prefix
 * carry a reference count and are copied when written (copy-on-write);
 * "vLLM 内部構造 (2) — PagedAttention", section "共有": many requests with
 * the same system prompt point at one set of physical blocks.
 *
 * For every layer l < num_layers and pair p < P with
 * (src, dst) = block_mapping[p]: block dst of key_caches[l] and of
 * value_caches[l] becomes a byte copy of block src (block_bytes bytes each,
 * = bs * Hkv * d * element size).  key_caches / value_caches are HOST arrays
 * of num_layers device pointers (at most 256 layers); the call copies them
 * into the launch, so the arrays may be freed when it returns.  block_bytes
 * must be a multiple of 16.
 *
 * The pairs are copied in no fixed order, so the destinations must be
 * distinct and must not be sources (the host that decides copy-on-write
 * guarantees this).  A pair with an id outside [0, NB) is always skipped.
 * When err_word is not NULL the pairs are also checked against each other:
 * a pair whose destination another in-pool pair also writes, or any
 * in-pool pair (itself included) reads, is skipped, and PKV_DEVERR_COPY_PAIR
 * is reported; the other pairs are copied.  This check scans the whole
 * mapping in every CTA of the copy (16 bytes per pair, from L2), which is
 * negligible for tens of pairs and grows with P * P for thousands.  With
 * err_word NULL nothing is checked and such pairs race.
 */
PKV_API pkv_status pkv_copy_blocks(void* const* key_caches, void* const* value_caches, int num_layers,
                           const int64_t* block_mapping, int P, int NB, size_t block_bytes,
                           int32_t* err_word, pkv_stream_t stream);

/*
 * Bytes of fixed device scratch behind pkv_paged_attention_decode_static
 * (32 MiB).
 */
#define PKV_STATIC_SCRATCH_BYTES (32u << 20)

/*
 * pkv_paged_attention_decode_static -- the same decode, for callers that
 * cannot allocate device memory.
 *
 * This call has no counterpart on the pages: it is a convenience of this
 * library.  pkv_paged_attention_decode needs a workspace that its caller
 * allocates.  Some callers cannot allocate device memory where they decode:
 * an engine that reserves all of its memory at start-up and forbids later
 * allocations, a latency-critical loop that must not wait on the allocator,
 * a foreign-language caller that holds raw pointers but no allocator.  This
 * entry point takes the same arguments minus the workspace and allocates
 * nothing: its scratch is a fixed array of PKV_STATIC_SCRATCH_BYTES in
 * device memory that the library defines at file scope.  Every GPU that
 * loads the library holds that array until the process exits.  The caller
 * still passes and owns every input and output.
 *
 * Limits and behaviour:
 *  - The arguments are checked as pkv_paged_attention_decode checks them,
 *    with the same status codes, before anything is enqueued.
 *  - The scratch the call needs is pkv_decode_workspace_size(...) for the
 *    same sizes and partition request.  If that exceeds
 *    PKV_STATIC_SCRATCH_BYTES the call returns PKV_ERR_WORKSPACE and
 *    enqueues nothing; a larger partition_size needs less scratch.
 *  - `stream` must belong to the current device (the array used is the
 *    current device's); a stream of another device gives
 *    PKV_ERR_INVALID_ARG and nothing is enqueued.
 *  - The first call on a device looks up the array's device address (with
 *    that device current) and caches it with the device's CUDA context.
 *    After a device reset (a new context) the next call looks the address
 *    up again.
 *  - Each call clears the array's 256-byte work-counter header on `stream`
 *    (a memset) before the decode; the rest keeps the previous call's
 *    contents and needs no clearing.
 *  - All calls share the one array per device: two calls whose work may
 *    overlap on the GPU (different streams, or different host threads)
 *    race and give wrong results.  Serialise them.
 *  - The call makes no cudaMalloc or cudaFree and no other allocating call.
 */
PKV_API pkv_status pkv_paged_attention_decode_static(void* out, const void* query, pkv_dtype q_dtype,
                                                     const void* key_cache, const void* value_cache,
                                                     pkv_dtype cache_dtype,
                                                     const int32_t* block_tables, int MB,
                                                     const int32_t* context_lens, int S, int max_context_len,
                                                     int Hq, int Hkv, int d, int bs, int NB,
                                                     float scale, float k_scale, float v_scale,
                                                     int partition_size,
                                                     int32_t* err_word, pkv_stream_t stream);

/*
 * paged_attention_prefill -- several query tokens per sequence, causal: a
 * chunk of a prompt (chunked prefill) or the tokens a speculative decoder
 * proposes, attending through the same block tables.
 *
 * Source: "LLM推論の基礎とvLLMの内部", section 6: chunked prefill runs a
 * long prompt in per-step pieces next to other requests' decodes; section 3:
 * the V1 scheduler gives every request the tokens it still has to compute,
 * speculative ones included, without separate prefill and decode phases.
 *
 * query/out [T, Hq, d] pack every sequence's queries: those of sequence s
 * are rows query_start[s] .. query_start[s+1] (int32 [S+1], device, rising,
 * query_start[S] = T).  They are the sequence's last q_len tokens, whose
 * K/V are already in the cache (pkv_paged_kv_write first): query i sits at
 * position p = context_lens[s] - q_len + i and attends to tokens 0..p.
 * partition_size splits long key ranges like the decode's (0 = library
 * choice, -1 = never, > 0 = that many tokens, a multiple of bs); then
 * `workspace` must hold pkv_prefill_workspace_size(...) bytes, its first
 * 256 bytes zero before first use.  max_query_len >= every q_len and
 * max_context_len >= every length (host values that size the launch).
 * Supported: bf16 query and bf16 cache (tensor cores), d in {64, 128}, bs in
 * {16, 32}; anything else returns PKV_ERR_UNSUPPORTED.  Runs a tcgen05
 * kernel (PKV_PREFILL_AUTO of pkv_paged_attention_prefill_ex).
 */
PKV_API size_t pkv_prefill_workspace_size(int S, int num_query_tokens, int max_query_len, int Hq, int Hkv, int d,
                                          int bs, int max_context_len, int partition_size);
PKV_API pkv_status pkv_paged_attention_prefill(void* out, const void* query, pkv_dtype q_dtype,
                                               const void* key_cache, const void* value_cache,
                                               pkv_dtype cache_dtype,
                                               const int32_t* block_tables, int MB,
                                               const int32_t* context_lens, const int32_t* query_start,
                                               int S, int num_query_tokens, int max_query_len,
                                               int max_context_len, int Hq, int Hkv, int d, int bs, int NB,
                                               float scale, int partition_size,
                                               void* workspace, size_t workspace_bytes,
                                               int32_t* err_word, pkv_stream_t stream);

/* Kernel choice for pkv_paged_attention_prefill_ex. */
typedef enum {
    PKV_PREFILL_AUTO = 0,         /* a tcgen05 kernel: two tiles per unit when the (sequence, K/V head)
                                     pairs average 256 or more (query, head) rows, else one */
    PKV_PREFILL_MMA_SYNC = 1,     /* warp-level mma.sync: tiles of 16 (query, head) rows, one warp each */
    PKV_PREFILL_TCGEN05 = 2,      /* tcgen05.mma with tensor-memory accumulators: tiles of 128 rows,
                                     one CTA each */
    PKV_PREFILL_TCGEN05_2TILE = 3 /* the same with two 128-row tiles per unit reading each K/V stage
                                     once, each tile with its own softmax warpgroup */
} pkv_prefill_kernel;

/*
 * Same as pkv_paged_attention_prefill, with an explicit kernel choice
 * (`kernel` is a pkv_prefill_kernel).  Both kernels compute the same
 * function with the same partitioning and workspace; the choice exists so
 * the two can be measured against each other.
 */
PKV_API pkv_status pkv_paged_attention_prefill_ex(void* out, const void* query, pkv_dtype q_dtype,
                                                  const void* key_cache, const void* value_cache,
                                                  pkv_dtype cache_dtype,
                                                  const int32_t* block_tables, int MB,
                                                  const int32_t* context_lens, const int32_t* query_start,
                                                  int S, int num_query_tokens, int max_query_len,
                                                  int max_context_len, int Hq, int Hkv, int d, int bs, int NB,
                                                  float scale, int partition_size,
                                                  void* workspace, size_t workspace_bytes,
                                                  int32_t* err_word, pkv_stream_t stream, int kernel);

/* ------------------------------------------------------------------------
 * Token tables and repacking.
 *
 * Source: "LLM推論の「見えないメモリ問題」を解く：トークンレベル仮想化でKV
 * キャッシュを再利用可能にする「vToken」", sections on token-level
 * virtualisation and asynchronous repacking: a token table maps each live
 * token of a sequence, in logical order, to its physical slot; a deletion
 * policy removes tokens from the table; repacking moves the survivors of
 * sparse blocks to free slots of other blocks, rewrites their table entries
 * and releases the emptied blocks.  Attention reads through the table, so
 * the cache pools and captured CUDA graphs are untouched by repacking.
 *
 * A slot is block * bs + offset, i.e. the row of the cache seen as
 * [NB * bs, Hkv, d].
 * ------------------------------------------------------------------------ */

/*
 * token_attention_decode -- the decode of pkv_paged_attention_decode, with
 * each sequence's K/V reached through its token table instead of a block
 * table: token_slots [S, MT] int32 (device) lists the slots of the
 * sequence's live tokens in logical order; num_tokens [S] (device) how many;
 * max_tokens >= every num_tokens (host value; <= MT).  Output, scales,
 * partitioning and workspace are those of the decode
 * (pkv_decode_workspace_size(S, Hq, d, max_tokens, partition_size)).
 * Supported: the tensor-core decode's dtypes (bf16 query and cache, or an
 * E4M3 cache with a bf16 or fp32 query), d in {64, 128}, bs in {16, 32};
 * anything else returns PKV_ERR_UNSUPPORTED.  A slot outside the pool is
 * treated as an absent token and reported (PKV_DEVERR_SLOT).
 */
PKV_API pkv_status pkv_token_attention_decode(void* out, const void* query, pkv_dtype q_dtype,
                                              const void* key_cache, const void* value_cache,
                                              pkv_dtype cache_dtype,
                                              const int32_t* token_slots, int MT,
                                              const int32_t* num_tokens, int S, int max_tokens,
                                              int Hq, int Hkv, int d, int bs, int NB,
                                              float scale, float k_scale, float v_scale,
                                              int partition_size,
                                              void* workspace, size_t workspace_bytes,
                                              int32_t* err_word, pkv_stream_t stream);

/*
 * repack_tokens -- apply moves [M, 4] int64 (device) = (sequence, logical
 * index, source slot, destination slot): for every layer, the token's K and
 * V rows (token_bytes = Hkv * d * element size bytes each) are copied from
 * the source slot to the destination, then token_slots[sequence][index]
 * becomes the destination.  key_caches / value_caches are host arrays of
 * num_layers (<= 256) device pointers.  Preconditions: destinations are free
 * slots, distinct, and no move's destination is another move's source; each
 * (sequence, index) appears once.  A move out of range or whose source is
 * not what the table holds is skipped and reported (PKV_DEVERR_MOVE).
 */
PKV_API pkv_status pkv_repack_tokens(void* const* key_caches, void* const* value_caches, int num_layers,
                                     int32_t* token_slots, int MT, int S, const int64_t* moves, int M,
                                     int NB, int bs, size_t token_bytes, int32_t* err_word,
                                     pkv_stream_t stream);

/*
 * vtoken_plan -- host planner for repacking (host arrays).  Per sequence,
 * over the blocks only that sequence uses (a block several sequences
 * reference is left alone): the sequence needs k = ceil(live tokens in
 * those blocks / bs) blocks; the k with the most live tokens stay (lower id
 * first on ties); its tokens in the others move, in logical order, to the
 * free slots of the kept blocks, lowest slot first; the others are then
 * empty and are listed in `freed` (ascending per sequence).  Writes up to
 * max_moves moves [.., 4] and max_freed block ids, and the counts needed in
 * *num_moves / *num_freed.  Returns PKV_ERR_INVALID_ARG for a slot outside
 * the pool or a sequence holding one slot twice, PKV_ERR_WORKSPACE when an
 * output array is too small (counts still set, arrays untouched).  Scratch
 * host memory during the call: one bit per slot of the pool and about ten
 * bytes per block, plus the moves found.
 */
PKV_API pkv_status pkv_vtoken_plan(const int32_t* token_slots, int MT, const int32_t* num_tokens, int S, int bs,
                                   int NB, int64_t* moves, int64_t max_moves, int64_t* num_moves,
                                   int32_t* freed, int64_t max_freed, int64_t* num_freed);

/* ------------------------------------------------------------------------
 * Sliding window with sinks.
 *
 * Source: "LLM推論の「見えないメモリ問題」を解く … vToken", section on token
 * eviction: keeping the first tokens and a window of recent ones bounds what
 * a decoding step reads.
 *
 * A query at position p sees token t when t <= p and (t < num_sinks or
 * t > p - window): the first num_sinks tokens of its sequence and the last
 * `window` tokens, its own among them.  window >= 1, num_sinks >= 0; a
 * window or sinks beyond a sequence's length hide nothing.  Blocks none of
 * whose tokens a call's queries see are not read, and neither are their
 * entries of the block table: a caller that manages its own blocks may have
 * reused them (the host block manager, pkv_pool_*, frees a sequence's blocks
 * all at once).  Tokens of a read block that no query sees may hold anything,
 * NaN included.
 * ------------------------------------------------------------------------ */

/*
 * Bytes of workspace for pkv_paged_attention_decode_window, and (window 0:
 * no window) for pkv_paged_attention_decode_kv4; 0 for invalid arguments.
 * It is used as pkv_decode_workspace_size describes, and holds partial
 * results for the tokens a window leaves visible only.
 *
 * The size does not grow with S or max_context_len alone: few sequences are
 * split further than many.  A loop may give every call the workspace of its
 * largest one: with partition_size 0 a call whose own choice wants more takes
 * fewer, longer partitions that fit, down to none (any workspace of 256 bytes
 * serves).  A workspace of the largest size over all shapes of the loop keeps
 * every call at its fastest.  An explicit partition_size is never replaced:
 * short of its size, the call returns PKV_ERR_WORKSPACE, as it does without a
 * workspace where it would split.  The same holds for the workspaces of
 * pkv_paged_attention_prefill_window (for which the number of queries counts
 * too) and, above the logits' part, pkv_token_attention_decode_scored.
 */
PKV_API size_t pkv_decode_window_workspace_size(int S, int Hq, int Hkv, int d, int bs, int max_context_len, int window,
                                                int num_sinks, int partition_size);

/*
 * paged_attention_decode_window -- pkv_paged_attention_decode_ex over the
 * visible tokens only (the sequence's query is at context_lens[s] - 1).
 * Every dtype, size, kernel choice and status of that call; partitions
 * divide the visible tokens.
 */
PKV_API pkv_status pkv_paged_attention_decode_window(void* out, const void* query, pkv_dtype q_dtype,
                                                     const void* key_cache, const void* value_cache,
                                                     pkv_dtype cache_dtype,
                                                     const int32_t* block_tables, int MB,
                                                     const int32_t* context_lens, int S, int max_context_len,
                                                     int Hq, int Hkv, int d, int bs, int NB,
                                                     float scale, float k_scale, float v_scale,
                                                     int window, int num_sinks, int partition_size,
                                                     void* workspace, size_t workspace_bytes,
                                                     int32_t* err_word, pkv_stream_t stream, int kernel);

/*
 * paged_attention_prefill_window -- pkv_paged_attention_prefill with each
 * query of the chunk under its own window.  The workspace is
 * pkv_prefill_window_workspace_size(...) bytes.  A K or V value that is not
 * finite, in a token that some query of the chunk sees, may reach other
 * queries of the same chunk (their weight 0 times it).
 */
PKV_API size_t pkv_prefill_window_workspace_size(int S, int num_query_tokens, int max_query_len, int Hq, int Hkv, int d,
                                                 int bs, int max_context_len, int window, int num_sinks,
                                                 int partition_size);
PKV_API pkv_status pkv_paged_attention_prefill_window(void* out, const void* query, pkv_dtype q_dtype,
                                                      const void* key_cache, const void* value_cache,
                                                      pkv_dtype cache_dtype,
                                                      const int32_t* block_tables, int MB,
                                                      const int32_t* context_lens, const int32_t* query_start,
                                                      int S, int num_query_tokens, int max_query_len,
                                                      int max_context_len, int Hq, int Hkv, int d, int bs, int NB,
                                                      float scale, int window, int num_sinks, int partition_size,
                                                      void* workspace, size_t workspace_bytes,
                                                      int32_t* err_word, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * A cache held in 4 bits.
 *
 * Source: "LLM推論の基礎とvLLMの内部", section 2: the bytes per K/V element
 * set how many tokens a pool holds; 4-bit codes with a scale and a zero per
 * 32 values take 5 bits a value (bf16: 16, E4M3: 8).
 *
 * key_cache / value_cache are byte arrays [NB, Hkv, bs * (d/2 + d/8)]: each
 * K/V head of a block holds its tokens' codes, then their fp16 scales, then
 * their fp16 zeros.  A row of d values x becomes y = x / k_scale (v_scale),
 * one IEEE fp32 divide, clamped to +-65504, and each group of 32 of them
 *   zero  = fp16(min y)
 *   scale = fp16(max(max y - zero, 0) / 15)
 *   code  = clamp(rint((y - zero) / scale), 0, 15), 0 where scale is 0
 * in fp32 with rounding to nearest even; the code stands for
 * (zero + scale * code) * k_scale.  A NaN in a group makes all of it NaN.
 * The tensor scales bring values into fp16's range; 1 suits values between
 * about 1e-3 and 1e4.  With G = d / 32, element e of token t of the block
 * is code c of the 32-bit word w of that head (code c in bits 4c .. 4c + 3):
 *   K: w = (4 t + e % 32 / 8) G + e / 32,              c = e % 8
 *   V: w = ((t / 8 * 8 + e % 32 / 4) 4 + t / 2 % 4) G + e / 32,
 *                                                      c = 4 (t % 2) + e % 4
 * and its scale (zero) is the half number, past the codes (and the scales),
 *   K: t G + e / 32          V: (t / 2 G + e / 32) 2 + t % 2
 * (integer divisions).  d in {64, 128}; bs in {16, 32}.  pkv_copy_blocks
 * copies such blocks with block_bytes = pkv_kv4_block_bytes(...).
 * ------------------------------------------------------------------------ */

/* Bytes of one block of a 4-bit K (or V) cache; 0 for unsupported sizes. */
PKV_API size_t pkv_kv4_block_bytes(int bs, int Hkv, int d);

/*
 * paged_kv4_write -- pkv_paged_kv_write into a 4-bit cache: key/value
 * [T, Hkv, d] (F32 or BF16), slot_mapping [T] as there; of a slot that one
 * call names twice the values are unspecified (codes of one token may meet
 * the scale of the other).
 */
PKV_API pkv_status pkv_paged_kv4_write(const void* key, const void* value, pkv_dtype in_dtype,
                                       void* key_cache, void* value_cache, const int64_t* slot_mapping, int T,
                                       int NB, int bs, int Hkv, int d, float k_scale, float v_scale,
                                       int32_t* err_word, pkv_stream_t stream);

/*
 * paged_kv4_read -- the values of the slots: key/value [T, Hkv, d] (F32, or
 * BF16 rounded to nearest even) of slots[i] (int64 [T]; a negative slot
 * leaves row i as it was, one outside the pool too and is reported), to move
 * a sequence to a cache of another dtype or to recompute with.
 */
PKV_API pkv_status pkv_paged_kv4_read(void* key, void* value, pkv_dtype out_dtype,
                                      const void* key_cache, const void* value_cache, const int64_t* slots, int T,
                                      int NB, int bs, int Hkv, int d, float k_scale, float v_scale,
                                      int32_t* err_word, pkv_stream_t stream);

/*
 * paged_attention_decode_kv4 -- pkv_paged_attention_decode over a 4-bit
 * cache, under a sliding window when window > 0 (0: every token).  bf16
 * query and output (anything else returns PKV_ERR_UNSUPPORTED).  The query
 * goes through fp16 for the products, after a power of two that brings the
 * largest finite value of up to 8 heads of a K/V head below 1024: finite
 * values up to 2^100 are fine, and a head keeps its bf16 precision down to
 * 2^-16 times the largest of those heads.  Workspace:
 * pkv_decode_window_workspace_size(...) with the same window and sinks.
 */
PKV_API pkv_status pkv_paged_attention_decode_kv4(void* out, const void* query, pkv_dtype q_dtype,
                                                  const void* key_cache, const void* value_cache,
                                                  const int32_t* block_tables, int MB,
                                                  const int32_t* context_lens, int S, int max_context_len,
                                                  int Hq, int Hkv, int d, int bs, int NB,
                                                  float scale, float k_scale, float v_scale,
                                                  int window, int num_sinks, int partition_size,
                                                  void* workspace, size_t workspace_bytes,
                                                  int32_t* err_word, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Eviction by accumulated attention weight.
 *
 * Source: "LLM推論の「見えないメモリ問題」を解く … vToken", section on token
 * eviction: policies that drop the tokens that received little attention
 * free slots inside blocks, which the token tables and pkv_repack_tokens
 * turn into free blocks.
 * ------------------------------------------------------------------------ */

/*
 * token_attention_decode_scored -- pkv_token_attention_decode (with an
 * explicit partition_size the same output, bit for bit; the library's choice
 * splits a small launch further here) that also adds, to scores[s][t] (fp32
 * [S, MT], row length MT as the table's) of every live token t, the attention
 * weights the sequence's query gives it, summed over the Hq query heads.  The sum
 * runs in a fixed order, so equal calls give equal bits; entries past
 * num_tokens[s] are left as they were, and a slot outside the pool gets
 * weight 0.  `workspace` must hold
 * pkv_token_attention_scored_workspace_size(...) bytes: the decode's, and
 * the logits of the step (about 4 bytes per token and query head).  Its
 * header must be zero before first use, as the decode's.
 */
PKV_API size_t pkv_token_attention_scored_workspace_size(int S, int Hq, int Hkv, int d, int bs, int max_tokens,
                                                         int partition_size);
PKV_API pkv_status pkv_token_attention_decode_scored(void* out, const void* query, pkv_dtype q_dtype,
                                                     const void* key_cache, const void* value_cache,
                                                     pkv_dtype cache_dtype,
                                                     const int32_t* token_slots, int MT,
                                                     const int32_t* num_tokens, float* scores, int S, int max_tokens,
                                                     int Hq, int Hkv, int d, int bs, int NB,
                                                     float scale, float k_scale, float v_scale,
                                                     int partition_size,
                                                     void* workspace, size_t workspace_bytes,
                                                     int32_t* err_word, pkv_stream_t stream);

/*
 * evict_tokens -- cut every sequence to at most `budget` tokens.  A sequence
 * of n = num_tokens[s] <= budget tokens keeps them all.  A longer one keeps
 * its first num_first tokens, its last num_recent, and of those between the
 * budget - num_first - num_recent with the largest scores (ties: the lowest
 * index; a NaN score is below every number).  Kept tokens stay in order:
 * new_slots[s] and new_scores[s] receive their slots and scores, new_num[s]
 * their count, and evicted[s] (or NULL) the n - new_num[s] dropped tokens'
 * slots, in order, for the caller's pool.  Arrays are [S, MT] (int32, fp32)
 * and [S]; entries past the counts are left as they were.  No output may
 * overlap an input or another output: a loop swaps two tables.
 * num_first + num_recent <= budget; MT <= 2^30.  A count outside [0, MT] is clamped and
 * reported (PKV_DEVERR_CONTEXT_LEN).
 */
PKV_API pkv_status pkv_evict_tokens(const int32_t* token_slots, const float* scores, const int32_t* num_tokens,
                                    int S, int MT, int budget, int num_first, int num_recent,
                                    int32_t* new_slots, float* new_scores, int32_t* new_num, int32_t* evicted,
                                    int32_t* err_word, pkv_stream_t stream);

/* ------------------------------------------------------------------------
 * A prompt's way into the cache.
 *
 * Source: "LLM推論の基礎とvLLMの内部", section 4 (a token's K/V goes to a
 * slot as it arrives) and section 6 (a step computes prompts next to decodes).
 * ------------------------------------------------------------------------ */

/*
 * rotary_kv_write -- rotary position embedding of Q and K, and
 * pkv_paged_kv_write of the rotated K and of V, in one pass.
 *
 * query [T, Hq, d], key / value [T, Hkv, d] of in_dtype (F32 or BF16), their
 * heads contiguous, their tokens *_stride elements apart (Hq * d or Hkv * d for
 * arrays of their own, the row length where one projection left all three
 * side by side).  Token i at position p = positions[i]: the first rotary_dim
 * values of every head of Q and K are pairs j (values j and rotary_dim/2 + j;
 * interleaved != 0: values 2j and 2j + 1), and a pair (a, b) becomes
 *   (a c - b s, b c + a s),  c = cos_sin[p][j], s = cos_sin[p][rotary_dim/2 + j]
 * (fp32 [max_position, rotary_dim]), each product and sum rounded to fp32.
 * The other values, and V, stay.  The results are rounded once per output:
 *   q_out [T, Hq, d], k_out [T, Hkv, d] (in_dtype; tokens *_out_stride apart;
 *         k_out or NULL), and
 *   the slot slot_mapping[i] of key_cache / value_cache (F32, BF16 or E4M3:
 *         e4m3(x / scale) as pkv_paged_kv_write), negative: not written.
 * A token with a negative position is padding: nothing of it is read or
 * written.  One past the table is skipped too and reported
 * (PKV_DEVERR_POSITION); a slot outside the pool is not written and reported.
 * NULL query and q_out (Hq 0): only K and V.  NULL caches, value and
 * slot_mapping: nothing is stored in a cache; with NULL key and k_out too
 * only Q is rotated.  q_out may be query and k_out key (same stride); outputs
 * must not overlap anything else.  Supported: d a multiple of 16, at most
 * 512; rotary_dim a multiple of 16, at most d; strides that are multiples of
 * 16 bytes.  T == 0 is a no-op.
 */
PKV_API pkv_status pkv_rotary_kv_write(const void* query, const void* key, const void* value, pkv_dtype in_dtype,
                                       int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                       const int64_t* positions, const float* cos_sin, int max_position,
                                       int rotary_dim, int interleaved,
                                       void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                       void* key_cache, void* value_cache, pkv_dtype cache_dtype,
                                       const int64_t* slot_mapping, int T, int NB, int bs, int Hq, int Hkv, int d,
                                       float k_scale, float v_scale, int32_t* err_word, pkv_stream_t stream);

/*
 * prompt_attention -- attention over whole packed prompts whose K and V lie
 * side by side, before or without a cache (pkv_paged_attention_prefill reads a
 * cache through block tables).
 *
 * query [Tq, Hq, d] packs S sequences: rows query_start[s] .. query_start[s+1]
 * (int32 [S+1], device, rising) are sequence s's, and rows key_start[s] ..
 * key_start[s+1] of key / value [Tk, Hkv, d] its keys; the two may be one
 * array.  Heads are contiguous, tokens *_stride elements apart (Hq * d or
 * Hkv * d for arrays of their own).  With q_len queries and k_len keys, query i
 * sits at position p = k_len - q_len + i; it sees
 *   causal == 0: every key of its sequence;
 *   causal != 0: keys t <= p, and with a window (window > 0; causal only) of
 *                these t < num_sinks or t > p - window.
 * out[i][h] = softmax(scale <q, k_t>) v_t over the keys it sees ([Tq, Hq, d],
 * contiguous), zeros where there is none.  Rows of out that are no sequence's
 * are left as they were.  max_query_len and max_key_len (host) bound the
 * lengths; a sequence that breaks a bound, or whose rows leave [0, Tq) or
 * [0, Tk), is skipped and reported (PKV_DEVERR_QUERY_LEN).  A V value that is
 * not finite may reach queries of the same sequence that see other keys but
 * not this one, by way of queries that do see it (their weight 0 times it); K
 * values do not, and a query that sees no key is zeros in any case.  Keys that
 * no query of their sequence sees (behind every window) may hold anything.
 *
 * Few rows over many keys are split: partition_size 0 = library choice, -1 =
 * never, > 0 = that many keys (a multiple of 128); then `workspace` must hold
 * pkv_prompt_workspace_size(...) bytes, its first 256 zero before first use
 * (a smaller one: fewer partitions, as pkv_decode_window_workspace_size
 * says).  Supported: bf16 (sums in fp32, weights rounded to bf16), d in {64,
 * 128}, strides that are multiples of 8 elements.  out must not overlap the
 * inputs.
 */
PKV_API size_t pkv_prompt_workspace_size(int S, int num_query_tokens, int max_query_len, int max_key_len, int Hq,
                                         int Hkv, int d, int window, int num_sinks, int partition_size);
PKV_API pkv_status pkv_prompt_attention(void* out, const void* query, const void* key, const void* value,
                                        pkv_dtype dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                        const int32_t* query_start, const int32_t* key_start, int S,
                                        int num_query_tokens, int num_key_tokens, int max_query_len, int max_key_len,
                                        int Hq, int Hkv, int d, float scale, int causal, int window, int num_sinks,
                                        int partition_size, void* workspace, size_t workspace_bytes,
                                        int32_t* err_word, pkv_stream_t stream);

/*
 * paged_attention_decode_shared -- pkv_paged_attention_decode of sequences in
 * groups whose first blocks are the same physical blocks (one system prompt,
 * several samples of a prompt, questions about one document).  The shared
 * blocks are read once per group and not once per sequence; the result is the
 * decode's, up to the order of its sums.
 *
 * Source: "vLLM 内部構造 (2) — PagedAttention", section "共有": many requests
 * point at one set of physical blocks.
 *
 * Group i (of G) is the sequences group_start[i] .. group_start[i+1] (int32
 * [G+1], device, rising); the first shared_lens[i] tokens (int32 [G], device;
 * counted in whole blocks, the rest is each sequence's own) of all of them are
 * read through the table of the first.  Sequences in no group, and groups
 * that share 0 tokens, are decoded as they are.  max_shared_len (host) bounds
 * every shared_lens[i], max_group_size the sequences of every group that
 * shares a block; a group that breaks a bound is reported
 * (PKV_DEVERR_QUERY_LEN) and decoded without sharing.  Groups that overlap
 * give unspecified results.  A sequence shorter than its group's shared tokens
 * is decoded on its own, and shared tokens that no sequence sees may hold
 * anything, NaN included.  A block id outside [0, NB) is reported and its
 * tokens are absent, as in the decode.
 *
 * sharing (a pkv_sharing): PKV_SHARE_AUTO reads the shared blocks once where
 * that is estimated to be faster, and otherwise decodes every sequence on its
 * own, without a look at the groups; PKV_SHARE_ALWAYS in any case.  The estimate
 * is by the bounds: sequences on their own would read 256 MB or more again if
 * there were G groups of max_group_size (at most S sequences) that share
 * max_shared_len.  So a group that shares nothing counts too: sequences before
 * the first group and behind the last are better in none.
 * partition_size: as in the decode, for the shared tokens (rounded up to 128)
 * and the others alike.  `workspace` must hold
 * pkv_decode_shared_workspace_size(...) bytes, its first 256 zero before first
 * use (a smaller one: fewer partitions, as pkv_decode_window_workspace_size
 * says, down to sequences on their own).  Where it shares, that is 4 (d + 2)
 * bytes per sequence, head and partition of the shared tokens and of
 * max_context_len own ones (any sequence may share nothing): for 64 / 8 heads of
 * 128 and 32,768 of 33,792 tokens shared, 211 MB for 64 sequences (the decode:
 * 47) and 1.4 GB for 1,024.  Supported: bf16 query and cache; anything else returns
 * PKV_ERR_UNSUPPORTED.
 */
typedef enum { PKV_SHARE_AUTO = 0, PKV_SHARE_ALWAYS = 1 } pkv_sharing;
PKV_API size_t pkv_decode_shared_workspace_size(int S, int G, int Hq, int Hkv, int d, int bs, int max_context_len,
                                                int max_shared_len, int max_group_size, int partition_size,
                                                int sharing);
PKV_API pkv_status pkv_paged_attention_decode_shared(void* out, const void* query, pkv_dtype q_dtype,
                                                     const void* key_cache, const void* value_cache,
                                                     pkv_dtype cache_dtype, const int32_t* block_tables, int MB,
                                                     const int32_t* context_lens, const int32_t* group_start,
                                                     const int32_t* shared_lens, int S, int G, int max_context_len,
                                                     int max_shared_len, int max_group_size, int Hq, int Hkv, int d,
                                                     int bs, int NB, float scale, int partition_size, void* workspace,
                                                     size_t workspace_bytes, int32_t* err_word, pkv_stream_t stream,
                                                     int sharing);

/* ------------------------------------------------------------------------
 * The calls of the four sections above with their arguments in one array,
 * for callers whose foreign-function interface pays per argument (the Python
 * binding's converts 27 arguments in 2.4 us and one in 0.3).  words[i] is the
 * call's argument i as 64 bits: pointers and sizes as they are, integers and
 * enumerations sign-extended, floats as doubles.  Returns what the call
 * returns, PKV_ERR_INVALID_ARG for an unknown call, no array, or an integer
 * that does not fit its parameter.
 * ------------------------------------------------------------------------ */
typedef enum {
    PKV_CALL_DECODE_WINDOW = 0,    /* pkv_paged_attention_decode_window */
    PKV_CALL_PREFILL_WINDOW = 1,   /* pkv_paged_attention_prefill_window */
    PKV_CALL_KV4_WRITE = 2,        /* pkv_paged_kv4_write */
    PKV_CALL_KV4_READ = 3,         /* pkv_paged_kv4_read */
    PKV_CALL_DECODE_KV4 = 4,       /* pkv_paged_attention_decode_kv4 */
    PKV_CALL_DECODE_SCORED = 5,    /* pkv_token_attention_decode_scored */
    PKV_CALL_EVICT = 6,            /* pkv_evict_tokens */
    PKV_CALL_ROTARY_WRITE = 7,     /* pkv_rotary_kv_write */
    PKV_CALL_PROMPT = 8,           /* pkv_prompt_attention */
    PKV_CALL_DECODE_SHARED = 9     /* pkv_paged_attention_decode_shared */
} pkv_call;
PKV_API pkv_status pkv_invoke(int call, const void* words);


/* ------------------------------------------------------------------------
 * Host block manager: the bookkeeping that produces the block tables, slot
 * mappings and copy-on-write pairs the device calls consume.  Host memory
 * only; nothing here touches the GPU.
 *
 * Source: "LLM推論の基礎とvLLMの内部", section 4 "PagedAttentionとブロック
 * 管理": blocks are handed to a request one at a time as it grows, each
 * request keeps a block table, block 0 is reserved as the null block, free
 * blocks wait in a doubly linked queue, and shared blocks carry a reference
 * count and are copied before a write.  Section 5: a full block's hash
 * chains its parent's hash, its tokens and extra keys; only full blocks are
 * cached; the last prompt token is always recomputed; a finished request
 * returns its blocks tail first with their hashes kept, and the queue is
 * reused from its front (least recently freed first).  Free blocks without
 * a hash are handed out before any cached block.
 *
 * Errors: PKV_ERR_INVALID_ARG for a null pool, an unknown or duplicate
 * sequence id, or bad sizes; PKV_ERR_WORKSPACE when the pool has too few
 * free blocks (nothing is changed then).  A pool is not thread-safe.
 * ---------------------------------------------------------------------- */
typedef struct pkv_block_pool pkv_block_pool;

/* A pool of num_blocks blocks of block_size tokens (block 0 reserved, so
 * num_blocks - 1 usable).  enable_prefix_caching != 0 turns on the hash
 * chain and reuse of cached blocks. */
PKV_API pkv_status pkv_pool_create(int num_blocks, int block_size, int enable_prefix_caching,
                                   pkv_block_pool** out);
PKV_API void pkv_pool_destroy(pkv_block_pool* pool);
/* Extra key mixed into every block hash (a LoRA id, a cache salt, ...):
 * pools with different keys never share cached blocks. */
PKV_API pkv_status pkv_pool_set_extra_key(pkv_block_pool* pool, uint64_t extra_key);
PKV_API int pkv_pool_num_free_blocks(const pkv_block_pool* pool);
PKV_API int pkv_pool_num_cached_blocks(const pkv_block_pool* pool);
/* Reference count of a physical block (-1 for a bad id). */
PKV_API int pkv_pool_block_ref_count(const pkv_block_pool* pool, int block);

/* Start sequence seq_id with its prompt tokens[0..n_tokens): reuse the
 * longest cached prefix of whole blocks (never the block holding the last
 * token's position if that would leave no token to compute), take new blocks
 * for the rest.  *num_cached_tokens (optional) receives the tokens found in
 * the cache.  The prompt's K/V then go to slots block_table[t / bs] * bs +
 * t % bs for t >= *num_cached_tokens. */
PKV_API pkv_status pkv_pool_add_sequence(pkv_block_pool* pool, int64_t seq_id, const int32_t* tokens,
                                         int n_tokens, int* num_cached_tokens);

/* One more token for seq_id.  *slot receives the cache slot of its K/V.  If
 * the last block was full a new block is taken; if it is shared with another
 * sequence (after pkv_pool_fork) it is copied first: *cow_src / *cow_dst
 * receive the (src, dst) pair to pass to pkv_copy_blocks before the write,
 * else -1. */
PKV_API pkv_status pkv_pool_append_token(pkv_block_pool* pool, int64_t seq_id, int32_t token, int64_t* slot,
                                         int64_t* cow_src, int64_t* cow_dst);

/* child_id shares every block of parent_id (reference counts + 1), as for
 * parallel sampling or beam search. */
PKV_API pkv_status pkv_pool_fork(pkv_block_pool* pool, int64_t parent_id, int64_t child_id);

/* End seq_id: its blocks lose one reference each, last block first. */
PKV_API pkv_status pkv_pool_free_sequence(pkv_block_pool* pool, int64_t seq_id);

/* One decode step for n sequences at once: token tokens[i] is appended to
 * seq_ids[i] (each id once).  slot_mapping[i] receives its slot -- the input
 * of pkv_paged_kv_write -- and the copy-on-write pairs go to
 * block_mapping[0 .. 2 * *num_copies) as (src, dst) -- the input of
 * pkv_copy_blocks, to run before the write.  block_mapping must have room
 * for 2 * n entries.  If the pool cannot cover the step, PKV_ERR_WORKSPACE is
 * returned and nothing changes. */
PKV_API pkv_status pkv_pool_append_tokens(pkv_block_pool* pool, const int64_t* seq_ids, const int32_t* tokens,
                                          int n, int64_t* slot_mapping, int64_t* block_mapping, int* num_copies);

/* The decode's inputs for n sequences: tables [n, max_blocks] (padded with
 * the null block) and context_lens [n]. */
PKV_API pkv_status pkv_pool_block_tables(const pkv_block_pool* pool, const int64_t* seq_ids, int n,
                                         int32_t* tables, int max_blocks, int32_t* context_lens);

/* Copy seq_id's block table into table[0..max_blocks), padded with the null
 * block 0; *num_blocks and *num_tokens (optional) receive its length.  A
 * NULL table only queries the lengths. */
PKV_API pkv_status pkv_pool_block_table(const pkv_block_pool* pool, int64_t seq_id, int32_t* table,
                                        int max_blocks, int* num_blocks, int* num_tokens);

/* Static, human-readable text for a status. */
PKV_API const char* pkv_status_string(pkv_status status);

/* Version of this library, e.g. "pkv 0.1.0 sm_103a". */
PKV_API const char* pkv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
