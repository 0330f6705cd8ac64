/*
 * pkd -- attention over a paged KV cache on GB300 (sm_103a).
 *
 * C ABI.  Every pointer named "device" is a CUDA device address owned by the
 * caller; the library never allocates, frees or synchronises on its own (the
 * one exception is pkd_workspace_check, which reads a status word back).
 * Calls are asynchronous on the stream passed as `stream` (a cudaStream_t;
 * NULL is the legacy default stream).  All functions are thread-safe; the
 * message of the last failure is kept per host thread (pkd_last_error).
 * A process may call the library on several GPUs: each kernel's launch
 * set-up is made once per device, with that device current.
 *
 * Sources of the operations (vLLM API pages, by title and section):
 *   [TS]   vllm.v1.attention.backends.flashinfer_ts -- module docstring
 *          ("Layout", "Sliding window"), FlashInferTSImpl.forward,
 *          FlashInferTSImpl._kv_views, FlashInferTSMetadataBuilder.build,
 *          ._restrict_to_window, ._get_plan, _kv_kernel_dtype.
 *   [DASH] vllm.v1.attention.ops.dash_attention -- flash_dash_attention.
 *   [FA]   vllm.v1.attention.backends.fa_utils --
 *          FlashAttentionCuTeDSLCompileSpec (Split-KV, return_softmax_lse).
 */
#ifndef PKD_H_
#define PKD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PKD_OK = 0,
    PKD_EINVAL = 1,          /* bad pointer, size, stride or alignment */
    PKD_EUNSUPPORTED = 2,    /* valid request outside what the kernels implement */
    PKD_ECUDA = 3,           /* a CUDA runtime/driver call failed (message has the CUDA error) */
    PKD_EDEVICE_BOUNDS = 4,  /* a kernel met an out-of-range page or length (see pkd_workspace_check) */
    PKD_ETIMEOUT = 5         /* a kernel gave up waiting on one of its own copies */
} pkd_status;

typedef enum {
    PKD_BF16 = 0,
    PKD_FP16 = 1,
    PKD_FP8_E4M3 = 2,        /* e4m3 "fn": uint8 storage, no infinities [TS _kv_kernel_dtype] */
    PKD_FP32 = 3
} pkd_dtype;

/* Flags for pkd_paged_decode (pkd_paged_attention and pkd_prefix_decode take
 * PKD_FLAG_CAUSAL and PKD_FLAG_TEST_TIMEOUT). */
#define PKD_FLAG_CAUSAL 1u      /* causal mask inside the query block, exact per-token window */
#define PKD_FLAG_MMA_SMALL_M 2u /* tensor cores for sq*Hq/Hkv < 16 (already the default; kept for callers) */
#define PKD_FLAG_FMA 4u         /* CUDA cores instead (only when sq*Hq/Hkv <= 8) */
#define PKD_FLAG_GRID 8u        /* the chunked grid: one CTA per Split-KV chunk */
#define PKD_FLAG_FLAT 16u       /* the persistent flat partition whatever the shapes (batch <= 1024) */
#define PKD_FLAG_BALANCED 32u   /* the persistent per-CTA partition (16-bit caches, tensor cores) */
/* q, block_table, seq_lens, out and lse are pinned host memory (cudaHostAlloc,
 * cudaMallocHost or cudaHostRegister), which under unified addressing has the
 * same address on the device: the kernels read and write it in place over the
 * host link, with no copy before or after the launch.  kv_cache and the
 * workspace stay device memory.  Each of those five pointers is checked with
 * cudaPointerGetAttributes (host memory mapped at the same address, else
 * PKD_EINVAL).  The tcgen05 kernel, whose q goes through a tensor-map copy,
 * is not used with it: its shapes run on the chunked grid instead (the
 * workspace size and kernel name follow the flag). */
#define PKD_FLAG_HOST_IO 128u
/* Diagnostic: every wait on a stage's copy tests its barrier once instead of
 * waiting up to 200 ms, so a call reports PKD_ETIMEOUT whenever a copy has not
 * landed by its first test.  The kernels still let every issued copy land
 * before they leave.  It exists to exercise the timeout path; zero the
 * workspace again (pkd_workspace_init) after such a call.  (Of the prompts of
 * pkd_paged_attention and pkd_prefix_decode: the waits for queries, in half of
 * the CTAs from their second work item on.) */
#define PKD_FLAG_TEST_TIMEOUT 64u

/* Library version, major*10000 + minor*100 + patch. */
int pkd_version(void);

/* Message of the last non-OK status returned on this host thread ("" if none). */
const char* pkd_last_error(void);

/*
 * Bytes of workspace pkd_paged_decode needs for a plan.  The plan is fixed by
 * the shapes and by max_kv_len, an upper bound on every seq_lens entry (the
 * constant K/V capacity of [TS FlashInferTSMetadataBuilder._max_kv_len]), so
 * one workspace serves every call with the same shapes, e.g. every replay of
 * a captured CUDA graph.  chunk_tokens is the Split-KV chunk (0 = automatic;
 * otherwise a multiple of page_size).  flags as for pkd_paged_decode.
 * Returns 0 for an invalid request (the reason is in pkd_last_error).
 */
size_t pkd_paged_decode_workspace_size(int batch, int sq, int num_heads, int num_kv_heads,
                                       int head_dim, int page_size, int max_kv_len,
                                       pkd_dtype kv_dtype, int window, int chunk_tokens,
                                       unsigned flags);

/*
 * Which kernel pkd_paged_decode launches for a plan (same arguments as
 * pkd_paged_decode_workspace_size): a static string such as
 * "chunked grid, tensor cores".  Host-only, no CUDA call.  Returns NULL for
 * an invalid request (the reason is in pkd_last_error).  The pages have no
 * counterpart of this call; it makes the library's choice of kernel visible
 * to callers and benchmarks.
 */
const char* pkd_paged_decode_kernel_name(int batch, int sq, int num_heads, int num_kv_heads, int head_dim,
                                         int page_size, int max_kv_len, pkd_dtype kv_dtype, int window,
                                         int chunk_tokens, unsigned flags);

/*
 * Zero a workspace (asynchronously on `stream`).  Needed once, before its
 * first use: every later call leaves the workspace ready for the next one.
 */
pkd_status pkd_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronise `stream`, read the workspace's status word and clear it.
 * Returns PKD_OK, PKD_EDEVICE_BOUNDS (a seq_lens entry above max_kv_len or
 * below 0, or a block-table entry outside [0, num_pages): the kernel skipped
 * those keys; or what a call's own comment says) or PKD_ETIMEOUT.  The kernels
 * never trap.
 */
pkd_status pkd_workspace_check(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Paged decode: attention of a uniform query block per request over that
 * request's keys in a paged cache [TS FlashInferTSImpl.forward].
 *
 *   q            device, [batch, sq, num_heads, head_dim] contiguous, q_dtype
 *   kv_cache     device, [num_pages, num_kv_heads, page_size, 2*head_dim]
 *                contiguous, kv_dtype.  K = [..., :head_dim], V = [..., head_dim:]
 *                (token stride 2*head_dim [TS _kv_views, "Layout"]); 16-byte aligned.
 *   block_table  device int32 [batch, block_table_stride]: token t of request b
 *                lives in page block_table[b, t / page_size], slot t % page_size.
 *                Columns past a request's last page are never read.
 *   seq_lens     device int32 [batch], each in [0, max_kv_len].
 *   out          device, [batch, sq, num_heads, head_dim], out_dtype (bf16, fp16, fp32)
 *   lse          device fp32 [batch, sq, num_heads] natural-log LSE, or NULL
 *   workspace    device, >= pkd_paged_decode_workspace_size(...) bytes,
 *                zeroed once by pkd_workspace_init; 256-byte aligned.
 * With PKD_FLAG_HOST_IO, q, block_table, seq_lens, out and lse are pinned
 * host memory instead, read and written by the kernels in place.
 *
 * Query head h reads KV head h / (num_heads / num_kv_heads).  Logits are
 * (scale * q_scale * k_scale) * q.k and the output is scaled by v_scale
 * (bmm1 / bmm2 of [TS forward]); for fp8 caches q is already fp8 with
 * scale q_scale (q_dtype must equal kv_dtype).
 *
 * Masks.  Without PKD_FLAG_CAUSAL every query token of the block sees every
 * visible key ("dense", [TS module docstring]).  window > 0 restricts the
 * visible keys to the page-aligned suffix of [TS _restrict_to_window]:
 *   start_page = max(0, floor((L - (window + sq - 1)) / page_size)),
 * keys [start_page * page_size, L), one start for the whole block.  With
 * PKD_FLAG_CAUSAL query token i (position L - sq + i) sees keys up to its
 * position and, when window > 0, from position - (window - 1) on
 * ([TS _get_plan] mask_type "causal", window_left = window - 1).
 * A query row with no visible key gets out = 0 and lse = -inf.
 *
 * Split-KV [FA num_splits]: the keys of a (request, kv head) may be shared
 * between several workers whose partial results are merged by LSE inside
 * the same launch.  By default a chunked grid runs one CTA per chunk of
 * chunk_tokens keys (0: chosen by the library: about 2048 CTAs, chunks of at
 * most 4096 keys -- 32 chunks for 64 (request, kv head) units of 131,072
 * keys).  16-bit query blocks of M = sq * num_heads / num_kv_heads = 17-32
 * rows with head_dim 128 and batch <= 512 (dense or causal) run instead on a
 * persistent kernel with one CTA per SM on the tcgen05 tensor cores: chunks
 * of at most chunk_tokens keys (0: a quarter of the longest visible range in
 * whole 128-key tiles, between 1024 and 2048 keys; 2048 at most), equal
 * within a request; with more chunks than SMs every CTA takes an equal
 * share of all 128-key tiles (consecutive chunks of a (request, kv head)
 * accumulate together), and only units cut by a share boundary leave
 * partial results, merged by LSE by the CTA that completes the unit's last
 * piece -- one launch.  Other 16-bit blocks of 17-32 rows run the
 * chunked grid with two warps sharing each chunk's stages, 16 rows each
 * (as few chunks of at most 4096 keys as possible).  fp8
 * caches with M > 16 run, for batch <= 1024, on a persistent grid that gives
 * every warp an equal slice of all requests' keys laid end to end.  PKD_FLAG_GRID, PKD_FLAG_FLAT and PKD_FLAG_BALANCED
 * (a persistent grid with an equal slice per CTA) force a kernel;
 * pkd_paged_decode_kernel_name says which one a call launches.
 *
 * Limits: head_dim 64 or 128; page_size a multiple of 16; num_heads a
 * multiple of num_kv_heads; M <= 32 on tensor cores, <= 8 on CUDA cores
 * (PKD_FLAG_FMA); fp8 caches need head_dim 128, and M > 16 with fp8 needs the
 * per-warp persistent grid.  Anything else: PKD_EUNSUPPORTED.  After a
 * PKD_ETIMEOUT, zero the workspace again before reusing it.
 */
pkd_status pkd_paged_decode(const void* q, pkd_dtype q_dtype,
                            const void* kv_cache, pkd_dtype kv_dtype, int64_t num_pages,
                            const int32_t* block_table, int64_t block_table_stride,
                            const int32_t* seq_lens,
                            int batch, int sq, int num_heads, int num_kv_heads, int head_dim,
                            int page_size, int max_kv_len,
                            float scale, float q_scale, float k_scale, float v_scale, int window,
                            void* out, pkd_dtype out_dtype, float* lse,
                            void* workspace, size_t workspace_bytes, int chunk_tokens,
                            unsigned flags, void* stream);

/*
 * pkd_paged_decode without a caller workspace.  The pages have no counterpart
 * of this call: it exists for callers that cannot allocate device memory at
 * the point where they run decode -- plug-ins whose host runtime owns all
 * device memory and hands none out, serving loops that must not allocate once
 * their memory budget is fixed, or C callers with no device allocator of
 * their own.
 *
 * It takes the same arguments as pkd_paged_decode minus the workspace and
 * uses instead a scratch array compiled into the library: 32 MiB of device
 * memory that every GPU loading the library holds until the process exits.
 * A plan whose workspace (pkd_paged_decode_workspace_size) exceeds 32 MiB is
 * rejected with PKD_EUNSUPPORTED.  fp8 caches with more than 16 query rows
 * per kv head always are: their persistent per-warp kernel keeps two partial
 * slots per worker warp whatever the batch (64 MiB at 32 rows).  The call
 * allocates nothing; it clears the part of the scratch it uses
 * (cudaMemsetAsync on `stream`) and launches the decode kernel.  The first
 * call on each device looks up the scratch address on that device (make it
 * before any stream capture); the address is kept for the process, so the
 * call must not be used across a cudaDeviceReset.  All calls share the one
 * scratch array: calls that may overlap on the GPU (different streams, or
 * different host threads on one device) race and must be serialised by the
 * caller.  The device-side status word (out-of-range lengths or pages, a
 * wait that timed out) is cleared by the next call: read it with
 * pkd_paged_decode_static_check before then.
 */
pkd_status pkd_paged_decode_static(const void* q, pkd_dtype q_dtype,
                                   const void* kv_cache, pkd_dtype kv_dtype, int64_t num_pages,
                                   const int32_t* block_table, int64_t block_table_stride,
                                   const int32_t* seq_lens,
                                   int batch, int sq, int num_heads, int num_kv_heads, int head_dim,
                                   int page_size, int max_kv_len,
                                   float scale, float q_scale, float k_scale, float v_scale, int window,
                                   void* out, pkd_dtype out_dtype, float* lse,
                                   int chunk_tokens, unsigned flags, void* stream);

/*
 * The device-side status word of the last pkd_paged_decode_static call on
 * the current device, like pkd_workspace_check on a caller workspace: waits
 * for `stream`, returns PKD_OK, PKD_EDEVICE_BOUNDS (a seq_lens entry outside
 * [0, max_kv_len] or a block-table entry outside [0, num_pages): those keys
 * were skipped) or PKD_ETIMEOUT (a kernel gave up waiting on its own copies),
 * and clears the word.  No counterpart in the pages (see
 * pkd_paged_decode_static).  Allocates nothing.
 */
pkd_status pkd_paged_decode_static_check(void* stream);

/*
 * KV-cache write [TS FlashInferTSImpl.do_kv_cache_update, reshape_and_cache_flash]:
 * the key and value rows of num_tokens new tokens go to their slots.
 *
 *   key, value    device [num_tokens, num_kv_heads, head_dim], in_dtype (bf16 or
 *                 fp16); rows of one token contiguous, key_stride / value_stride
 *                 elements between tokens (multiples of 8); 16-byte aligned
 *   slot_mapping  device int64 [num_tokens]: slot s is page s / page_size,
 *                 offset s % page_size; s < 0 (padding) and slots past the
 *                 cache write nothing
 *   kv_cache      device [num_pages, num_kv_heads, page_size, 2*head_dim]
 *                 kv_dtype: key into [..., :head_dim], value into [..., head_dim:]
 *
 * kv_dtype == in_dtype stores the input bits.  PKD_FP8_E4M3 stores
 * e4m3(x / k_scale) for keys and e4m3(x / v_scale) for values: the quotient is
 * an IEEE fp32 division, rounded to nearest even and saturated to +-448.
 */
pkd_status pkd_cache_write(const void* key, const void* value, pkd_dtype in_dtype, int64_t key_stride,
                           int64_t value_stride, const int64_t* slot_mapping, int64_t num_tokens,
                           int num_kv_heads, int head_dim, int page_size, int64_t num_pages,
                           void* kv_cache, pkd_dtype kv_dtype, float k_scale, float v_scale, void* stream);

/*
 * Rotary step of a layer in one launch: queries rotated, keys rotated and
 * appended to the paged cache with their values (pkd_cache_write with the
 * position rotation on the way).
 *
 *   q             device [num_tokens, num_heads, head_dim], in_dtype (bf16 or fp16),
 *                 q_stride elements between tokens; NULL with num_heads == 0
 *   key, value    device [num_tokens, num_kv_heads, head_dim], in_dtype
 *                 (strides: multiples of 8 elements; all pointers 16-byte aligned)
 *   positions     device int64 [num_tokens]
 *   cos_sin       device fp32 [max_position, rotary_dim], 16-byte aligned: row p
 *                 holds rotary_dim/2 cosines, then rotary_dim/2 sines of position p
 *   slot_mapping  device int64 [num_tokens], as for pkd_cache_write; slots >= 0
 *                 must be distinct (two tokens in one slot race)
 *   kv_cache      as for pkd_cache_write
 *   q_out         device [num_tokens, num_heads, head_dim], q_out_dtype, q_out_stride
 *                 elements between tokens: in_dtype, or PKD_FP8_E4M3 for
 *                 e4m3(rot(q) / q_scale), the pre-quantised q of an fp8 decode.
 *                 May be q itself (same dtype and stride); no other overlap.
 *
 * Pair j of a head is (x[j], x[j + rotary_dim/2]), or (x[2j], x[2j+1]) when
 * interleaved is not 0; it becomes (x1 c - x2 s, x2 c + x1 s).  Dims from
 * rotary_dim on are copied.  Computed in fp32, rounded once to the type that
 * is stored; values are stored as pkd_cache_write stores them.  A token whose
 * position lies outside [0, max_position) writes nothing; a token whose slot
 * is negative (padding) or past the cache writes its q_out row only.
 * Limits: head_dim 64 or 128; rotary_dim a multiple of 16 up to head_dim.
 */
pkd_status pkd_rope_cache_write(const void* q, int64_t q_stride, const void* key, int64_t key_stride,
                                const void* value, int64_t value_stride, pkd_dtype in_dtype,
                                const int64_t* positions, const float* cos_sin, int64_t max_position,
                                int rotary_dim, int interleaved, const int64_t* slot_mapping,
                                int64_t num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                int page_size, int64_t num_pages, void* kv_cache, pkd_dtype kv_dtype,
                                float k_scale, float v_scale, void* q_out, int64_t q_out_stride,
                                pkd_dtype q_out_dtype, float q_scale, void* stream);

/*
 * Score modifications and masks of pkd_paged_attention; zero-initialised: none.
 *   softcap       c > 0 (1e-20 to 1e20): the scaled score s becomes c * tanh(s / c)
 *   alibi_slopes  device fp32 [num_heads]: slope * |position - key| is then
 *                 subtracted (a distance bias), or NULL
 *   window        w > 0: a token at position p sees keys from p - (w - 1) on
 *   prefix_lens   device int32 [batch]: with PKD_FLAG_CAUSAL, keys below the
 *                 request's prefix_lens entry are visible to all its tokens (a
 *                 prefix mask; the window still applies), or NULL
 *   doc_start     device int32 [total_tokens]: first key that a query token
 *                 sees (a document mask for packed documents), or NULL
 */
typedef struct {
    float softcap;
    const float* alibi_slopes;
    int window;
    const int32_t* prefix_lens;
    const int32_t* doc_start;
} pkd_score_options;

/* Bytes at the start of a workspace of pkd_paged_attention or pkd_prefix_decode
 * that must be zero before its first use (the rest is written before it is read). */
#define PKD_ATTENTION_WORKSPACE_HEAD (256 + 4 * 65536)

/*
 * Workspace bytes of pkd_paged_attention, and the kernel it launches.  Host
 * only; the plan is fixed by these arguments (of the options: the window, and
 * whether prefix_lens is given).
 * 0 / NULL for an invalid request (the reason is in pkd_last_error).
 */
size_t pkd_paged_attention_workspace_size(int batch, int64_t total_tokens, int max_query_len, int num_heads,
                                          int num_kv_heads, int head_dim, int page_size, int max_kv_len,
                                          pkd_dtype kv_dtype, const pkd_score_options* options);
const char* pkd_paged_attention_kernel_name(int batch, int64_t total_tokens, int max_query_len, int num_heads,
                                            int num_kv_heads, int head_dim, int page_size, int max_kv_len,
                                            pkd_dtype kv_dtype, const pkd_score_options* options);

/*
 * Attention of ragged query tokens over a paged cache: whole prompts, chunks
 * of prompts, and steps of single tokens, mixed in one call, with capped
 * scores, a distance bias, and window, prefix and document masks.
 *
 *   q            device [total_tokens, num_heads, head_dim], q_dtype == kv_dtype,
 *                q_stride elements between tokens (a multiple of 16 bytes)
 *   kv_cache, block_table, seq_lens  as for pkd_paged_decode; seq_lens[b] = L counts
 *                the keys of request b including those of its query tokens
 *                (already in the cache).  block_table may be NULL with max_kv_len 0
 *   query_start  device int32 [batch + 1]: request b's query tokens are rows
 *                [query_start[b], query_start[b + 1]) of q, at most max_query_len;
 *                rows of q outside every request are neither read into a result
 *                nor written in out and lse
 *   out          device [total_tokens, num_heads, head_dim] contiguous, out_dtype;
 *                no part of it may lie in q
 *   lse          device fp32 [total_tokens, num_heads] natural-log LSE, or NULL
 *   workspace    at least pkd_paged_attention_workspace_size bytes, 256-byte
 *                aligned, its first PKD_ATTENTION_WORKSPACE_HEAD bytes zeroed once
 *                (pkd_workspace_init); every call leaves it ready for the next of
 *                this function or pkd_prefix_decode, whatever its plan.  Calls that
 *                may overlap (streams, graphs) need one each.
 *                After PKD_ETIMEOUT zero those bytes again.
 *                pkd_workspace_check reads its status word (PKD_EDEVICE_BOUNDS also
 *                for a query_start that falls, leaves [0, total_tokens] or holds
 *                more than max_query_len tokens: clamped; rows of requests that
 *                then overlap are not all written)
 *   flags        PKD_FLAG_CAUSAL or 0 (and the diagnostic PKD_FLAG_TEST_TIMEOUT)
 *
 * Token i of request b (n tokens) has position p = L - n + i.  It sees keys
 * [0, L), with PKD_FLAG_CAUSAL those up to p (and its prefix_lens), less what
 * the window and doc_start exclude.  A token that sees no key gets out = 0 and
 * lse = -inf.  Keys and values before the first and behind the last key that a
 * request's tokens see do not enter its results, whatever they hold; the values
 * between must be finite also for the tokens that do not see them (with weight 0).
 * Sums run in fp32: the keys that a token sees times the largest value among
 * them must stay below its range.
 * Limits: head_dim 64 or 128; page_size a multiple of 16; num_heads/num_kv_heads
 * <= 128; batch <= 2048, batch * num_kv_heads <= 65536; max_kv_len <= 2^29;
 * scale * q_scale * k_scale > 0; fp8 caches need head_dim 128.
 */
pkd_status pkd_paged_attention(const void* q, pkd_dtype q_dtype, int64_t q_stride, const void* kv_cache,
                               pkd_dtype kv_dtype, int64_t num_pages, const int32_t* block_table,
                               int64_t block_table_stride, const int32_t* seq_lens, const int32_t* query_start,
                               int batch, int64_t total_tokens, int max_query_len, int num_heads, int num_kv_heads,
                               int head_dim, int page_size, int max_kv_len, float scale, float q_scale,
                               float k_scale, float v_scale, const pkd_score_options* options, void* out,
                               pkd_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                               unsigned flags, void* stream);

/*
 * Attention over whole prompts, packed one behind the other, from their own
 * projections: nothing is read from a paged cache.
 *
 *   q            device [total_tokens, num_heads, head_dim], dtype (bf16 or fp16)
 *   k, v         device [total_keys, num_kv_heads, head_dim], dtype; q_stride, k_stride
 *                and v_stride elements between tokens (multiples of 8), so that all three
 *                may be parts of one fused projection; 16-byte aligned
 *   query_start, key_start  device int32 [batch + 1]: prompt b's tokens are rows
 *                [query_start[b], query_start[b + 1]) of q, at most max_query_len, its
 *                keys rows [key_start[b], key_start[b + 1]) of k and v, at most
 *                max_kv_len.  key_start NULL: query_start (total_keys == total_tokens)
 *   softcap, window  as in pkd_score_options (0: none)
 *   out, lse     as for pkd_paged_attention; no part of out may lie in q, k or v
 *   workspace, flags  as for pkd_paged_attention (status: starts that fall, leave the
 *                tensors or exceed the bounds are clamped)
 *
 * Token i of n has position L - n + i among its prompt's L keys: with PKD_FLAG_CAUSAL it
 * sees keys up to that (fewer tokens than keys are the prompt's last ones).  Rows of no
 * prompt, tokens that see no key, and which values must be finite: as for
 * pkd_paged_attention; other prompts' keys and values do not enter a prompt's results.
 * Limits as there; total_keys <= 2^29.
 */
size_t pkd_packed_attention_workspace_size(int batch, int64_t total_tokens, int max_query_len, int num_heads,
                                           int num_kv_heads, int head_dim, int max_kv_len, pkd_dtype dtype, int window);
pkd_status pkd_packed_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, pkd_dtype dtype, const int32_t* query_start,
                                const int32_t* key_start, int batch, int64_t total_tokens, int64_t total_keys,
                                int max_query_len, int max_kv_len, int num_heads, int num_kv_heads, int head_dim,
                                float scale, float softcap, int window, void* out, pkd_dtype out_dtype, float* lse,
                                void* workspace, size_t workspace_bytes, unsigned flags, void* stream);

/*
 * Decode of a batch whose requests share long prefixes, each prefix computed
 * once for all its requests.
 *
 *   q             device [batch, sq, num_heads, head_dim], q_dtype == kv_dtype
 *   prefix_table  device int32 [groups, prefix_table_stride], prefix_lens device
 *                 int32 [groups]: the pages and length of each shared prefix, in
 *                 the same kv_cache
 *   group_start   device int32 [groups + 1], rising: requests [group_start[g],
 *                 group_start[g + 1]) follow prefix g; others follow none.  NULL
 *                 with one group: every request follows it
 *   block_table, seq_lens  the requests' own keys, after the prefix (seq_lens[b]
 *                 keys; the first page of a request's row starts behind the prefix)
 *   out, lse      as for pkd_paged_decode, over the prefix's and the own keys; out
 *                 not in q
 *   softcap       as in pkd_score_options (0: none)
 *   flags         PKD_FLAG_CAUSAL: token i sees its request's own keys up to
 *                 position seq_lens[b] - sq + i; the prefix is seen whole
 *                 (and the diagnostic PKD_FLAG_TEST_TIMEOUT)
 *
 * The workspace is as for pkd_paged_attention.  max_prefix_len and max_kv_len
 * bound prefix_lens and seq_lens; a table whose bound is 0 may be NULL.  Limits as for
 * pkd_paged_attention, groups <= 2048.
 */
size_t pkd_prefix_decode_workspace_size(int batch, int sq, int num_heads, int num_kv_heads, int head_dim,
                                        int page_size, int groups, int max_prefix_len, int max_kv_len,
                                        pkd_dtype kv_dtype);
pkd_status pkd_prefix_decode(const void* q, pkd_dtype q_dtype, const void* kv_cache, pkd_dtype kv_dtype,
                             int64_t num_pages, const int32_t* prefix_table, int64_t prefix_table_stride,
                             const int32_t* prefix_lens, const int32_t* group_start, int groups, int max_prefix_len,
                             const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens,
                             int batch, int sq, int num_heads, int num_kv_heads, int head_dim, int page_size,
                             int max_kv_len, float scale, float q_scale, float k_scale, float v_scale,
                             float softcap, void* out, pkd_dtype out_dtype, float* lse, void* workspace,
                             size_t workspace_bytes, unsigned flags, void* stream);

/*
 * Attention weight that each key of a paged cache received: what keeps a cache of
 * bounded size (pkd_evict_select, pkd_cache_compact) knows its keys by.
 *
 *   weights[b, h, t] = decay * prior[b, h, t]
 *                    + sum over tokens i of request b and query heads g of kv head h
 *                      of exp(s(i, g, t) - lse(i, g))
 * with the scaled (and capped) scores and the masks of pkd_paged_attention, whose LSE
 * over the same keys makes the exponential a probability.
 *
 *   q, kv_cache, block_table, seq_lens, query_start, max_query_len, softcap, window,
 *                flags  as for pkd_paged_attention (V is not read; of the table the columns
 *                of max_kv_len keys are read, and those behind a length not used)
 *   last_queries w > 0: only the last w tokens of each request weigh its keys
 *   lse          device fp32 [total_tokens, num_heads]; a token of lse -inf weighs nothing
 *   prior        device fp32 [batch, num_kv_heads, >= max_kv_len], or NULL: 0.  Rows
 *                of keys contiguous, strides in elements (up to 2^40).  Not read for keys of the
 *                call's own tokens (the last query_start[b + 1] - query_start[b] of
 *                seq_lens[b]), nor behind seq_lens[b]: they start at 0
 *   weights      device fp32, laid out like prior with strides of its own; may be prior
 *                itself, no other overlap.  Entries behind seq_lens[b] are left as they
 *                were
 *   workspace    as for pkd_paged_attention (its status word: lengths, starts and pages
 *                out of range; keys on such a page receive nothing)
 *                (of PKD_FLAG_TEST_TIMEOUT only more than 16 rows, last_queries or
 *                max_query_len tokens times num_heads / num_kv_heads, take notice)
 *
 * Sums run in fp32, in an order fixed by the arguments: results repeat bit for bit.  A
 * key that no token sees receives 0 whatever its K holds.  Limits as for
 * pkd_paged_attention.  The workspace size is 0 for an invalid request.
 */
size_t pkd_key_weights_workspace_size(int batch, int64_t total_tokens, int max_query_len, int last_queries,
                                      int num_heads, int num_kv_heads, int head_dim, int page_size, int max_kv_len,
                                      pkd_dtype kv_dtype);
pkd_status pkd_key_weights(const void* q, pkd_dtype q_dtype, int64_t q_stride, const void* kv_cache,
                           pkd_dtype kv_dtype, int64_t num_pages, const int32_t* block_table,
                           int64_t block_table_stride, const int32_t* seq_lens, const int32_t* query_start, int batch,
                           int64_t total_tokens, int max_query_len, int last_queries, int num_heads,
                           int num_kv_heads, int head_dim, int page_size, int max_kv_len, float scale, float q_scale,
                           float k_scale, float softcap, int window, const float* lse, const float* prior,
                           int64_t prior_batch_stride, int64_t prior_head_stride, float decay, float* weights,
                           int64_t weights_batch_stride, int64_t weights_head_stride, void* workspace,
                           size_t workspace_bytes, unsigned flags, void* stream);

/*
 * The keys of each request and kv head that stay in a cache of at most `budget` keys.
 *
 *   weights      device fp32 [batch, num_kv_heads, keys], rows contiguous, strides in
 *                elements (up to 2^40).  NaN counts as -inf
 *   seq_lens     device int32 [batch], clamped to [0, keys]
 *   positions    device int32 [batch, num_kv_heads, keys]: where in its request each key
 *                stood, once earlier compactions have put them out of order, with
 *                context_lens, device int32 [batch]: the tokens that the request has
 *                seen.  NULL both: key t stands at t of seq_lens[b]
 *   kept         device int32 [batch, num_kv_heads, budget]: the indexes of the
 *                n = min(seq_lens[b], budget) keys that stay, rising; -1 behind them
 *   kept_lens    device int32 [batch]: n.  Neither kept nor kept_lens may overlap an
 *                input (kept_lens may not be seq_lens) or the other
 *
 * Kept are the keys at the first `sinks` and the last `recent` positions, then those of
 * the largest weight, of equal ones the lowest index.  pool (odd, up to 255): a key's
 * weight is the largest of the pool keys around it that are neither sinks nor recent.
 * Limits: sinks + recent <= budget; pool is 1 with positions; keys <= 2^29.
 */
pkd_status pkd_evict_select(const float* weights, int64_t weights_batch_stride, int64_t weights_head_stride,
                            int64_t keys, const int32_t* seq_lens, int batch, int num_kv_heads, int budget, int sinks,
                            int recent, int pool, const int32_t* positions, int64_t positions_batch_stride,
                            int64_t positions_head_stride, const int32_t* context_lens, int32_t* kept,
                            int32_t* kept_lens, void* stream);
/* The same with a workspace (256-byte aligned, 256 bytes or more, zeroed once; any other
 * call's on the stream will do), whose status word reports seq_lens outside [0, keys]. */
pkd_status pkd_evict_select_checked(const float* weights, int64_t weights_batch_stride, int64_t weights_head_stride,
                                    int64_t keys, const int32_t* seq_lens, int batch, int num_kv_heads, int budget,
                                    int sinks, int recent, int pool, const int32_t* positions,
                                    int64_t positions_batch_stride, int64_t positions_head_stride,
                                    const int32_t* context_lens, int32_t* kept, int32_t* kept_lens, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * Compaction of a paged cache, in place: of the n = kept_lens[b] rows that stay of a
 * request and kv head, those at index n or behind move into the free slots below n (the
 * m-th such row into the m-th free slot), so that the request's keys are [0, n).  No
 * other row moves: the keys' order changes, which attention without a window does not
 * see (their rotary positions are in them).
 *
 *   kept, kept_lens  as pkd_evict_select leaves them: rising indexes per (request, kv head)
 *   block_table  device int32 [batch, block_table_stride], table_columns of them in use
 *   weights, positions  device [batch, num_kv_heads, weights_keys / positions_keys] (fp32 /
 *                int32; rows contiguous, strides in elements up to 2^40; a key or more)
 *                move along, or NULL
 *
 * A row moves with its weight and position or not at all: not where its index lies behind
 * the table, weights or positions, or its source or target page outside the pool.  Its
 * slot then holds what it held, an evicted key, and kept_lens still counts it: give the
 * arrays that the choice was made from, and look at the status of
 * pkd_cache_compact_checked.
 * The pages of the slots below n must be one request's own (pages that requests share
 * behind them are only read).  K and V bits are copied.  Limits: head_dim 64 or 128.
 */
pkd_status pkd_cache_compact(void* kv_cache, pkd_dtype kv_dtype, int64_t num_pages, const int32_t* block_table,
                             int64_t block_table_stride, int table_columns, const int32_t* kept,
                             const int32_t* kept_lens, int batch, int num_kv_heads, int head_dim, int page_size,
                             int budget, float* weights, int64_t weights_batch_stride, int64_t weights_head_stride,
                             int64_t weights_keys, int32_t* positions, int64_t positions_batch_stride,
                             int64_t positions_head_stride, int64_t positions_keys, void* stream);
/* The same with a workspace (as for pkd_evict_select_checked), whose status word reports
 * rows that did not move, and kept_lens outside [0, budget]. */
pkd_status pkd_cache_compact_checked(void* kv_cache, pkd_dtype kv_dtype, int64_t num_pages, const int32_t* block_table,
                                     int64_t block_table_stride, int table_columns, const int32_t* kept,
                                     const int32_t* kept_lens, int batch, int num_kv_heads, int head_dim, int page_size,
                                     int budget, float* weights, int64_t weights_batch_stride, int64_t weights_head_stride,
                                     int64_t weights_keys, int32_t* positions, int64_t positions_batch_stride,
                                     int64_t positions_head_stride, int64_t positions_keys, void* workspace,
                                     size_t workspace_bytes, void* stream);

/*
 * DASH segmented attention with its combine [DASH flash_dash_attention].
 *
 *   q        device [n, num_heads, head_dim], dtype (bf16 or fp16)
 *   k, v     device [n * (topk*bs + local), num_kv_heads, head_dim], dtype, contiguous
 *   used     device int32 [n * (topk + 1)]: valid prefix length of each segment;
 *            query i's segment g < topk starts at row i*(topk*bs+local) + g*bs
 *            (capacity bs), its local segment at i*(topk*bs+local) + topk*bs
 *            (capacity local).  Values are clamped to [0, capacity].
 *   bias     device fp32 [n, topk] prior of each gathered segment (the local
 *            segment's prior is 0); may be NULL when topk == 0.
 *   out      device [n, num_heads, head_dim], dtype
 *   seg_out  device fp32 [n, topk+1, num_heads, head_dim] per-segment outputs, or NULL
 *   seg_lse  device fp32 [n, topk+1, num_heads] per-segment natural-log LSE, or NULL
 *
 * Each (query, segment, head) is softmax attention over the segment's used
 * rows with scale head_dim^-0.5, giving (o_g, lse_g); an empty segment gives
 * (0, -inf).  out = sum_g w_g o_g with w = softmax over live segments
 * (used > 0) of lse_g + prior_g; a query with no live segment gets 0.
 * Limits: head_dim 64 or 128, bs and local multiples of 8, num_heads a
 * multiple of num_kv_heads with num_heads / num_kv_heads <= 16.
 */
pkd_status pkd_segmented_attention(const void* q, const void* k, const void* v, pkd_dtype dtype,
                                   const int32_t* used, const float* bias,
                                   int n, int num_heads, int num_kv_heads, int head_dim,
                                   int topk, int bs, int local,
                                   void* out, float* seg_out, float* seg_lse, void* stream);

/*
 * DASH segmented attention read straight from the paged cache: the segments
 * are key ranges of the query's own request, gathered through the block
 * table instead of being copied into contiguous k/v first (the copy that
 * feeds [DASH flash_dash_attention]).
 *
 *   q            device [n, num_heads, head_dim], dtype (bf16 or fp16)
 *   kv_cache     device [num_pages, num_kv_heads, page_size, 2*head_dim], dtype
 *   block_table  device int32 [n, block_table_stride]: row i is query i's request
 *   seg_start    device int32 [n, topk+1]: position of the first key of each
 *                segment in that request ([topk gathered, local] order)
 *   used         device int32 [n, topk+1]: keys in each segment, clamped to
 *                [0, bs] (gathered) or [0, local] (local segment) and to max_kv_len
 *   bias, out, seg_out, seg_lse as for pkd_segmented_attention
 *
 * Segment g of query i holds keys [seg_start, seg_start + used) of request i;
 * everything else (scale, per-segment (o, lse), the combine) is as in
 * pkd_segmented_attention.  page_size must be a multiple of 16; pages outside
 * [0, num_pages) are skipped.
 */
pkd_status pkd_segmented_attention_paged(const void* q, pkd_dtype dtype, const void* kv_cache,
                                         int64_t num_pages, const int32_t* block_table,
                                         int64_t block_table_stride, const int32_t* seg_start,
                                         const int32_t* used, const float* bias, int n, int num_heads,
                                         int num_kv_heads, int head_dim, int page_size, int topk, int bs,
                                         int local, int max_kv_len, void* out, float* seg_out,
                                         float* seg_lse, void* stream);

/*
 * LSE merge of partial attention results: the Split-KV merge [FA] and, with a
 * prior and a live mask, the segment combine [DASH flash_dash_attention].
 *
 *   part_out  device fp32 [n, parts, heads, head_dim]
 *   part_lse  device fp32 [n, parts, heads] natural-log LSE of each part
 *   prior     device fp32 [n, parts] added to each part's LSE, or NULL
 *   live      device int32 [n, parts]; part p of row n is dead when <= 0, or NULL
 *   out       device [n, heads, head_dim], out_dtype (bf16, fp16, fp32)
 *   lse_out   device fp32 [n, heads] = ln sum_{live p} exp(lse_p + prior_p), or NULL
 *
 * out = sum over live parts of exp(lse_p + prior_p - lse_out) * part_out_p;
 * a dead part (or one with lse -inf) is never read; a row with no live part
 * gets out = 0 and lse_out = -inf.  Limits: head_dim <= 256, parts <= 1024.
 */
pkd_status pkd_lse_merge(const float* part_out, const float* part_lse, const float* prior,
                         const int32_t* live, int n, int parts, int heads, int head_dim,
                         void* out, pkd_dtype out_dtype, float* lse_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKD_H_ */
