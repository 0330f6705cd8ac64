// C entry points of the choice of the keys that stay and of the compaction.
#include "evict.cuh"
#include "launch.h"
#include "page_math.h"

namespace {

using pkd::report;

constexpr int kMaxKeys = 1 << 29;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// [B, H] rows of `keys` values: given with sane strides, or not given.
pkd_status check_rows(const void* p, int64_t sb, int64_t sh, int64_t keys, bool written, int B, int H, const char* name) {
    if (!p) return PKD_OK;
    if (!aligned(p, 4)) return report(PKD_EINVAL, "%s must be 4-byte aligned", name);
    // (sums of strides and keys stay far from 2^63)
    if ((B > 1 && sb > kMaxStride) || (H > 1 && sh > kMaxStride))
        return report(PKD_EUNSUPPORTED, "%s strides %lld, %lld: more than 2^40", name, (long long)sb, (long long)sh);
    const bool apart = ((H == 1 || sh >= keys) && (B == 1 || sb >= (H - 1) * sh + keys)) ||
                       ((B == 1 || sb >= keys) && (H == 1 || sh >= (B - 1) * sb + keys));
    if (sb < 0 || sh < 0 || (written && !apart))
        return report(PKD_EINVAL, "%s strides %lld, %lld: negative, or rows overlap", name, (long long)sb, (long long)sh);
    return PKD_OK;
}

// The bytes of 4-byte values [B, H] rows of `keys` (none: not given).
struct Span {
    uintptr_t from, past;
    bool meets(const Span& x) const { return from < x.past && x.from < past; }
};
Span span_of(const void* p, int64_t sb, int64_t sh, int64_t B, int64_t H, int64_t keys) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return {at, p && keys > 0 ? at + 4 * ((B - 1) * sb + (H - 1) * sh + keys) : at};
}

pkd_status check_sizes(int B, int H, int64_t keys, int budget) {
    if (B < 0 || H < 1 || keys < 0 || budget < 1)
        return report(PKD_EINVAL, "invalid shape: batch=%d num_kv_heads=%d keys=%lld budget=%d", B, H, (long long)keys, budget);
    if (B > 65535 || H > 65535) return report(PKD_EUNSUPPORTED, "batch %d or num_kv_heads %d > 65535", B, H);
    if (keys > kMaxKeys || budget > kMaxKeys)
        return report(PKD_EUNSUPPORTED, "%lld keys or a budget of %d: more than 2^29", (long long)keys, budget);
    return PKD_OK;
}

// The status word of a call's workspace; none without one.
pkd_status check_workspace(const void* workspace, size_t bytes) {
    if (workspace && (!aligned(workspace, 256) || bytes < 256))
        return report(PKD_EINVAL, "the workspace must be 256-byte aligned and hold 256 bytes or more");
    return PKD_OK;
}

pkd_status done(cudaError_t e, const char* what) {
    return e == cudaSuccess ? PKD_OK : report(PKD_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

}  // namespace

extern "C" {

pkd_status pkd_evict_select_checked(const float* weights, int64_t weights_batch_stride, int64_t weights_head_stride,
                                    int64_t keys, const int32_t* seq_lens, int batch, int num_kv_heads, int budget,
                                    int sinks, int recent, int pool, const int32_t* positions,
                                    int64_t positions_batch_stride, int64_t positions_head_stride,
                                    const int32_t* context_lens, int32_t* kept, int32_t* kept_lens, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    pkd_status st = check_sizes(batch, num_kv_heads, keys, budget);
    if (st == PKD_OK) st = check_workspace(workspace, workspace_bytes);
    if (st != PKD_OK) return st;
    if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
        return report(PKD_EINVAL, "sinks (%d) and recent (%d) must be >= 0 and together within the budget (%d)", sinks, recent, budget);
    if (pool < 1 || pool % 2 == 0 || pool > 255) return report(PKD_EINVAL, "pool must be odd, 1 to 255 (got %d)", pool);
    if (!positions != !context_lens) return report(PKD_EINVAL, "positions and context_lens come together");
    if (positions && pool > 1) return report(PKD_EUNSUPPORTED, "pool over keys out of order (positions) is not supported");
    if (batch == 0) return PKD_OK;
    if ((!weights && keys > 0) || !seq_lens || !kept || !kept_lens) return report(PKD_EINVAL, "null pointer argument");
    if (!aligned(seq_lens, 4) || !aligned(context_lens, 4) || !aligned(kept, 4) || !aligned(kept_lens, 4))
        return report(PKD_EINVAL, "misaligned pointer");
    st = check_rows(weights, weights_batch_stride, weights_head_stride, keys, false, batch, num_kv_heads, "weights");
    if (st != PKD_OK) return st;
    st = check_rows(positions, positions_batch_stride, positions_head_stride, keys, false, batch, num_kv_heads, "positions");
    if (st != PKD_OK) return st;
    // results are written while other CTAs still read: a length that became kept_lens, say
    const int64_t rows = (int64_t)batch * num_kv_heads;
    const Span in[4] = {span_of(weights, weights_batch_stride, weights_head_stride, batch, num_kv_heads, keys),
                        span_of(positions, positions_batch_stride, positions_head_stride, batch, num_kv_heads, keys),
                        span_of(seq_lens, 1, 0, batch, 1, 1), span_of(context_lens, 1, 0, batch, 1, 1)};
    const Span to = span_of(kept, budget, 0, rows, 1, budget), lens = span_of(kept_lens, 1, 0, batch, 1, 1);
    for (const Span& x : in)
        if (x.meets(to) || x.meets(lens))
            return report(PKD_EINVAL, "kept or kept_lens overlaps weights, positions, seq_lens or context_lens");
    if (to.meets(lens)) return report(PKD_EINVAL, "kept overlaps kept_lens");
    pkd::SelectParams p = {};
    p.weights = weights;
    p.positions = positions;
    p.seq_lens = seq_lens;
    p.context_lens = context_lens;
    p.kept = kept;
    p.kept_lens = kept_lens;
    p.status = static_cast<int32_t*>(workspace);
    p.weights_b = weights_batch_stride;
    p.weights_h = weights_head_stride;
    p.positions_b = positions_batch_stride;
    p.positions_h = positions_head_stride;
    p.B = batch;
    p.H = num_kv_heads;
    p.keys = (int)keys;
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    p.pool = pool;
    return done(pkd::launch_evict_select(p, (cudaStream_t)stream), "pkd_evict_select launch");
}

pkd_status pkd_evict_select(const float* weights, int64_t weights_batch_stride, int64_t weights_head_stride, int64_t keys,
                            const int32_t* seq_lens, int batch, int num_kv_heads, int budget, int sinks, int recent,
                            int pool, const int32_t* positions, int64_t positions_batch_stride,
                            int64_t positions_head_stride, const int32_t* context_lens, int32_t* kept,
                            int32_t* kept_lens, void* stream) {
    return pkd_evict_select_checked(weights, weights_batch_stride, weights_head_stride, keys, seq_lens, batch, num_kv_heads,
                                    budget, sinks, recent, pool, positions, positions_batch_stride, positions_head_stride,
                                    context_lens, kept, kept_lens, nullptr, 0, stream);
}

pkd_status pkd_cache_compact_checked(void* kv_cache, pkd_dtype kv_dtype, int64_t num_pages, const int32_t* block_table,
                                     int64_t block_table_stride, int table_columns, const int32_t* kept,
                                     const int32_t* kept_lens, int batch, int num_kv_heads, int head_dim, int page_size,
                                     int budget, float* weights, int64_t weights_batch_stride, int64_t weights_head_stride,
                                     int64_t weights_keys, int32_t* positions, int64_t positions_batch_stride,
                                     int64_t positions_head_stride, int64_t positions_keys, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    pkd_status st = check_sizes(batch, num_kv_heads, 0, budget);
    if (st == PKD_OK) st = check_workspace(workspace, workspace_bytes);
    if (st != PKD_OK) return st;
    if (table_columns < 0 || page_size < 1 || num_pages < 1)
        return report(PKD_EINVAL, "invalid shape: table_columns=%d page_size=%d num_pages=%lld", table_columns, page_size,
                      (long long)num_pages);
    if (head_dim != 64 && head_dim != 128) return report(PKD_EUNSUPPORTED, "head_dim %d not supported (64 or 128)", head_dim);
    if (kv_dtype != PKD_BF16 && kv_dtype != PKD_FP16 && kv_dtype != PKD_FP8_E4M3)
        return report(PKD_EUNSUPPORTED, "kv dtype %d not supported (bf16, fp16, fp8-e4m3)", (int)kv_dtype);
    if (batch == 0) return PKD_OK;
    if (!kv_cache || !kept || !kept_lens || (!block_table && table_columns > 0)) return report(PKD_EINVAL, "null pointer argument");
    if (!aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(kept, 4) || !aligned(kept_lens, 4))
        return report(PKD_EINVAL, "misaligned pointer (kv_cache: 16 B)");
    if (block_table_stride < table_columns)
        return report(PKD_EINVAL, "block_table stride %lld < %d columns", (long long)block_table_stride, table_columns);
    if (num_pages > 0x7fffffffll / ((int64_t)num_kv_heads * page_size))
        return report(PKD_EUNSUPPORTED, "cache too large: num_pages*num_kv_heads*page_size must be < 2^31");
    // a row moves only with all of its values: keys that every given array has
    int64_t keys = (int64_t)table_columns * page_size;
    if (weights && weights_keys < keys) keys = weights_keys;
    if (positions && positions_keys < keys) keys = positions_keys;
    if (keys < 0) return report(PKD_EINVAL, "negative number of keys");
    if ((weights && weights_keys == 0) || (positions && positions_keys == 0))
        return report(PKD_EINVAL, "weights and positions must have keys");  // no row could move with its values
    if (keys > kMaxKeys) keys = kMaxKeys;
    st = check_rows(weights, weights_batch_stride, weights_head_stride, keys, true, batch, num_kv_heads, "weights");
    if (st != PKD_OK) return st;
    st = check_rows(positions, positions_batch_stride, positions_head_stride, keys, true, batch, num_kv_heads, "positions");
    if (st != PKD_OK) return st;
    pkd::CompactParams p = {};
    p.cache = static_cast<uint8_t*>(kv_cache);
    p.block_table = block_table;
    p.kept = kept;
    p.kept_lens = kept_lens;
    p.weights = weights;
    p.positions = positions;
    p.status = static_cast<int32_t*>(workspace);
    p.bt_stride = block_table_stride;
    p.num_pages = num_pages;
    p.weights_b = weights_batch_stride;
    p.weights_h = weights_head_stride;
    p.positions_b = positions_batch_stride;
    p.positions_h = positions_head_stride;
    p.B = batch;
    p.H = num_kv_heads;
    p.P = page_size;
    p.keys = (int)keys;
    p.budget = budget;
    p.row_bytes = 2 * head_dim * (kv_dtype == PKD_FP8_E4M3 ? 1 : 2);
    pkd::page_magic(page_size, p.pmagic, p.pmshift);
    return done(pkd::launch_cache_compact(p, (cudaStream_t)stream), "pkd_cache_compact launch");
}

pkd_status pkd_cache_compact(void* kv_cache, pkd_dtype kv_dtype, int64_t num_pages, const int32_t* block_table,
                             int64_t block_table_stride, int table_columns, const int32_t* kept, const int32_t* kept_lens,
                             int batch, int num_kv_heads, int head_dim, int page_size, int budget, float* weights,
                             int64_t weights_batch_stride, int64_t weights_head_stride, int64_t weights_keys,
                             int32_t* positions, int64_t positions_batch_stride, int64_t positions_head_stride,
                             int64_t positions_keys, void* stream) {
    return pkd_cache_compact_checked(kv_cache, kv_dtype, num_pages, block_table, block_table_stride, table_columns, kept,
                                     kept_lens, batch, num_kv_heads, head_dim, page_size, budget, weights,
                                     weights_batch_stride, weights_head_stride, weights_keys, positions,
                                     positions_batch_stride, positions_head_stride, positions_keys, nullptr, 0, stream);
}

}  // extern "C"
