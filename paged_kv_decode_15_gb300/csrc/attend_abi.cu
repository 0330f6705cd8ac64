// C entry points of ragged paged attention and shared-prefix decode:
// validation, the plan (kernel, Split-KV, workspace), launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attend.cuh"
#include "attend_launch.h"
#include "attend_prompt.cuh"
#include "page_math.h"

namespace {

using pkd::report;

// Workspace: a header (status word; queue words of the two passes), arrival
// counters, partial results.  Header and counters have the same place in every
// plan and are left zero by every call, so one workspace, zeroed once, serves
// any plan that fits in it.
constexpr size_t kHeader = 256;
constexpr size_t kQueueWord[2] = {16, 32};
constexpr int kMaxUnits = 1 << 16;
constexpr size_t kPartials = kHeader + size_t(kMaxUnits) * 4;
static_assert(kPartials == PKD_ATTENTION_WORKSPACE_HEAD, "the zeroed part");
constexpr int kSms = 152;         // the plan is a host function: GB300's SM count
constexpr int kStepCtas = 2048;   // as for the decode grid
constexpr int kStepMaxChunk = 4096;
constexpr int kMaxKeys = 1 << 29; // keys of a request: sums of a key index and a chunk fit 32 bits

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int up(int x, int a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int elt_bytes(pkd_dtype dt) { return dt == PKD_FP8_E4M3 ? 1 : dt == PKD_FP32 ? 4 : 2; }

struct AttendPlan {
    bool step;                // the step grid, else the tcgen05 kernel
    int G, rows, chunk, max_splits;
    long long pairs, units;   // row-tile pairs of a kv head, split units of all kv heads, at most
    int ref_up;               // AttendParams: where a row's reference lies above its maximum
    size_t lse_bytes, out_bytes;  // partial results
    size_t fold_bytes;        // of sums over more than kPtFold key tiles: two row tiles a CTA
    size_t bytes() const { return lse_bytes + out_bytes + fold_bytes; }
};

// Reference of a row's weights in the tcgen05 kernel, for items of at most `keys` keys.
// It moves when the row's maximum outgrows the room above it, and every move sends a
// warp through the slow path (with 2^8 of room, half of the key tiles of scores with a
// spread of 3 had one).
// fp16 weights (fp16 and e4m3 caches) must stay below 2^16, and below 2^-14 they lose
// bits: each is off by 2^-25 at most.  A maximum that starts at 2^up leaves 2^(15 - up)
// of room, and the small weights together are off by keys * 2^-(25 + up) of the sum at
// most: 2^-13 up to 2^26 keys.  (Started at 1, 131072 weights of e^-18 beside one of 1
// were lost, 2^-9 of the sum.)  Up to 8192 keys up = 1.
// bf16 has fp32's range, and so has V: weights above 1 could take O out of it (with a
// room of 2^40 above 1, values above 3e26 did).  A maximum that starts at 2^-20 has that
// room below 1, and loses only weights below 2^-106 of its own.
int plan_reference(long long keys, pkd_dtype kv) {
    if (kv == PKD_BF16) return 20;
    int up = 1;
    while (up < 14 && keys > 1ll << (12 + up)) ++up;
    return -up;
}

pkd_status check_shape(int B, long long T, int Hq, int Hkv, int D, int P, int max_kv_len, pkd_dtype kv) {
    if (B < 0 || T < 0 || Hq < 1 || Hkv < 1 || P < 1 || max_kv_len < 0)
        return report(PKD_EINVAL, "invalid shape: batch=%d tokens=%lld num_heads=%d num_kv_heads=%d page_size=%d "
                      "max_kv_len=%d", B, T, Hq, Hkv, P, max_kv_len);
    if (Hq % Hkv) return report(PKD_EUNSUPPORTED, "num_heads (%d) must be a multiple of num_kv_heads (%d)", Hq, Hkv);
    if (Hq / Hkv > pkd::kPtRows)
        return report(PKD_EUNSUPPORTED, "num_heads/num_kv_heads = %d > %d", Hq / Hkv, pkd::kPtRows);
    if (D != 64 && D != 128) return report(PKD_EUNSUPPORTED, "head_dim %d not supported (64 or 128)", D);
    if (P % 16) return report(PKD_EUNSUPPORTED, "page_size %d must be a multiple of 16", P);
    if (kv != PKD_BF16 && kv != PKD_FP16 && kv != PKD_FP8_E4M3)
        return report(PKD_EUNSUPPORTED, "kv dtype %d not supported (bf16, fp16, fp8-e4m3)", (int)kv);
    if (kv == PKD_FP8_E4M3 && D != 128) return report(PKD_EUNSUPPORTED, "fp8 caches need head_dim 128");
    if (B > pkd::kPtMaxBatch) return report(PKD_EUNSUPPORTED, "batch %d > %d", B, pkd::kPtMaxBatch);
    if (max_kv_len > kMaxKeys) return report(PKD_EUNSUPPORTED, "lengths of up to %d keys are not supported (2^29)", max_kv_len);
    if (Hkv > 65535) return report(PKD_EUNSUPPORTED, "num_kv_heads %d > 65535", Hkv);
    if (T > 0x7fffffffll / Hq) return report(PKD_EUNSUPPORTED, "tokens*num_heads must be < 2^31");
    return PKD_OK;
}

pkd_status check_options(const pkd_score_options& o) {
    if (o.softcap != 0.f && !(o.softcap >= 1e-20f && o.softcap <= 1e20f))
        return report(PKD_EINVAL, "softcap must be 0 (none) or between 1e-20 and 1e20");
    if (!aligned(o.alibi_slopes, 4) || !aligned(o.prefix_lens, 4) || !aligned(o.doc_start, 4))
        return report(PKD_EINVAL, "alibi_slopes, prefix_lens and doc_start must be 4-byte aligned");
    return PKD_OK;
}

// Plan of one pass over `T` query tokens of B requests, at most max_q tokens
// each.  vis: keys that one request's tokens can span.
pkd_status plan_attend(int B, long long T, int max_q, int Hq, int Hkv, int D, int P, long long vis, pkd_dtype kv,
                       bool partials, bool own_step, AttendPlan& pl) {
    pl = AttendPlan{};
    pl.G = Hq / Hkv;
    pl.rows = max_q * pl.G;
    pl.step = own_step;
    const size_t rows = (size_t)T * Hq;
    if (pl.step) {
        // about kStepCtas CTAs, chunks of 256 to 4096 keys (the decode grid's rule)
        const long long units = std::max(1ll, (long long)B * Hkv);
        long long splits = std::max((kStepCtas + units - 1) / units, (vis + kStepMaxChunk - 1) / kStepMaxChunk);
        // a batch that leaves SMs idle at that goes down to 128 (one request of 611
        // keys: 8.9 us, 256 keys 10.0, 512 12.5, 64 9.1)
        const long long least = units * ((vis + 255) / 256) < 2 * kSms ? 128 : 256;
        long long chunk = std::max((vis + splits - 1) / std::max(splits, 1ll), least);
        chunk = (chunk + P - 1) / P * P;
        if (chunk / P > pkd::kMaxCtaPages) chunk = (long long)pkd::kMaxCtaPages * P;
        pl.chunk = (int)chunk;
        pl.max_splits = vis > 0 ? (int)((vis + chunk - 1) / chunk) : 1;
        pl.units = units;
        const size_t parts = (size_t)units * pl.max_splits * pl.rows;
        if (units > kMaxUnits) return report(PKD_EUNSUPPORTED, "batch*num_kv_heads must be <= %d", kMaxUnits);
        pl.lse_bytes = pl.max_splits > 1 ? up256(parts * 4) : 0;
        pl.out_bytes = pl.max_splits > 1 ? up256(parts * D * 4) : 0;
        return PKD_OK;
    }
    // row-tile pairs: at least what all tokens fill, at most one more per request
    const int pair = 2 * (pkd::kPtRows / pl.G);
    const long long least = std::max((T + pair - 1) / pair, 1ll), most = T / pair + B;
    pl.pairs = most;
    pl.units = most * Hkv;
    // the keys are split while the row tiles alone leave SMs idle: about two
    // items per SM, chunks of whole tiles, at least 512 keys (256 for partials,
    // whose join is a launch of its own)
    // (partials: one item per SM for a single prefix, whose items are alike, else three)
    long long splits = least * Hkv >= kSms ? 1 : (2 * kSms + least * Hkv - 1) / (least * Hkv);
    if (partials) {
        splits = B == 1 ? kSms / (least * Hkv) : 3 * kSms / (most * Hkv);
        if (splits < 1) splits = 1;
    }
    const long long floor_chunk = partials ? 256 : 512;
    long long chunk = std::max((vis + splits - 1) / splits, floor_chunk);
    chunk = (chunk + pkd::kPtKeys - 1) / pkd::kPtKeys * pkd::kPtKeys;
    pl.chunk = (int)chunk;
    // + 15: an item's keys start on a 16-key boundary
    pl.max_splits = vis > 0 ? (int)((vis + 15 + pl.chunk - 1) / pl.chunk) : 1;
    // unsplit: a chunk beyond every length (first key + chunk stays below 2^31)
    if (least * Hkv >= kSms && !partials) pl.max_splits = 1, pl.chunk = kMaxKeys;
    pl.ref_up = plan_reference(std::min<long long>(vis, pl.chunk), kv);
    if (pl.units * pl.max_splits >= 1ll << 31) return report(PKD_EUNSUPPORTED, "too many work items");
    const size_t parts = (partials || pl.max_splits > 1) ? rows * pl.max_splits : 0;
    if (pl.max_splits > 1 && !partials && pl.units > kMaxUnits)
        return report(PKD_EUNSUPPORTED, "too many row tiles for split keys");
    pl.lse_bytes = up256(parts * 4);
    pl.out_bytes = up256(parts * D * 4);
    if (std::min<long long>(vis + 15, pl.chunk) > (long long)pkd::kPtFold * pkd::kPtKeys)
        pl.fold_bytes = (size_t)kSms * 2 * pkd::kPtRows * (D + 4) * 4;
    return PKD_OK;
}

pkd_status plan_paged_attention(int B, long long T, int max_q, int Hq, int Hkv, int D, int P, int max_kv_len,
                                pkd_dtype kv, const pkd_score_options& o, AttendPlan& pl) {
    pkd_status st = check_shape(B, T, Hq, Hkv, D, P, max_kv_len, kv);
    if (st != PKD_OK) return st;
    // (the most that a batch of no requests brings is 0)
    if (max_q < 0 || (max_q == 0 && T > 0)) return report(PKD_EINVAL, "max_query_len must be >= 1 (got %d)", max_q);
    max_q = (int)std::max(1ll, std::min<long long>(max_q, T));
    long long vis = max_kv_len;
    // a window bounds the span of a request's keys, unless prefix keys are seen past the position
    if (o.window > 0 && !o.prefix_lens) vis = std::min(vis, (long long)o.window + max_q - 1 + 15);
    const bool step = (long long)max_q * (Hq / Hkv) <= 16;
    return plan_attend(B, T, max_q, Hq, Hkv, D, P, vis, kv, false, step, pl);
}

struct PrefixPlan {
    AttendPlan pre, own;
    size_t off_own, off_own_lse, off_own_out, bytes;  // own keys: partials, then results
};

pkd_status plan_prefix(int B, int sq, int Hq, int Hkv, int D, int P, int groups, int max_prefix_len, int max_kv_len,
                       pkd_dtype kv, PrefixPlan& pl) {
    if (max_prefix_len > kMaxKeys)
        return report(PKD_EUNSUPPORTED, "prefixes of up to %d keys are not supported (2^29)", max_prefix_len);
    if (sq < 1 || groups < 1 || max_prefix_len < 0)
        return report(PKD_EINVAL, "invalid shape: sq=%d groups=%d max_prefix_len=%d", sq, groups, max_prefix_len);
    pkd_status st = check_shape(B, (long long)B * sq, Hq, Hkv, D, P, max_kv_len, kv);
    if (st != PKD_OK) return st;
    if (groups > pkd::kPtMaxBatch) return report(PKD_EUNSUPPORTED, "groups %d > %d", groups, pkd::kPtMaxBatch);
    const int T = B * sq;
    const bool step = (long long)sq * (Hq / Hkv) <= 16;
    st = plan_attend(groups, T, T > 0 ? T : 1, Hq, Hkv, D, P, max_prefix_len, kv, true, false, pl.pre);
    if (st != PKD_OK) return st;
    st = plan_attend(B, T, std::min(sq, std::max(T, 1)), Hq, Hkv, D, P, max_kv_len, kv, false, step, pl.own);
    if (st != PKD_OK) return st;
    pl.off_own = kPartials + pl.pre.bytes();
    pl.off_own_lse = pl.off_own + pl.own.bytes();
    pl.off_own_out = pl.off_own_lse + up256((size_t)T * Hq * 4);
    pl.bytes = pl.off_own_out + up256((size_t)T * Hq * D * 4);
    return PKD_OK;
}

// Parameters common to the passes.
void fill(pkd::AttendParams& a, const AttendPlan& pl, uint8_t* ws, int pass, size_t off_partials, int B, long long T,
          int Hq, int Hkv, int P, int max_kv_len, int64_t num_pages, float scale2, float softcap, unsigned flags) {
    std::memset(&a, 0, sizeof a);
    a.status = reinterpret_cast<int32_t*>(ws);
    a.queue = a.status + kQueueWord[pass];
    a.counters = reinterpret_cast<int32_t*>(ws + kHeader);
    a.part_lse = reinterpret_cast<float*>(ws + off_partials);
    a.part_out = reinterpret_cast<float*>(ws + off_partials + pl.lse_bytes);
    a.fold = reinterpret_cast<float4*>(ws + off_partials + pl.lse_bytes + pl.out_bytes);
    a.B = B;
    a.T = (int)T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = pl.G;
    a.P = P;
    a.q_mul = 1;
    a.max_kv_len = max_kv_len;
    a.num_pages = num_pages;
    a.max_pairs = (int)pl.pairs;
    a.chunk = pl.chunk;
    a.max_splits = pl.max_splits;
    pkd::page_magic(P, a.pmagic, a.pmshift);
    a.scale_log2 = scale2;
    a.ref_up = (float)pl.ref_up;
    a.ref_pow = std::ldexp(1.f, pl.ref_up);
    if (softcap > 0.f) {
        // c tanh(s / c) with s = scale q.k: e^{2 s / c} = 2^(q.k * cap_in)
        a.cap_in = 2.f * scale2 / softcap;
        a.cap_log2 = softcap * pkd::kLog2e;
        // tanh(y) = y P(y^2) for |y| <= 0.6, P interpolating tanh(y)/y at the five
        // Chebyshev points of y^2 in [0, 0.36] (P off by 7.5e-8 at most, y P by 3.9e-8);
        // y = k q.k, and k and the scale go into the coefficients where they stay in
        // fp32's range
        static const double c[5] = {0.99999992596295, -0.3333230204036953, 0.1331006442560933, -0.05209665340812269,
                                    0.015468751301830112};
        const double k = (double)scale2 / ((double)softcap * pkd::kLog2e);
        double power = scale2;
        for (int i = 0; i < 5; ++i, power *= k * k) a.cap_c[i] = (float)(c[i] * power);
        a.cap_far = k > 2e-4 && k < 1e3 && scale2 > 1e-6f && scale2 < 1e6f ? (float)(0.6 / k) : -1.f;
    }
    a.wait_ns = (flags & PKD_FLAG_TEST_TIMEOUT) ? 0 : pkd::kWaitNs;
}

pkd_status cuda_fail(cudaError_t e, const char* what) {
    return report(PKD_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// One pass on the planned kernel.
pkd_status launch_pass(const pkd::AttendParams& a, const AttendPlan& pl, const void* kv_cache, pkd_dtype kv, int D,
                       bool partials, bool overlap, cudaStream_t stream, const char* what) {
    const uint64_t rows = (uint64_t)a.num_pages * a.Hkv * a.P;
    const int row_bytes = 2 * D * elt_bytes(kv);
    cudaError_t e;
    if (pl.step) {
        CUtensorMap tmap;
        pkd_status st = pkd::stage_map(tmap, kv_cache, rows, row_bytes, kv);
        if (st != PKD_OK) return st;
        pkd::DecodeParams d;
        std::memset(&d, 0, sizeof d);
        d.q = a.q;
        d.block_table = a.block_table;
        d.seq_lens = a.seq_lens;
        d.out = a.out;
        d.lse = a.lse;
        d.status = a.status;
        d.counters = a.counters;
        d.part_lse = a.part_lse;
        d.part_out = a.part_out;
        d.bt_stride = a.bt_stride;
        d.num_pages = a.num_pages;
        d.B = a.B;
        d.Hq = a.Hq;
        d.Hkv = a.Hkv;
        d.G = a.G;
        d.M = pl.rows;
        d.P = a.P;
        d.max_kv_len = a.max_kv_len;
        d.chunk = a.chunk;
        d.max_splits = a.max_splits;
        d.out_dtype = a.out_dtype;
        d.pmagic = a.pmagic;
        d.pmshift = a.pmshift;
        d.v_scale = a.v_scale;
        d.wait_ns = a.wait_ns;
        e = pkd::launch_attend_step(D, (int)kv, pl.rows > 8 ? 2 : 1, tmap, a, d, dim3(a.max_splits, a.Hkv, a.B), overlap,
                                    stream);
    } else {
        CUtensorMap kvmap, qmap;
        pkd_status st = pkd::half_stage_map(kvmap, kv_cache, rows, row_bytes, kv);
        if (st != PKD_OK) return st;
        st = pkd::query_map(qmap, a.q, D, a.Hq, (uint64_t)a.T, a.q_stride, a.G, pkd::kPtRows / a.G, kv);
        if (st != PKD_OK) return st;
        e = pkd::launch_attend_prompt(D, (int)kv, kvmap, qmap, a, partials, overlap, pl.units * pl.max_splits, stream);
    }
    return e == cudaSuccess ? PKD_OK : cuda_fail(e, what);
}

pkd_status check_call(const void* q, pkd_dtype q_dtype, int64_t q_stride, const void* kv_cache, pkd_dtype kv_dtype,
                      int64_t num_pages, int Hq, int Hkv, int D, int P, float scale, float q_scale, float k_scale,
                      float v_scale, float softcap, const void* out, pkd_dtype out_dtype, const float* lse,
                      const void* workspace, size_t workspace_bytes, size_t need) {
    if (q_dtype != kv_dtype)
        return report(PKD_EUNSUPPORTED, "q dtype (%d) must equal the cache dtype (%d)", (int)q_dtype, (int)kv_dtype);
    if (out_dtype != PKD_BF16 && out_dtype != PKD_FP16 && out_dtype != PKD_FP32)
        return report(PKD_EUNSUPPORTED, "out dtype %d not supported (bf16, fp16, fp32)", (int)out_dtype);
    if (!q || !kv_cache || !out || !workspace) return report(PKD_EINVAL, "null pointer argument");
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(lse, 4))
        return report(PKD_EINVAL, "misaligned pointer (q, kv_cache, out: 16 B; workspace: 256 B)");
    if (q_stride < (int64_t)Hq * D || (q_stride * elt_bytes(q_dtype)) % 16)
        return report(PKD_EINVAL, "q_stride must be >= num_heads*head_dim and a multiple of 16 bytes");
    if (q_stride > (int64_t)1 << 38) return report(PKD_EUNSUPPORTED, "q_stride > 2^38 elements");  // a tensor map's limit
    if (num_pages < 1) return report(PKD_EINVAL, "num_pages must be >= 1");
    if (num_pages > 0x7fffffffll / ((int64_t)Hkv * P))
        return report(PKD_EUNSUPPORTED, "cache too large: num_pages*num_kv_heads*page_size must be < 2^31");
    if (workspace_bytes < need)
        return report(PKD_EINVAL, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
    const float s = scale * q_scale * k_scale;
    if (!(s > 0.f) || !std::isfinite(s * pkd::kLog2e) || !std::isfinite(v_scale))
        return report(PKD_EINVAL, "scale*q_scale*k_scale must be positive and finite, v_scale finite");
    if (softcap > 0.f && !std::isfinite(2.f * s * pkd::kLog2e / softcap))
        return report(PKD_EINVAL, "softcap too small for scale*q_scale*k_scale: their quotient overflows");
    return PKD_OK;
}

pkd_status check_table(const int32_t* table, int64_t stride, const int32_t* lens, int max_len, int P, const char* name) {
    // (no keys, no columns: such a table may be null, and is not read)
    if ((!table && max_len > 0) || !lens) return report(PKD_EINVAL, "null pointer argument");
    if (!aligned(table, 4) || !aligned(lens, 4)) return report(PKD_EINVAL, "misaligned %s or lengths", name);
    const int64_t need = ((int64_t)max_len + P - 1) / P;
    if (stride < need)
        return report(PKD_EINVAL, "%s stride %lld < ceil(max length/page_size) = %lld", name, (long long)stride,
                      (long long)need);
    return PKD_OK;
}

// Results may be written while other CTAs still read q.
pkd_status check_overlap(const void* q, pkd_dtype q_dtype, int64_t q_stride, const void* out, pkd_dtype out_dtype,
                         int64_t T, int Hq, int D) {
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t q1 = q0 + ((T - 1) * q_stride + (int64_t)Hq * D) * elt_bytes(q_dtype);
    const uintptr_t o1 = o0 + T * Hq * D * elt_bytes(out_dtype);
    return q0 < o1 && o0 < q1 ? report(PKD_EINVAL, "out overlaps q") : PKD_OK;
}

const pkd_score_options kNoOptions = {0.f, nullptr, 0, nullptr, nullptr};

}  // namespace

cudaError_t pkd::launch_attend_prompt(int D, int kv_dtype, const CUtensorMap& kvmap, const CUtensorMap& qmap,
                                      const AttendParams& p, bool partials, bool overlap, long long items,
                                      cudaStream_t stream) {
    int grid = 1;
    cudaError_t e = persistent_grid(1, (int)std::min<long long>(items, kSms), grid);
    if (e != cudaSuccess) return e;
    if (kv_dtype == PKD_FP8_E4M3)
        return D == 128 ? launch_prompt_fp8_d128(kvmap, qmap, p, partials, overlap, grid, stream) : cudaErrorInvalidValue;
    if (kv_dtype == PKD_BF16)
        return D == 128 ? launch_prompt_bf16_d128(kvmap, qmap, p, partials, overlap, grid, stream)
                        : launch_prompt_bf16_d64(kvmap, qmap, p, partials, overlap, grid, stream);
    return D == 128 ? launch_prompt_fp16_d128(kvmap, qmap, p, partials, overlap, grid, stream)
                    : launch_prompt_fp16_d64(kvmap, qmap, p, partials, overlap, grid, stream);
}

extern "C" {

size_t pkd_paged_attention_workspace_size(int batch, int64_t total_tokens, int max_query_len, int num_heads,
                                          int num_kv_heads, int head_dim, int page_size, int max_kv_len,
                                          pkd_dtype kv_dtype, const pkd_score_options* options) {
    AttendPlan pl;
    const pkd_score_options& o = options ? *options : kNoOptions;
    return plan_paged_attention(batch, total_tokens, max_query_len, num_heads, num_kv_heads, head_dim, page_size,
                                max_kv_len, kv_dtype, o, pl) == PKD_OK ? kPartials + pl.bytes() : 0;
}

const char* pkd_paged_attention_kernel_name(int batch, int64_t total_tokens, int max_query_len, int num_heads,
                                            int num_kv_heads, int head_dim, int page_size, int max_kv_len,
                                            pkd_dtype kv_dtype, const pkd_score_options* options) {
    AttendPlan pl;
    const pkd_score_options& o = options ? *options : kNoOptions;
    if (plan_paged_attention(batch, total_tokens, max_query_len, num_heads, num_kv_heads, head_dim, page_size,
                             max_kv_len, kv_dtype, o, pl) != PKD_OK)
        return nullptr;
    return pl.step ? "step grid, tensor cores" : "persistent tcgen05 kernel, row tiles in TMEM";
}

pkd_status pkd_paged_attention(const void* q, pkd_dtype q_dtype, int64_t q_stride, const void* kv_cache,
                               pkd_dtype kv_dtype, int64_t num_pages, const int32_t* block_table,
                               int64_t block_table_stride, const int32_t* seq_lens, const int32_t* query_start,
                               int batch, int64_t total_tokens, int max_query_len, int num_heads, int num_kv_heads,
                               int head_dim, int page_size, int max_kv_len, float scale, float q_scale, float k_scale,
                               float v_scale, const pkd_score_options* options, void* out, pkd_dtype out_dtype,
                               float* lse, void* workspace, size_t workspace_bytes, unsigned flags, void* stream) {
    AttendPlan pl;
    const pkd_score_options& o = options ? *options : kNoOptions;
    pkd_status st = check_options(o);
    if (st != PKD_OK) return st;
    st = plan_paged_attention(batch, total_tokens, max_query_len, num_heads, num_kv_heads, head_dim, page_size,
                              max_kv_len, kv_dtype, o, pl);
    if (st != PKD_OK) return st;
    if (flags & ~(PKD_FLAG_CAUSAL | PKD_FLAG_TEST_TIMEOUT))
        return report(PKD_EUNSUPPORTED, "pkd_paged_attention takes PKD_FLAG_CAUSAL (and PKD_FLAG_TEST_TIMEOUT) only");
    if (o.prefix_lens && !(flags & PKD_FLAG_CAUSAL))
        return report(PKD_EINVAL, "prefix_lens needs PKD_FLAG_CAUSAL (without it every key is visible already)");
    if (batch == 0 || total_tokens == 0) return PKD_OK;
    st = check_call(q, q_dtype, q_stride, kv_cache, kv_dtype, num_pages, num_heads, num_kv_heads, head_dim, page_size,
                    scale, q_scale, k_scale, v_scale, o.softcap, out, out_dtype, lse, workspace, workspace_bytes,
                    kPartials + pl.bytes());
    if (st != PKD_OK) return st;
    st = check_table(block_table, block_table_stride, seq_lens, max_kv_len, page_size, "block_table");
    if (st != PKD_OK) return st;
    if (!query_start || !aligned(query_start, 4)) return report(PKD_EINVAL, "query_start is null or misaligned");
    st = check_overlap(q, q_dtype, q_stride, out, out_dtype, total_tokens, num_heads, head_dim);
    if (st != PKD_OK) return st;
    pkd::AttendParams a;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    fill(a, pl, ws, 0, kPartials, batch, total_tokens, num_heads, num_kv_heads, page_size, max_kv_len, num_pages,
         scale * q_scale * k_scale * pkd::kLog2e, o.softcap, flags);
    a.q = q;
    a.q_stride = q_stride;
    a.block_table = block_table;
    a.bt_stride = block_table_stride;
    a.seq_lens = seq_lens;
    a.query_start = query_start;
    a.prefix_lens = o.prefix_lens;
    a.doc_start = o.doc_start;
    a.slopes = o.alibi_slopes;
    a.window = o.window > 0 ? std::min(o.window, 2 * kMaxKeys) : 0;  // positions less a window stay above -2^31
    a.causal = (flags & PKD_FLAG_CAUSAL) ? 1 : 0;
    a.max_q = max_query_len;
    a.out = out;
    a.lse = lse;
    a.out_dtype = (int)out_dtype;
    a.v_scale = v_scale;
    return launch_pass(a, pl, kv_cache, kv_dtype, head_dim, false, false, (cudaStream_t)stream,
                       "pkd_paged_attention launch");
}

size_t pkd_prefix_decode_workspace_size(int batch, int sq, int num_heads, int num_kv_heads, int head_dim,
                                        int page_size, int groups, int max_prefix_len, int max_kv_len,
                                        pkd_dtype kv_dtype) {
    PrefixPlan pl;
    return plan_prefix(batch, sq, num_heads, num_kv_heads, head_dim, page_size, groups, max_prefix_len, max_kv_len,
                       kv_dtype, pl) == PKD_OK ? pl.bytes : 0;
}

pkd_status pkd_prefix_decode(const void* q, pkd_dtype q_dtype, const void* kv_cache, pkd_dtype kv_dtype,
                             int64_t num_pages, const int32_t* prefix_table, int64_t prefix_table_stride,
                             const int32_t* prefix_lens, const int32_t* group_start, int groups, int max_prefix_len,
                             const int32_t* block_table, int64_t block_table_stride, const int32_t* seq_lens, int batch,
                             int sq, int num_heads, int num_kv_heads, int head_dim, int page_size, int max_kv_len,
                             float scale, float q_scale, float k_scale, float v_scale, float softcap, void* out,
                             pkd_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes, unsigned flags,
                             void* stream) {
    PrefixPlan pl;
    pkd_score_options o = kNoOptions;
    o.softcap = softcap;
    pkd_status st = check_options(o);
    if (st != PKD_OK) return st;
    st = plan_prefix(batch, sq, num_heads, num_kv_heads, head_dim, page_size, groups, max_prefix_len, max_kv_len,
                     kv_dtype, pl);
    if (st != PKD_OK) return st;
    if (flags & ~(PKD_FLAG_CAUSAL | PKD_FLAG_TEST_TIMEOUT))
        return report(PKD_EUNSUPPORTED, "pkd_prefix_decode takes PKD_FLAG_CAUSAL (and PKD_FLAG_TEST_TIMEOUT) only");
    if (batch == 0) return PKD_OK;
    st = check_call(q, q_dtype, (int64_t)num_heads * head_dim, kv_cache, kv_dtype, num_pages, num_heads, num_kv_heads,
                    head_dim, page_size, scale, q_scale, k_scale, v_scale, softcap, out, out_dtype, lse, workspace,
                    workspace_bytes, pl.bytes);
    if (st != PKD_OK) return st;
    st = check_table(block_table, block_table_stride, seq_lens, max_kv_len, page_size, "block_table");
    if (st != PKD_OK) return st;
    st = check_table(prefix_table, prefix_table_stride, prefix_lens, max_prefix_len, page_size, "prefix_table");
    if (st != PKD_OK) return st;
    if ((!group_start && groups != 1) || !aligned(group_start, 4))
        return report(PKD_EINVAL, "group_start is misaligned, or null with more than one group");
    st = check_overlap(q, q_dtype, (int64_t)num_heads * head_dim, out, out_dtype, (int64_t)batch * sq, num_heads, head_dim);
    if (st != PKD_OK) return st;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const long long T = (long long)batch * sq;
    const float scale2 = scale * q_scale * k_scale * pkd::kLog2e;
    cudaStream_t s = (cudaStream_t)stream;
    // the rows of a group's requests are one dense query block over its prefix
    pkd::AttendParams a;
    fill(a, pl.pre, ws, 0, kPartials, groups, T, num_heads, num_kv_heads, page_size, max_prefix_len, num_pages, scale2, softcap,
         flags);
    a.q = q;
    a.q_stride = (long long)num_heads * head_dim;
    a.block_table = prefix_table;
    a.bt_stride = prefix_table_stride;
    a.seq_lens = prefix_lens;
    a.query_start = group_start;
    a.q_mul = sq;
    a.sq = (int)T;  // without group_start: one group of every request
    a.max_q = (int)T;
    a.v_scale = 1.f;
    st = launch_pass(a, pl.pre, kv_cache, kv_dtype, head_dim, true, false, s, "pkd_prefix_decode prefix launch");
    if (st != PKD_OK) return st;
    // each request's own keys: beside the prefix (programmatic dependent launch)
    pkd::AttendParams b;
    fill(b, pl.own, ws, 1, pl.off_own, batch, T, num_heads, num_kv_heads, page_size, max_kv_len, num_pages, scale2,
         softcap, flags);
    b.q = q;
    b.q_stride = a.q_stride;
    b.block_table = block_table;
    b.bt_stride = block_table_stride;
    b.seq_lens = seq_lens;
    b.sq = sq;
    b.max_q = sq;
    b.causal = (flags & PKD_FLAG_CAUSAL) ? 1 : 0;
    b.out = ws + pl.off_own_out;
    b.lse = reinterpret_cast<float*>(ws + pl.off_own_lse);
    b.out_dtype = PKD_FP32;
    b.v_scale = 1.f;
    st = launch_pass(b, pl.own, kv_cache, kv_dtype, head_dim, false, true, s, "pkd_prefix_decode launch");
    if (st != PKD_OK) return st;
    pkd::PrefixMergeParams m;
    std::memset(&m, 0, sizeof m);
    m.part_lse = a.part_lse;
    m.part_out = a.part_out;
    m.own_lse = b.lse;
    m.own_out = static_cast<const float*>(b.out);
    m.group_start = group_start;
    m.prefix_lens = prefix_lens;
    m.out = out;
    m.lse = lse;
    m.groups = groups;
    m.rows = (int)(T * num_heads);
    m.rows_per_request = sq * num_heads;
    m.chunk = pl.pre.chunk;
    m.max_prefix_len = max_prefix_len;
    m.max_splits = pl.pre.max_splits;
    m.out_dtype = (int)out_dtype;
    m.v_scale = v_scale;
    const cudaError_t e = pkd::launch_prefix_merge(head_dim, m, s);
    return e == cudaSuccess ? PKD_OK : cuda_fail(e, "pkd_prefix_decode join launch");
}

}  // extern "C"
