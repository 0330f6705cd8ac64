// Shared pieces of the ragged paged-attention kernels (pkd_paged_attention,
// pkd_prefix_decode): launch parameters, a request's query tokens, the key
// interval each token sees, and the score modifications.
//
// Every mask here leaves a query token one interval of keys [lo, hi):
//   hi = L, or causal: max(pos + 1, prefix_len) (a prefix mask), capped at L
//   lo = 0, raised to pos - (window - 1) and to the token's doc_start
// so the kernels carry two integers per row and never read a mask.
#pragma once

#include "decode_common.cuh"

namespace pkd {

struct AttendParams {
    const void* q;                // [T, Hq, D], token stride q_stride elements
    const int32_t* block_table;   // [B, bt_stride]
    const int32_t* seq_lens;      // [B]
    const int32_t* query_start;   // [B + 1] (times q_mul), or null: sq tokens per request
    const int32_t* prefix_lens;   // [B] or null
    const int32_t* doc_start;     // [T] or null
    const int32_t* key_start;     // packed keys (pkd_packed_attention): [B + 1], rows of k and v
    const float* slopes;          // [Hq] or null
    void* out;                    // [T, Hq, D]
    float* lse;                   // [T, Hq] or null
    int32_t* status;
    int32_t* queue;               // next work item, CTAs done (tcgen05 kernel)
    int32_t* counters;            // arrivals per split unit
    float* part_lse;              // log2 domain
    float* part_out;
    float4* fold;                 // tcgen05 kernel: per CTA, what long sums were folded into
    long long bt_stride, num_pages, q_stride;
    int B, T, Hq, Hkv, G, P;
    int sq, q_mul, max_q, max_kv_len;
    int total_keys;               // packed keys: rows of k and v
    int max_pairs;                // row-tile pairs of a kv head that the plan has room for (tcgen05 kernel)
    int window, causal;
    int chunk, max_splits, out_dtype;
    uint32_t pmagic;
    int pmshift;
    float scale_log2;             // logit = q.k * scale_log2 (log2 units), without a cap
    float cap_in, cap_log2;       // with one: cap_log2 * tanh(q.k * cap_in / (2 log2 e)); cap_log2 = 0: none
    float cap_c[5], cap_far;      // the capped logit as q.k times a polynomial in (q.k)^2, for |q.k| <= cap_far
    // tcgen05 kernel: a row's weights are 2^(logit - m), m = its maximum + ref_up when the
    // reference was set; ref_pow = 2^ref_up
    float ref_up, ref_pow;
    float v_scale;
    uint64_t wait_ns;             // limit of a wait on a copy (0: a single test, PKD_FLAG_TEST_TIMEOUT)
};

// Programmatic dependent launch: let the next launch start (every CTA says so once),
// and wait for the launch before this one to have completed (no wait without one).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Query tokens [q0, q0 + n) of request b, clamped to [0, T] and to max_q
// tokens; a bad query_start raises the status word when `report` is set.
__device__ __forceinline__ void request_tokens(const AttendParams& p, int b, int& q0, int& n, bool report) {
    if (!p.query_start) {
        q0 = b * p.sq;
        n = p.sq;
        return;
    }
    long long s = static_cast<long long>(p.query_start[b]) * p.q_mul;
    long long e = static_cast<long long>(p.query_start[b + 1]) * p.q_mul;
    const bool bad = s < 0 || e < s || e > p.T || e - s > p.max_q;
    if (bad) {
        if (report) atomicOr(p.status, kErrBounds);
        s = s < 0 ? 0 : s > p.T ? p.T : s;
        e = e < s ? s : e > p.T ? p.T : e;
        if (e - s > p.max_q) e = s + p.max_q;
    }
    q0 = static_cast<int>(s);
    n = static_cast<int>(e - s);
}

__device__ __forceinline__ int request_len(const AttendParams& p, int b, bool report) {
    int L = p.seq_lens[b];
    if (L < 0 || L > p.max_kv_len) {
        if (report) atomicOr(p.status, kErrBounds);
        L = L < 0 ? 0 : p.max_kv_len;
    }
    return L;
}

// Keys [lo, hi) that query token i of a request (first token q0, n tokens,
// length L, prefix keys `prefix`) sees; empty intervals come back as [0, 0).
__device__ __forceinline__ void token_keys(const AttendParams& p, int q0, int n, int L, int prefix, int i, int& lo,
                                           int& hi) {
    const int pos = L - n + i;
    hi = p.causal ? max(pos + 1, prefix) : L;
    hi = min(hi, L);
    lo = p.window > 0 ? max(0, pos - (p.window - 1)) : 0;
    if (p.doc_start) lo = max(lo, p.doc_start[q0 + i]);
    if (lo >= hi) lo = hi = 0;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c tanh(scale q.k / c) in log2 units, y = scale q.k / c, with x = q.k * cap_in =
// 2 y log2 e: tanh(y) = 1 - 2 / (1 + 2^x), off by 2^-23 of the cap or so; near 0,
// where that would be lost on a large cap, y times the first terms of tanh's series
// (|y| < 0.174, off by 1.8e-8 of y at most).  2^inf and 2^-inf give +-1.
__device__ __forceinline__ float capped(float qk, float cap_in, float cap_log2) {
    const float x = qk * cap_in, y = x * 0.34657359f, z = y * y;
    const float near = y * fmaf(z, fmaf(z, fmaf(z, -0.053968254f, 0.13333334f), -0.33333334f), 1.f);
    const float far = fmaf(-2.f, rcp_approx(1.f + fast_exp2(x)), 1.f);
    return cap_log2 * (fabsf(x) < 0.5f ? near : far);
}

// The D / 32 dims of a row that lane `lane` holds (from lane * D / 32 on).
template <int D>
__device__ __forceinline__ void load_row(const float* row, int lane, float (&v)[D / 32]) {
    if constexpr (D == 128) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(row) + lane);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(row) + lane);
        v[0] = x.x; v[1] = x.y;
    }
}

// out[row] = v * scale, rounded once to its type.
template <int D>
__device__ __forceinline__ void store_row(void* out, long long row, const float (&v)[D / 32], float scale, int lane,
                                          int dtype) {
    float x[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) x[e] = v[e] * scale;
    if (dtype == 3) {
        float* dst = static_cast<float*>(out) + row * D + lane * (D / 32);
        if constexpr (D == 128)
            *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
        else
            *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
    } else {
        uint32_t h[D / 64];
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
            h[e] = dtype == 0 ? pack2<true>(x[2 * e], x[2 * e + 1]) : pack2<false>(x[2 * e], x[2 * e + 1]);
        uint16_t* dst = static_cast<uint16_t*>(out) + row * D + lane * (D / 32);
        if constexpr (D == 128)
            *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
        else
            *reinterpret_cast<uint32_t*>(dst) = h[0];
    }
}

// Merge the partial results of one row by LSE (log2 units), a warp per row: part s
// has its LSE at pl[s * step] and its output at po + s * step * D.  All LSEs first,
// one per lane, then eight outputs in flight; a part without keys is never
// read.  Partials come from other CTAs: L2 loads.  acc: the weighted sum, mx: the
// largest LSE, ws: the sum of the weights.
template <int D>
__device__ __forceinline__ void merge_row(const float* pl, const float* po, long long step, int np, int lane,
                                          float (&acc)[D / 32], float& mx, float& ws) {
    constexpr int E = D / 32, N = 8;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    mx = -INFINITY;
    ws = 0.f;
    const float first = lane < np ? __ldcg(pl + lane * step) : -INFINITY;
    mx = first;
    for (int s = 32 + lane; s < np; s += 32) mx = fmaxf(mx, __ldcg(pl + s * step));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    if (mx == -INFINITY) return;
    for (int s0 = 0; s0 < np; s0 += 32) {
        const float l = s0 == 0 ? first : s0 + lane < np ? __ldcg(pl + (s0 + lane) * step) : -INFINITY;
        const float wl = l == -INFINITY ? 0.f : fast_exp2(l - mx);
        ws += wl;
        const int m = min(32, np - s0);
        for (int j = 0; j < m; j += N) {
            float v[N][E], w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                w[i] = __shfl_sync(kFull, wl, (j + i) & 31);
                if (j + i >= m) w[i] = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] = 0.f;
                if (w[i] > 0.f) load_row<D>(po + (s0 + j + i) * step * D, lane, v[i]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(w[i], v[i][e], acc[e]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kFull, ws, o);
}

}  // namespace pkd
