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
    const float* slopes;          // [Hq] or null
    void* out;                    // [T, Hq, D]
    float* lse;                   // [T, Hq] or null
    int32_t* status;
    int32_t* queue;               // next work item, CTAs done (tcgen05 kernel)
    int32_t* counters;            // arrivals per split unit
    float* part_lse;              // log2 domain
    float* part_out;
    long long bt_stride, num_pages, q_stride;
    int B, T, Hq, Hkv, G, P;
    int sq, q_mul, max_q, max_kv_len;
    int window, causal;
    int chunk, max_splits, out_dtype;
    uint32_t pmagic;
    int pmshift;
    float scale_log2;             // logit = q.k * scale_log2 (log2 units), without a cap
    float cap_in, cap_log2;       // with one: cap_log2 * tanh(q.k * cap_in / (2 log2 e)); cap_log2 = 0: none
    float cap_c[5], cap_far;      // the capped logit as q.k times a polynomial in (q.k)^2, for |q.k| <= cap_far
    float v_scale;
    uint64_t wait_ns;
};

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

// c tanh(scale q.k / c) in log2 units: tanh(y) = 1 - 2 / (1 + e^{2y}), with
// e^{2y} = 2^(q.k * cap_in).  Absolute error about 2^-23 of the cap; the two ends
// (2^inf, 2^-inf) give +-1.
__device__ __forceinline__ float capped(float qk, float cap_in, float cap_log2) {
    return cap_log2 * fmaf(-2.f, rcp_approx(1.f + fast_exp2(qk * cap_in)), 1.f);
}

}  // namespace pkd
