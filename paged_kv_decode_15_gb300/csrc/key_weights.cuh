// Attention weight received by the keys of a paged cache (pkd_key_weights): launch
// parameters and what its kernels share.
//
//   w[b, h, t] = decay * prior[b, h, t] + sum over the weighing tokens i of request b and
//                the query heads g of kv head h of  exp(s(i, g, t) - lse(i, g))
// with the scores s and the masks of pkd_paged_attention, whose LSE turns a score into
// a probability without a second softmax: no maximum, no sum over keys.  K alone is
// read, and every key's sum is one thread's (or one lane quad's): no atomics, the same
// bits every time.
#pragma once

#include "attend.cuh"

namespace pkd {

struct WeighParams {
    AttendParams a;               // q, the table, lengths, masks and scores
    const uint8_t* cache;
    const float* lse;             // [T, Hq] natural log
    const float* prior;           // [B, Hkv, keys] with strides, or null
    float* weights;               // the same layout; may be prior itself
    long long prior_b, prior_h, weights_b, weights_h;
    float decay;
    int last;                     // the last tokens of each request that weigh (0: all)
    int run, stay;                // tcgen05 kernel: key blocks of an item; query tiles stay for all of them
};

// The weighing tokens of a request: token i of m is row first + i of q, at position
// L - m + i.  Keys from `fresh` on are the call's own (no earlier weight).
struct WeighRequest {
    int first, m, L, fresh;
};
__device__ __forceinline__ WeighRequest weigh_request(const WeighParams& w, int b, bool report) {
    WeighRequest r;
    int q0, n;
    request_tokens(w.a, b, q0, n, report);
    r.L = request_len(w.a, b, report);
    r.m = w.last > 0 ? min(n, w.last) : n;
    r.first = q0 + n - r.m;
    r.fresh = r.L - n;
    return r;
}

}  // namespace pkd
