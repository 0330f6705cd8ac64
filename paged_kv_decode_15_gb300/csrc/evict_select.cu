// pkd_evict_select: which keys of each (request, kv head) stay.
//
// A key's rank is a 32-bit number that rises with its (pooled) weight; protected keys
// have the largest.  The n-th largest rank is found three bits at a time from the top:
// every round counts the keys under the current prefix by their next three bits (a
// count per thread and digit, a warp sum, a sum over the warps), so that the time does
// not depend on how the weights are spread, and nothing is ordered by atomics.  Then
// one pass in the order of the keys writes those above the threshold, and as many of
// those on it as are still missing, the lowest indexes first.
#include "evict.cuh"
#include "ptx.cuh"

namespace pkd {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;

// The rank of a weight: rises with it, NaN as -inf, -0 as +0, below that of a protected key.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return x != x ? 0x007fffffu : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
    __shared__ int counts[2][kSelWarps][8];
    __shared__ int above[kSelWarps], on[kSelWarps];
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int L = min(max(p.seq_lens[b], 0), p.keys), n = min(L, p.budget);
    int32_t* kept = p.kept + (static_cast<long long>(b) * p.H + h) * p.budget;
    if (h == 0 && tid == 0) p.kept_lens[b] = n;
    for (int i = n + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
    if (L <= p.budget) {
        for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
        return;
    }
    const float* w = p.weights + b * p.weights_b + h * p.weights_h;
    const int32_t* pos = p.positions ? p.positions + b * p.positions_b + h * p.positions_h : nullptr;
    const int context = pos ? max(p.context_lens[b], 0) : L;
    const int first = p.sinks, past = context - p.recent, side = p.pool / 2;
    auto rank = [&](int t) {
        const int at = pos ? pos[t] : t;
        if (at < first || at >= past) return 0xffffffffu;
        float x = w[t];
        if (side) {
            const int z = min(t + side, past - 1);
            for (int s = max(t - side, first); s <= z; ++s) x = fmaxf(x, w[s]);  // (a NaN beside a number counts not)
        }
        return rank_of(x);
    };

    uint32_t prefix = 0;
    int missing = n;  // of the keys under the prefix
    int shift = 32;
    for (int round = 0; shift > 0; ++round) {
        const int bits = min(3, shift);
        shift -= bits;
        int c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int t = tid; t < L; t += kSelThreads) {
            const uint32_t r = rank(t);
            if (bits + shift < 32 && (r >> (shift + bits)) != prefix) continue;
            const int d = (r >> shift) & ((1 << bits) - 1);
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] += d == e;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = __reduce_add_sync(kFull, c[e]);
        int(*all)[8] = counts[round & 1];
        if (lane == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) all[warp][e] = c[e];
        __syncthreads();
        int digit = 0, count = 0;
        for (digit = 7; digit >= 0; --digit) {
            count = 0;
            for (int k = 0; k < kSelWarps; ++k) count += all[k][digit];
            if (count >= missing) break;
            missing -= count;
        }
        prefix = prefix << bits | digit;
        if (count == missing) break;  // all keys under the prefix stay
    }
    // The keys above the prefix stay, and the first `missing` of those under it.  A warp
    // takes a run of consecutive keys.
    const int run = (L + kSelThreads - 1) / kSelThreads * 32, t0 = warp * run, t1 = min(t0 + run, L);
    int na = 0, no = 0;
    for (int t = t0 + lane; t < t0 + run; t += 32) {
        const uint32_t r = t < t1 ? rank(t) >> shift : 0u;
        na += __popc(__ballot_sync(kFull, t < t1 && r > prefix));
        no += __popc(__ballot_sync(kFull, t < t1 && r == prefix));
    }
    if (lane == 0) above[warp] = na, on[warp] = no;
    __syncthreads();
    na = no = 0;
    for (int k = 0; k < warp; ++k) na += above[k], no += on[k];
    const unsigned below = (1u << lane) - 1;
    for (int t = t0 + lane; t < t0 + run; t += 32) {
        const uint32_t r = t < t1 ? rank(t) >> shift : 0u;
        const unsigned va = __ballot_sync(kFull, t < t1 && r > prefix), vo = __ballot_sync(kFull, t < t1 && r == prefix);
        const int a = na + __popc(va & below), o = no + __popc(vo & below);
        if ((va >> lane & 1) || ((vo >> lane & 1) && o < missing)) kept[a + min(o, missing)] = t;
        na += __popc(va);
        no += __popc(vo);
    }
}

cudaError_t launch_evict_select(const SelectParams& p, cudaStream_t stream) {
    evict_select_kernel<<<dim3(p.H, p.B), kSelThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkd
