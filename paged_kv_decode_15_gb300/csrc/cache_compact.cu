// pkd_cache_compact: the rows that stay go below the new length.
//
// Of the n kept rows of a (request, kv head) those that lie below n stay where they
// are; the others, from the c-th on, fill the free slots below n, in order.  Sources
// lie at n or behind, targets below: in place without any order between the copies,
// and no more rows move than must.  The m-th free slot is m + i, i the first kept row
// with kept[i] - i > m (kept[i] - i slots are free before it): a binary search.
#include <algorithm>

#include "evict.cuh"
#include "launch.h"
#include "page_math.h"
#include "ptx.cuh"

namespace pkd {

constexpr int kCompactThreads = 256;

// LANES lanes of 16 bytes to a row.
template <int LANES>
__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(const CompactParams p) {
    constexpr int ROWB = LANES * 16;
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
    const int n = min(max(p.kept_lens[b], 0), p.budget);
    const int32_t* kept = p.kept + (static_cast<long long>(b) * p.H + h) * p.budget;
    const int32_t* table = p.block_table + b * p.bt_stride;
    // the first i in [0, n) for which f is true, f rising
    auto first = [&](auto f) {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (f(mid)) hi = mid; else lo = mid + 1;
        }
        return lo;
    };
    const int stay = first([&](int i) { return kept[i] >= n; });
    auto row_of = [&](int t) -> long long {
        const int col = page_div(t, p.pmagic, p.pmshift), page = table[col];
        if (page < 0 || page >= p.num_pages) return -1;
        return (static_cast<long long>(page) * p.H + h) * p.P + (t - col * p.P);
    };
    const int warp = blockIdx.x * (kCompactThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kCompactThreads / 32);
    for (int m0 = 32 * warp; m0 < n - stay; m0 += 32 * warps) {
        // a lane looks up one row's way
        long long from = -1, to = -1;
        const int m = m0 + lane;
        if (m < n - stay) {
            const int s = kept[stay + m], d = m + first([&](int i) { return kept[i] - i > m; });
            if (s >= n && s < p.keys && d < n && d < p.keys) {
                from = row_of(s);
                to = row_of(d);
                if (from < 0 || to < 0) from = -1;
                if (from >= 0) {
                    if (p.weights) {
                        float* w = p.weights + b * p.weights_b + h * p.weights_h;
                        w[d] = w[s];
                    }
                    if (p.positions) {
                        int32_t* x = p.positions + b * p.positions_b + h * p.positions_h;
                        x[d] = x[s];
                    }
                }
            }
        }
        constexpr int R = 32 / LANES, N = 8;  // rows of a load instruction, instructions in flight
        const int part = lane % LANES;
#pragma unroll 1
        for (int k = 0; k < 32; k += R * N) {
            uint4 v[N];
            long long dst[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int src = (k + i * R + lane / LANES) & 31;
                const long long f = __shfl_sync(kFull, from, src);
                dst[i] = __shfl_sync(kFull, to, src);
                if (f < 0) dst[i] = -1;
                if (f >= 0) v[i] = __ldcs(reinterpret_cast<const uint4*>(p.cache + f * ROWB) + part);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (dst[i] >= 0) reinterpret_cast<uint4*>(p.cache + dst[i] * ROWB)[part] = v[i];
        }
    }
}

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream) {
    const int parts = std::max(1, (p.budget + kCompactThreads - 1) / kCompactThreads);
    const dim3 grid(std::min(parts, 65535), p.H, p.B);
    switch (p.row_bytes) {
        case 512: cache_compact_kernel<32><<<grid, kCompactThreads, 0, stream>>>(p); break;
        case 256: cache_compact_kernel<16><<<grid, kCompactThreads, 0, stream>>>(p); break;
        case 128: cache_compact_kernel<8><<<grid, kCompactThreads, 0, stream>>>(p); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace pkd
