// Shared-prefix decode: the join, by LSE, of the prefix's partial results (one
// per chunk of the prefix) with the result over the request's own keys.
//
// One warp per output row; lane l holds dims l * D/32 onwards.  Everything it
// reads was written by the launches before it and mostly still lies in L2: 2048 rows
// of 19 chunks (20 MB) take 9 us, launch included.
#include "attend.cuh"
#include "attend_launch.h"

namespace pkd {

template <int D>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixMergeParams p) {
    constexpr int E = D / 32;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= p.rows) return;
    // the request's group: group_start[g] <= b < group_start[g + 1]
    const int b = row / p.rows_per_request;
    int np = 0;
    if (!p.group_start || (b >= p.group_start[0] && b < p.group_start[p.groups])) {
        int lo = 0, hi = p.group_start ? p.groups : 1;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.group_start[mid] <= b) lo = mid; else hi = mid;
        }
        const int len = min(max(p.prefix_lens[lo], 0), p.max_prefix_len);
        np = min((len + p.chunk - 1) / p.chunk, p.max_splits);
    }
    wait_dependency();  // the two passes before it
    float acc[E], mx, ws;
    merge_row<D>(p.part_lse + row, p.part_out + static_cast<long long>(row) * D, p.rows, np, lane, acc, mx, ws);
    const float own = p.own_lse[row] * kLog2e;
    if (own != -INFINITY) {
        const float top = fmaxf(mx, own);
        const float a = mx == -INFINITY ? 0.f : fast_exp2(mx - top), w = fast_exp2(own - top);
        float own_row[E];
        load_row<D>(p.own_out + static_cast<long long>(row) * D, lane, own_row);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * own_row[e];
        ws = ws * a + w;
        mx = top;
    }
    const float sc = ws > 0.f ? p.v_scale / ws : 0.f;
    store_row<D>(p.out, row, acc, sc, lane, p.out_dtype);
    if (lane == 0 && p.lse) p.lse[row] = ws > 0.f ? (mx + __log2f(ws)) * kLn2 : -INFINITY;
}

cudaError_t launch_prefix_merge(int D, const PrefixMergeParams& p, cudaStream_t stream) {
    if (p.rows == 0) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>((p.rows + 3) / 4));
    return D == 128 ? launch_kernel(prefix_merge_kernel<128>, grid, 128, 0, true, stream, p)
                    : launch_kernel(prefix_merge_kernel<64>, grid, 128, 0, true, stream, p);
}

}  // namespace pkd
