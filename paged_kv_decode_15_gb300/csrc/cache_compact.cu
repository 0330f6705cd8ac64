// pkd_cache_compact: the rows that stay go below the new length.
//
// Of the n kept rows of a (request, kv head) those that lie below n stay where they
// are; the others, from the c-th on, fill the free slots below n, in order.  Sources
// lie at n or behind, targets below: in place without any order between the copies,
// and no more rows move than must.  The m-th free slot is m + i, i the first kept row
// with kept[i] - i > m (kept[i] - i slots are free before it): a binary search, in shared
// memory, where every CTA of a (request, kv head) has its kept list (longer ones are
// searched where they are).  Bound by the rows' bytes, read and written (32 lists of 4096
// of up to 32768 keys, 512-byte rows: 24.1 us, 4.7 TB/s, 0.69 of the copy); for few rows by
// the chain lengths - list - table - rows of trips to memory (512 lists of 1024 of 1088
// keys: 6.6 us, of which the bytes take 5).  Searched in global memory: 31 and 22 us.
#include <algorithm>

#include "evict.cuh"
#include "launch.h"
#include "page_math.h"
#include "ptx.cuh"

namespace pkd {

constexpr int kCompactThreads = 256, kCompactWarps = kCompactThreads / 32;
constexpr int kCompactList = 10240;  // kept rows in shared memory
constexpr int kCompactFlight = 8;    // load instructions of a warp in flight

// LANES lanes of 16 bytes to a row.
template <int LANES>
__global__ void __launch_bounds__(kCompactThreads, 4) cache_compact_kernel(const CompactParams p) {
    constexpr int ROWB = LANES * 16, R = 32 / LANES, ROWS = R * kCompactFlight;  // rows of a warp at a time
    static_assert(ROWS <= 32, "a lane finds one row's way");
    extern __shared__ int32_t list[];
    __shared__ int stays;
    const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int given = p.kept_lens[b], n = min(max(given, 0), p.budget);
    const int32_t* kept = p.kept + (static_cast<long long>(b) * p.H + h) * p.budget;
    const int32_t* table = p.block_table + b * p.bt_stride;
    const bool local = p.budget <= kCompactList;
    if (tid == 0) {
        stays = 0;
        if (p.status && n != given) atomicOr(p.status, kErrBounds);
    }
    __syncthreads();
    // rows that stay where they are, and the list
    int count = 0;
    for (int i0 = 0; i0 < n; i0 += 4 * kCompactThreads) {
        int x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e * kCompactThreads + tid;
            x[e] = i < n ? kept[i] : 0x7fffffff;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e * kCompactThreads + tid;
            if (i < n && local) list[i] = x[e];
            count += i < n && x[e] < n;
        }
    }
    count = __reduce_add_sync(kFull, count);
    if (lane == 0 && count) atomicAdd(&stays, count);
    __syncthreads();
    const int stay = stays, moves = n - stay;
    auto at = [&](int i) { return local ? list[i] : kept[i]; };
    auto row_of = [&](int t) -> long long {
        const int col = page_div(t, p.pmagic, p.pmshift), page = table[col];
        if (page < 0 || page >= p.num_pages) return -1;
        return (static_cast<long long>(page) * p.H + h) * p.P + (t - col * p.P);
    };
    // a warp's rows at a time: a lane finds the way of one; few rows are spread over all warps
    const int warps = gridDim.x * kCompactWarps, share = (moves + warps - 1) / warps;
    const int batch = min(32, (share + ROWS - 1) / ROWS * ROWS);
    for (int m0 = (blockIdx.x * kCompactWarps + warp) * batch; m0 < moves; m0 += warps * batch) {
        // a lane looks up one row's way
        long long from = -1, to = -1;
        const int m = m0 + lane;
        if (lane < batch && m < moves) {
            int lo = 0, hi = stay;  // the first i < stay with kept[i] - i > m, or stay
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (at(mid) - mid > m) hi = mid; else lo = mid + 1;
            }
            const int s = at(stay + m), d = m + lo;
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
            if (from < 0 && p.status) atomicOr(p.status, kErrBounds);  // the row is lost to the new length
        }
        const int part = lane % LANES;
#pragma unroll 1
        for (int k = 0; k < batch; k += ROWS) {
            uint4 v[kCompactFlight];
#pragma unroll
            for (int i = 0; i < kCompactFlight; ++i) {
                const long long f = __shfl_sync(kFull, from, (k + i * R + lane / LANES) & 31);
                if (f >= 0) v[i] = __ldcg(reinterpret_cast<const uint4*>(p.cache + f * ROWB) + part);
            }
#pragma unroll
            for (int i = 0; i < kCompactFlight; ++i) {
                const int src = (k + i * R + lane / LANES) & 31;
                const long long f = __shfl_sync(kFull, from, src), d = __shfl_sync(kFull, to, src);
                if (f >= 0) reinterpret_cast<uint4*>(p.cache + d * ROWB)[part] = v[i];
            }
        }
    }
}

template <int LANES>
static cudaError_t launch_one(const CompactParams& p, cudaStream_t stream) {
    // CTAs of a (request, kv head): four per SM in all at most (one wave: a second one cost 1.4
    // of 7.6 us where 512 lists got two CTAs each), no more than its rows feed
    constexpr int kRows = 32 / LANES * kCompactFlight * kCompactWarps;
    const long long units = static_cast<long long>(p.B) * p.H;
    const int most = std::min((p.budget + kRows - 1) / kRows, 65535);
    const int parts = static_cast<int>(std::max(1ll, std::min<long long>(most, 4 * 152 / std::max(units, 1ll))));
    const size_t smem = p.budget <= kCompactList ? p.budget * sizeof(int32_t) : 0;
    cache_compact_kernel<LANES><<<dim3(parts, p.H, p.B), kCompactThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactParams& p, cudaStream_t stream) {
    switch (p.row_bytes) {
        case 512: return launch_one<32>(p, stream);
        case 256: return launch_one<16>(p, stream);
        case 128: return launch_one<8>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace pkd
