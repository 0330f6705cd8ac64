// pkd_evict_select: which keys of each (request, kv head) stay.
//
// A key's rank is a 32-bit number that rises with its (pooled) weight; protected keys
// have the largest.  The n-th largest rank is found by three histograms, of its upper
// 11 bits, then, among the keys that share those of the threshold, of the next 11 and of
// the last 10 (fewer where a histogram ends on a bin of which all keys stay): counts
// in shared memory by integer atomics, whose order changes nothing, and a scan from the
// top.  Keys without any weight, often a third of them, are counted apart by votes.  Then
// the keys above the threshold, and as many of those on it as are still missing, the
// lowest indexes first, are written in the order of the keys: a warp owns a run of
// consecutive keys, counts, and writes behind the warps before it.
//
// A row is read once; its ranks stay in registers, up to KPT per thread (0: rows too long
// for that are read again in every pass).  Long rows, and few rows, are spread over a
// cluster of CTAs that add their histograms up in the first one's shared memory.
#include <cooperative_groups.h>

#include "evict.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkd {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32, kSelBins = 2048;
constexpr int kSelMaxKpt = 32, kSelMaxCluster = 8;
constexpr uint32_t kRankZero = 0x80000000u, kRankKept = 0xffffffffu;

// The rank of a weight: rises with it, NaN as -inf, -0 as +0, below that of a protected key.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return x != x ? 0x007fffffu : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

struct SelectShared {
    int hist[kSelBins];
    int warp_sum[kSelWarps], above[kSelWarps], on[kSelWarps];
    int found[3];                           // the threshold's bin, keys still missing in it, its count
    int cta_above[kSelMaxCluster], cta_on[kSelMaxCluster];
};

template <int KPT, bool kCluster>
__global__ void __launch_bounds__(kSelThreads, KPT <= 16 ? 2 : 1) evict_select_kernel(const SelectParams p) {
    __shared__ SelectShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int rank = 0, ctas = 1;
    if constexpr (kCluster) {
        rank = static_cast<int>(cg::this_cluster().block_rank());
        ctas = static_cast<int>(cg::this_cluster().num_blocks());
    }
    const int h = blockIdx.x / ctas, b = blockIdx.y, all = ctas * kSelThreads, me = rank * kSelThreads + tid;
    const int L = min(max(p.seq_lens[b], 0), p.keys), n = min(L, p.budget);
    int32_t* kept = p.kept + (static_cast<long long>(b) * p.H + h) * p.budget;
    if (h == 0 && me == 0) p.kept_lens[b] = n;
    for (int i = n + me; i < p.budget; i += all) kept[i] = -1;
    if (L <= p.budget) {
        for (int i = me; i < n; i += all) kept[i] = i;
        return;
    }
    const float* w = p.weights + b * p.weights_b + h * p.weights_h;
    const int32_t* pos = p.positions ? p.positions + b * p.positions_b + h * p.positions_h : nullptr;
    const int context = pos ? max(p.context_lens[b], 0) : L;
    const int first = p.sinks, past = context - p.recent, side = p.pool / 2;

    // the warp's run of keys: chunks of 32 from t0 on
    const int chunks = (L + 32 * kSelWarps * ctas - 1) / (32 * kSelWarps * ctas);
    const int t0 = (rank * kSelWarps + warp) * 32 * chunks + lane;
    auto rank_at = [&](int i) -> uint32_t {
        const int t = t0 + 32 * i;
        if (i >= chunks || t >= L) return 0;  // no key
        const int at = pos ? pos[t] : t;
        float x = w[t];
        if (at < first || at >= past) return kRankKept;
        if (side) {
            const int z = min(t + side, past - 1);
            for (int s = max(t - side, first); s <= z; ++s) x = fmaxf(x, w[s]);  // (a NaN beside a number counts not)
        }
        return rank_of(x);
    };
    constexpr bool kKept = KPT > 0;
    uint32_t r[kKept ? KPT : 1];
    if constexpr (kKept)
#pragma unroll
        for (int i = 0; i < KPT; ++i) r[i] = rank_at(i);
    // f(rank of the lane's key, its index), chunk by chunk
    auto each = [&](auto f) {
        if constexpr (kKept) {
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                if (i >= chunks) break;
                f(r[i], t0 + 32 * i);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < chunks; ++i) f(rank_at(i), t0 + 32 * i);
        }
    };

    // ------------------------------------------------------ the threshold
    uint32_t prefix = 0;
    int missing = n, shift = 32;
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
        const int bits = round < 2 ? 11 : 10, bins = 1 << bits;
        const int up = shift;  // bits below the prefix
        shift -= bits;
        for (int i = tid; i < bins; i += kSelThreads) sh.hist[i] = 0;
        if constexpr (kCluster) cg::this_cluster().sync(); else __syncthreads();
        int zeros = 0;
        each([&](uint32_t x, int) {
            const bool in = x != 0 && (round == 0 || (x >> (up & 31)) == prefix), zero = in && x == kRankZero;
            zeros += __popc(__ballot_sync(kFull, zero));
            if (in && !zero) atomicAdd(&sh.hist[(x >> shift) & (bins - 1)], 1);
        });
        if (lane == 0 && zeros) atomicAdd(&sh.hist[(kRankZero >> shift) & (bins - 1)], zeros);
        if constexpr (kCluster) {
            // the counts of all CTAs, in the first one's
            __syncthreads();
            int* total = cg::this_cluster().map_shared_rank(sh.hist, 0);
            if (rank)
                for (int i = tid; i < bins; i += kSelThreads)
                    if (sh.hist[i]) atomicAdd(total + i, sh.hist[i]);
            cg::this_cluster().sync();
        } else {
            __syncthreads();
        }
        if (rank == 0) {
            // from the top: a thread takes `per` bins, the highest first
            const int per = bins / kSelThreads;
            int c[4], mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[e] = e < per ? sh.hist[bins - 1 - (tid * per + e)] : 0;
                mine += c[e];
            }
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, sum, o);
                if (lane >= o) sum += y;
            }
            if (lane == 31) sh.warp_sum[warp] = sum;
            __syncthreads();
            int before = sum - mine;
#pragma unroll
            for (int k = 0; k < kSelWarps; ++k)
                if (k < warp) before += sh.warp_sum[k];
            // the bin in which the count reaches `missing`
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (before < missing && before + c[e] >= missing) {
                    int found[3] = {bins - 1 - (tid * per + e), missing - before, c[e]};
                    for (int k = 0; k < ctas; ++k) {
                        int* dst = sh.found;
                        if constexpr (kCluster) dst = cg::this_cluster().map_shared_rank(sh.found, k);
                        dst[0] = found[0];
                        dst[1] = found[1];
                        dst[2] = found[2];
                    }
                }
                before += c[e];
            }
        }
        if constexpr (kCluster) cg::this_cluster().sync(); else __syncthreads();
        prefix = prefix << bits | static_cast<uint32_t>(sh.found[0]);
        missing = sh.found[1];
        if (missing == sh.found[2]) break;  // all keys of the bin stay
    }

    // ------------------------------ those above it, and the first on it
    int na = 0, no = 0;
    each([&](uint32_t x, int) {
        na += __popc(__ballot_sync(kFull, x >> shift > prefix));
        no += __popc(__ballot_sync(kFull, x != 0 && x >> shift == prefix));
    });
    if (lane == 0) sh.above[warp] = na, sh.on[warp] = no;
    __syncthreads();
    int ta = 0, to = 0, sa = 0, so = 0;  // of the warps before, of the CTA
#pragma unroll
    for (int k = 0; k < kSelWarps; ++k) {
        if (k == warp) ta = sa, to = so;
        sa += sh.above[k];
        so += sh.on[k];
    }
    if constexpr (kCluster) {
        if (tid < ctas) {
            cg::this_cluster().map_shared_rank(sh.cta_above, tid)[rank] = sa;
            cg::this_cluster().map_shared_rank(sh.cta_on, tid)[rank] = so;
        }
        cg::this_cluster().sync();
        for (int k = 0; k < rank; ++k) ta += sh.cta_above[k], to += sh.cta_on[k];
    }
    const unsigned below = (1u << lane) - 1;
    each([&](uint32_t x, int t) {
        const bool over = x >> shift > prefix, at = x != 0 && x >> shift == prefix;
        const unsigned va = __ballot_sync(kFull, over), vo = __ballot_sync(kFull, at);
        const int a = ta + __popc(va & below), o = to + __popc(vo & below);
        if (over || (at && o < missing)) kept[a + min(o, missing)] = t;
        ta += __popc(va);
        to += __popc(vo);
    });
}

template <int KPT>
static cudaError_t launch_kpt(const SelectParams& p, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.H * cluster, p.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cluster > 1 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<KPT, true>, p)
                       : cudaLaunchKernelEx(&cfg, evict_select_kernel<KPT, false>, p);
}

cudaError_t launch_evict_select(const SelectParams& p, cudaStream_t stream) {
    // CTAs of a row: as many as its ranks need registers, and while SMs are idle and a thread
    // has more than eight keys
    const long long rows = static_cast<long long>(p.B) * p.H;
    int cluster = 1;
    while (cluster < kSelMaxCluster &&
           (p.keys > cluster * kSelThreads * kSelMaxKpt || (rows * cluster < 152 && p.keys > cluster * kSelThreads * 8)))
        cluster *= 2;
    const int kpt = (p.keys + cluster * kSelThreads - 1) / (cluster * kSelThreads);
    if (kpt <= 4) return launch_kpt<4>(p, cluster, stream);
    if (kpt <= 8) return launch_kpt<8>(p, cluster, stream);
    if (kpt <= 16) return launch_kpt<16>(p, cluster, stream);
    if (kpt <= 32) return launch_kpt<32>(p, cluster, stream);
    return launch_kpt<0>(p, cluster, stream);
}

}  // namespace pkd
