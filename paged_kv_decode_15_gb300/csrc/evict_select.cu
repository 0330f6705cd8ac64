// pkd_evict_select: which keys of each (request, kv head) stay.
//
// A key's rank is a 32-bit number that rises with its (pooled) weight; protected keys
// have the largest.  The n-th largest rank is found by three histograms, of its upper
// 11 bits, then, among the keys that share those of the threshold, of the next 11 and of
// the last 10 (fewer where a histogram ends on a bin of which all keys stay): counts
// in shared memory by integer atomics, whose order changes nothing, and a scan from the
// top.  Keys without any weight, often a third of them, are counted apart, by thread.  Then
// the keys above the threshold, and as many of those on it as are still missing, the
// lowest indexes first, are written in the order of the keys: a thread owns consecutive
// keys, counts, and writes behind the threads before it.
//
// A row is read once, through shared memory (whose words are spread so that threads KPT
// keys apart seldom meet in a bank), where the neighbours of a pooled weight are too; ranks
// stay in registers, up to KPT per thread (0: rows too long for that are read again in every
// pass).  Long rows, and few rows, are spread over a cluster of CTAs that add their
// histograms up in the first one's shared memory.
//
// What bounds it (512 rows of 1024 to 4096 keys, pooled over 7: 16.4 us; 32 rows of up to
// 131072 keys, clusters of eight: 26.5 us, one such row 23; eight rows of 1088 keys: 7.0 us;
// bytes alone would take 1, 2, 0 and 0 us): instructions where there are many rows (issue slots
// 63 % active, 235 instructions to 32 keys: each of the two or three rounds walks all of a
// thread's ranks again), the chain of the rounds' scans and barriers where there are few.
// Three bits a round, counted in registers, took 124 and 567 us; pooled from global memory 18.4;
// three cluster barriers a round, not two, 27; ranks in shared memory, walked in rolled loops
// (the unrolled ones wait for their instructions), 17.9 and 24.4.
#include <cooperative_groups.h>

#include <type_traits>

#include "evict.cuh"
#include "launch.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pkd {

constexpr int kSelBins = 2048, kSelMaxCluster = 8;
constexpr int kSelMaxSide = 127;  // neighbours to either side of a pooled weight
constexpr uint32_t kRankZero = 0x80000000u, kRankKept = 0xffffffffu;

// The rank of a weight: rises with it, NaN as -inf, -0 as +0, below that of a protected key.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return x != x ? 0x007fffffu : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

struct SelectShared {
    int hist[2][kSelBins];                  // of this round, of the next
    int warp_sum[16], above[16], on[16];
    int found[3];                           // the threshold's bin, keys still missing in it, its count
    int cta_above[kSelMaxCluster], cta_on[kSelMaxCluster];
};

// Threads x KPT keys of a CTA; 1024 threads' worth of CTAs fit an SM at least.
template <int kSelThreads, int KPT, bool kCluster>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) evict_select_kernel(const SelectParams p) {
    constexpr int kSelWarps = kSelThreads / 32, kPer = kSelBins / kSelThreads;
    __shared__ SelectShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int rank = 0, ctas = 1;
    if constexpr (kCluster) {
        rank = static_cast<int>(cg::this_cluster().block_rank());
        ctas = static_cast<int>(cg::this_cluster().num_blocks());
    }
    const int h = blockIdx.x / ctas, b = blockIdx.y, all = ctas * kSelThreads, me = rank * kSelThreads + tid;
    const int given = p.seq_lens[b], L = min(max(given, 0), p.keys), n = min(L, p.budget);
    int32_t* kept = p.kept + (static_cast<long long>(b) * p.H + h) * p.budget;
    if (h == 0 && me == 0) {
        p.kept_lens[b] = n;
        if (p.status && L != given) atomicOr(p.status, kErrBounds);
    }
    for (int i = n + me; i < p.budget; i += all) kept[i] = -1;
    if (L <= p.budget) {
        for (int i = me; i < n; i += all) kept[i] = i;
        return;
    }
    const float* w = p.weights + b * p.weights_b + h * p.weights_h;
    const int32_t* pos = p.positions ? p.positions + b * p.positions_b + h * p.positions_h : nullptr;
    const int context = pos ? max(p.context_lens[b], 0) : L;
    const int first = p.sinks, past = context - p.recent, side = p.pool / 2;

    // the thread's keys: `own` from t0 on
    const int own = (L + all - 1) / all, t0 = me * own;
    auto masked = [&](int t) { return t >= first && t < past && t < L ? w[t] : -INFINITY; };
    constexpr bool kKept = KPT > 0;
    uint32_t r[kKept ? KPT : 1];
    auto rank_at = [&](int t) -> uint32_t {  // (rows that are read again)
        if (t >= L) return 0;  // no key
        const int at = pos ? pos[t] : t;
        if (at < first || at >= past) return kRankKept;
        float x = w[t];
        for (int d = 1; d <= side; ++d) x = fmaxf(x, fmaxf(masked(max(t - d, 0)), masked(t + d)));
        return rank_of(x);
    };
    if constexpr (kKept) {
        extern __shared__ float stage[];
        const int c0 = rank * kSelThreads * own, span = kSelThreads * own + 2 * side;  // stage[0] is key c0 - side
        auto word = [](int i) { return i + i / 32; };
        if (pos) {
            for (int i0 = tid; i0 < span; i0 += 4 * kSelThreads) {
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = c0 + i0 + e * kSelThreads;
                    x[e] = 0;
                    if (i0 + e * kSelThreads < span && t < L) {
                        const int at = pos[t];
                        x[e] = at < first || at >= past ? kRankKept : rank_of(w[t]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i0 + e * kSelThreads < span) stage[word(i0 + e * kSelThreads)] = __uint_as_float(x[e]);
            }
        } else {
            // (asynchronous copies: all of a thread's weights in flight)
            for (int i = tid; i < span; i += kSelThreads) {
                const int t = c0 - side + i;
                if (t >= first && t < past && t < L)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(stage + word(i))), "l"(w + t) : "memory");
                else
                    stage[word(i)] = -INFINITY;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        __syncthreads();
        // the largest weight around each of the thread's keys (a NaN beside a number counts not)
        const int mine = tid * own + side;
        float x[KPT];
        auto window = [&](auto reach) {
            constexpr int kSide = decltype(reach)::value;
            float v[KPT + 2 * kSide];
#pragma unroll
            for (int i = 0; i < KPT + 2 * kSide; ++i) v[i] = i < own + 2 * kSide ? stage[word(mine - kSide + i)] : 0.f;
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                x[i] = v[i + kSide];
#pragma unroll
                for (int d = 1; d <= kSide; ++d) x[i] = max3(x[i], v[i + kSide - d], v[i + kSide + d]);
            }
        };
        // Windows of up to seven keys are in registers, unrolled for their reach; wider ones loop
        // over shared memory (512 rows of 1024 to 4096 keys: 3 keys 13.8 us, looped over 14.6; 7 keys
        // 14.9; 9 keys looped over 17.5, unrolled 15.1: every reach more is one more copy of this
        // pass in twelve kernels)
        switch (side) {
            case 0: window(std::integral_constant<int, 0>{}); break;
            case 1: window(std::integral_constant<int, 1>{}); break;
            case 2: window(std::integral_constant<int, 2>{}); break;
            case 3: window(std::integral_constant<int, 3>{}); break;
            default:
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    if (i >= own) break;
                    x[i] = stage[word(mine + i)];
                    for (int d = 1; d <= side; ++d) x[i] = max3(x[i], stage[word(mine + i - d)], stage[word(mine + i + d)]);
                }
        }
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int t = t0 + i;
            r[i] = 0;  // no key
            if (i >= own || t >= L) continue;
            if (pos)
                r[i] = __float_as_uint(x[i]);
            else
                r[i] = t < first || t >= past ? kRankKept : rank_of(x[i]);
        }
    }
    // f(rank of the thread's key, its index)
    auto each = [&](auto f) {
        if constexpr (kKept) {
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                if (i >= own) break;
                f(r[i], t0 + i);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < own; ++i) f(rank_at(t0 + i), t0 + i);
        }
    };

    // ------------------------------------------------------ the threshold
    // a thread of the scan reads `kPer` neighbouring bins: they lie a row apart, threads side by side
    auto place = [&](int bin) { return (bin % kPer) * kSelThreads + bin / kPer; };
    for (int i = tid; i < 2 * kSelBins; i += kSelThreads) sh.hist[0][i] = 0;
    if constexpr (kCluster) cg::this_cluster().sync(); else __syncthreads();
    uint32_t prefix = 0;
    int missing = n, shift = 32;
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
        const int bits = round < 2 ? 11 : 10, bins = 1 << bits;
        const int up = shift;  // bits below the prefix
        shift -= bits;
        int* hist = sh.hist[round & 1];
        if (round)  // read by the first CTA in the round before, wanted again in the next one
            for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[(round + 1) & 1][i] = 0;
        int zeros = 0;
        each([&](uint32_t x, int) {
            const bool in = x != 0 && (round == 0 || (x >> (up & 31)) == prefix), zero = in && x == kRankZero;
            zeros += zero;
            if (in && !zero) atomicAdd(&hist[place((x >> shift) & (bins - 1))], 1);
        });
        zeros = __reduce_add_sync(kFull, zeros);
        if (lane == 0 && zeros) atomicAdd(&hist[place((kRankZero >> shift) & (bins - 1))], zeros);
        if constexpr (kCluster) {
            // the counts of all CTAs, in the first one's
            __syncthreads();
            int* total = cg::this_cluster().map_shared_rank(hist, 0);
            if (rank)
                for (int i = tid; i < kSelBins; i += kSelThreads)
                    if (hist[i]) atomicAdd(total + i, hist[i]);
            cg::this_cluster().sync();
        } else {
            __syncthreads();
        }
        if (rank == 0) {
            // from the top: a thread takes kPer bins, the highest first (of the last round's
            // 1024 bins the upper half of the threads' are empty)
            const int top = kSelBins / kPer - 1 - tid;  // its row of bins
            int c[kPer], mine = 0;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                c[e] = hist[(kPer - 1 - e) * kSelThreads + top];
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
            for (int e = 0; e < kPer; ++e) {
                if (before < missing && before + c[e] >= missing) {
                    int found[3] = {top * kPer + kPer - 1 - e, missing - before, c[e]};
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
    int ta = 0, to = 0;  // of the thread, then of the threads before it
    each([&](uint32_t x, int) {
        ta += x >> shift > prefix;
        to += x != 0 && x >> shift == prefix;
    });
    {
        const int a = ta, o = to;
#pragma unroll
        for (int e = 1; e < 32; e <<= 1) {
            const int x = __shfl_up_sync(kFull, ta, e), y = __shfl_up_sync(kFull, to, e);
            if (lane >= e) ta += x, to += y;
        }
        if (lane == 31) sh.above[warp] = ta, sh.on[warp] = to;
        ta -= a;
        to -= o;
    }
    __syncthreads();
    int sa = 0, so = 0;  // of the CTA
#pragma unroll
    for (int k = 0; k < kSelWarps; ++k) {
        if (k == warp) ta += sa, to += so;
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
    each([&](uint32_t x, int t) {
        const bool over = x >> shift > prefix, at = x != 0 && x >> shift == prefix;
        if (over || (at && to < missing)) kept[ta + min(to, missing)] = t;
        ta += over;
        to += at;
    });
}

template <int T, int KPT>
static cudaError_t launch_one(const SelectParams& p, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.H * cluster, p.B);
    cfg.blockDim = dim3(T);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    // a CTA's keys and their neighbours, a word in 33 left free
    constexpr int kMost = KPT ? T * KPT + 2 * kSelMaxSide : 0;
    if constexpr (KPT > 0) cfg.dynamicSmemBytes = (kMost + kMost / 32 + 1) * sizeof(float);
    static PerDevice state, state_cluster;
    cudaError_t e = cluster > 1 ? kernel_setup(state_cluster, evict_select_kernel<T, KPT, true>, T, (int)cfg.dynamicSmemBytes)
                                : kernel_setup(state, evict_select_kernel<T, KPT, false>, T, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
    return cluster > 1 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<T, KPT, true>, p)
                       : cudaLaunchKernelEx(&cfg, evict_select_kernel<T, KPT, false>, p);
}

cudaError_t launch_evict_select(const SelectParams& p, cudaStream_t stream) {
    // CTAs of a row: as many as its ranks need registers, and while SMs are idle and a CTA
    // has more than 4096 keys
    const long long rows = static_cast<long long>(p.B) * p.H;
    int cluster = 1;
    while (cluster < kSelMaxCluster && (p.keys > cluster * 16384 || (rows * cluster < 152 && p.keys > cluster * 4096))) cluster *= 2;
    const int keys = (p.keys + cluster - 1) / cluster;
    if (keys <= 1024) return launch_one<256, 4>(p, cluster, stream);
    if (keys <= 2048) return launch_one<256, 8>(p, cluster, stream);
    if (keys <= 4096) return launch_one<256, 16>(p, cluster, stream);
    if (keys <= 8192) return launch_one<512, 16>(p, cluster, stream);
    if (keys <= 16384) return launch_one<512, 32>(p, cluster, stream);
    return launch_one<512, 0>(p, cluster, stream);
}

}  // namespace pkd
