// Ragged paged attention for steps of a few tokens: requests whose query rows
// (tokens x heads of a kv head) are at most 16, with capped scores, a distance
// bias and interval masks.
//
// The decode grid's structure with the score modifications in the softmax: one
// CTA of four warps per (Split-KV chunk, kv head, request), each warp streaming
// 16-key stages through its own ring of TMA copies, products on mma.sync
// (the rows are too few for a tcgen05 tile), partial results merged by LSE by
// the last chunk to arrive.  Memory bound: every visible key is read once.
// A lane holds two of the (at most 16) rows: their intervals, positions and slopes
// stay in registers; a stage inside every row's interval skips the mask.
//
// 64 requests, 145k keys x 8 kv heads in bf16, capped: 94 us, 0.94 of the copy
// bandwidth.  4 requests, 309k keys x 8 kv heads in e4m3 with a bias: 117 us, 0.80: there
// a key is half the bytes and the same conversions and biases, and the ALU pipe is 49%
// busy.  One request of 611 keys: 9 us, a chain of start-up loads, stages and join.
#pragma once

#include "attend.cuh"
#include "fp8_warp.cuh"
#include "mma_warp.cuh"

namespace pkd {

constexpr int kStepRows = 16;

template <class W, int D, int ELT, int NBUF>
struct StepShape {
    static constexpr int KBOX = D * ELT / 128;
    static constexpr int HALF = KBOX * 2048;
    static constexpr int STAGE = 2 * HALF;
    static constexpr int QSTRIDE = D * 2 + 16;
    static constexpr int OSTRIDE = D + 4;
    static constexpr int RING = kNW * NBUF * STAGE;
    static constexpr int MERGE = kNW * kStepRows * OSTRIDE * 4;
    static constexpr int BIG = RING > MERGE ? RING : MERGE;
    static constexpr int OFF_BARS = BIG;
    static constexpr int OFF_PAGES = OFF_BARS + kNW * NBUF * 8;
    static constexpr int OFF_Q = OFF_PAGES + kMaxCtaPages * 4 + 16;
    static constexpr int OFF_ML = OFF_Q + (W::kCtaQ ? kStepRows * QSTRIDE : 0);
    static constexpr int OFF_FLAG = OFF_ML + 2 * kNW * kStepRows * 4;
    static constexpr int SMEM = OFF_FLAG + 16 + 1024;
};

// q row r = i * G + g of a request: token q0 + i, head hk * G + g.
template <int ELT, int D>
__device__ __forceinline__ const uint8_t* step_q_row(const AttendParams& a, int q0, int hk, int r) {
    const int i = r / a.G, g = r - i * a.G;
    return static_cast<const uint8_t*>(a.q) +
           ELT * (static_cast<long long>(q0 + i) * a.q_stride + static_cast<long long>(hk * a.G + g) * D);
}

template <class W, int D, int ELT, int NBUF>
__device__ __forceinline__ void attend_step(const CUtensorMap& tmap, const AttendParams& a, const DecodeParams& d) {
    using S = StepShape<W, D, ELT, NBUF>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BARS);
    int* pages = reinterpret_cast<int*>(smem + S::OFF_PAGES);
    uint8_t* qs = smem + S::OFF_Q;
    float* wm = reinterpret_cast<float*>(smem + S::OFF_ML);
    float* wl = wm + kNW * kStepRows;
    int* flag = reinterpret_cast<int*>(smem + S::OFF_FLAG);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- the request's rows and the interval of keys that some row sees
    CtaWork w;
    w.split = blockIdx.x;
    w.hk = blockIdx.y;
    w.b = blockIdx.z;
    const bool first = blockIdx.x == 0 && blockIdx.y == 0;
    int q0, n;
    request_tokens(a, w.b, q0, n, tid == 0 && first);
    if (n == 0) return;
    const int L = request_len(a, w.b, tid == 0 && first);
    const int prefix = a.prefix_lens ? a.prefix_lens[w.b] : 0;
    w.L = L;
    const int M = n * a.G;
    int lo_all = 0x7fffffff, hi_all = 0, lo_in = 0, hi_in = 0x7fffffff;  // union and intersection of the rows' intervals
    for (int i = 0; i < n; ++i) {
        int lo, hi;
        token_keys(a, q0, n, L, prefix, i, lo, hi);
        if (lo < hi) {
            lo_all = min(lo_all, lo);
            hi_all = max(hi_all, hi);
        }
        lo_in = max(lo_in, lo);
        hi_in = min(hi_in, hi);
    }
    const int begin = lo_all & ~(kStageTok - 1);  // stages start on 16-key boundaries of the request
    w.nsplit = hi_all > 0 ? (hi_all - begin + a.chunk - 1) / a.chunk : 0;
    if (w.split >= max(w.nsplit, 1)) return;

    if (w.nsplit == 0) {
        for (int e = tid; e < M * D; e += blockDim.x) {
            const int r = e / D, i = r / a.G;
            const long long row = static_cast<long long>(q0 + i) * a.Hq + w.hk * a.G + (r - i * a.G);
            store_out(d.out, row * D + e % D, 0.f, d.out_dtype);
            if (e % D == 0 && d.lse) d.lse[row] = -INFINITY;
        }
        return;
    }
    const DecodeParams& p = d;  // the stage helpers' parameters
    w.t0 = begin + w.split * a.chunk;
    w.t1 = min(w.t0 + a.chunk, hi_all);
    // this lane's rows g and g + 8
    const int g = lane >> 2, tg = lane & 3;
    int row_lo[2], row_hi[2], row_pos[2];
    float row_slope[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 8 * h + g, i = r / a.G;
        row_lo[h] = row_hi[h] = row_pos[h] = 0;
        row_slope[h] = 0.f;
        if (r < M) {
            token_keys(a, q0, n, L, prefix, i, row_lo[h], row_hi[h]);
            row_pos[h] = L - n + i - 2 * tg;  // less the lane's first key of a stage
            if (a.slopes) row_slope[h] = a.slopes[w.hk * a.G + (r - i * a.G)] * kLog2e;
        }
    }

    const int nst = (w.t1 - w.t0 + kStageTok - 1) / kStageTok;
    const int my_n = nst > warp ? (nst - warp + kNW - 1) / kNW : 0;
    uint8_t* ring_gen = smem + warp * NBUF * S::STAGE;
    const uint32_t ring = smem_u32(ring_gen);
    const uint32_t bar0 = smem_u32(bars + warp * NBUF);
    const uint64_t pol = policy_evict_first();
    if (lane == 0) {
        // the warp's own barriers, and its first copies ahead of the page list
        if (warp == 0) prefetch_tmap(&tmap);
        for (int k = 0; k < NBUF; ++k) mbar_init(bar0 + 8 * k, 1);
        fence_barrier_init();
        for (int k = 0; k < NBUF && k < my_n; ++k) {
            const int tok = w.t0 + (warp + k * kNW) * kStageTok;
            const int pg = p.block_table[static_cast<long long>(w.b) * p.bt_stride + page_col(p, tok)];
            const uint32_t bar = bar0 + 8 * k;
            if (pg < 0 || pg >= p.num_pages) {  // skipped; reported when the page list is built
                mbar_arrive(bar);
                continue;
            }
            mbar_arrive_expect_tx(bar, S::STAGE);
            tma_load_3d(ring + k * S::STAGE, &tmap, 0, (pg * p.Hkv + w.hk) * p.P + page_slot(p, tok), 0, bar, pol);
        }
    }
    load_cta_pages(p, w, pages);
    if constexpr (W::kCtaQ) {
        constexpr int VPR = D * 2 / 16;
        for (int e = tid; e < kStepRows * VPR; e += blockDim.x) {
            const int r = e / VPR, v = e % VPR;
            uint4 val = make_uint4(0u, 0u, 0u, 0u);
            if (r < M) val = __ldg(reinterpret_cast<const uint4*>(step_q_row<2, D>(a, q0, w.hk, r)) + v);
            *reinterpret_cast<uint4*>(qs + r * S::QSTRIDE + v * 16) = val;
        }
    }
    __syncthreads();

    W wp;
    if constexpr (W::kCtaQ) {
        wp.load_q(smem_u32(qs), S::QSTRIDE, lane);
    } else {
        // e4m3 A fragments straight from global memory (zero padding rows)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h * 8 + g;
            const uint32_t* row = r < M ? reinterpret_cast<const uint32_t*>(step_q_row<1, D>(a, q0, w.hk, r)) : nullptr;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                wp.q8[0][kk][h] = row ? __ldg(row + kk * 8 + tg) : 0u;
                wp.q8[0][kk][2 + h] = row ? __ldg(row + kk * 8 + 4 + tg) : 0u;
            }
        }
    }
    wp.reset();

    const float scale2 = a.scale_log2, cap_in = a.cap_in, cap_log2 = a.cap_log2;
    const bool bias = a.slopes != nullptr;
    int timed_out = 0, consumed = 0;
    for (int k = 0; k < my_n; ++k) {
        const int buf = k % NBUF;
        // one answer for the warp: its lanes go on, or give up, together
        if (!__all_sync(kFull, mbar_wait(bar0 + 8 * buf, (k / NBUF) & 1, p.status, p.wait_ns))) {
            timed_out = 1;
            break;
        }
        consumed = k + 1;
        const int tok0 = w.t0 + (warp + k * kNW) * kStageTok;
        int nvalid = min(kStageTok, w.t1 - tok0);
        if (page_of(p, w, pages, tok0) < 0) nvalid = 0;
        const uint32_t st = ring + buf * S::STAGE;
        uint8_t* st_gen = ring_gen + buf * S::STAGE;
        if (nvalid < kStageTok) zero_tail_v<D, ELT>(st_gen, nvalid, lane);
        if (tok0 < lo_all) {
            // V rows before every row's interval: stored values that no row may meet
            const int head = lo_all - tok0;
            for (int c = lane; c < head * S::KBOX * 8; c += 32) {
                const int row = c / (S::KBOX * 8), rem = c % (S::KBOX * 8);
                *reinterpret_cast<uint4*>(st_gen + S::HALF + (rem >> 3) * 2048 + row * 128 + (rem & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            __syncwarp();
        }
        const bool masked = nvalid < kStageTok || tok0 < lo_in || tok0 + kStageTok > hi_in;
        // the distance of the lane's first key of the stage; the others lie constants behind it
        float dist[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) dist[h] = bias ? static_cast<float>(row_pos[h] - tok0) : 0.f;
        wp.consume_scored(
            st, S::HALF, nvalid, masked,
            [&](float qk, int, int h, int kt) {
                float s = cap_log2 > 0.f ? capped(qk, cap_in, cap_log2) : qk * scale2;
                if (bias) s = fmaf(-row_slope[h], fabsf(dist[h] - static_cast<float>(kt - 2 * tg)), s);
                return s;
            },
            [&](int row, int kt) {
                const int h = row >> 3;
                return tok0 + kt >= (h ? row_lo[1] : row_lo[0]) && tok0 + kt < (h ? row_hi[1] : row_hi[0]);
            },
            lane);
        __syncwarp();
        if (lane == 0 && k + NBUF < my_n) {
            fence_proxy_async();
            issue_stage<D, ELT>(&tmap, p, w, pages, warp + (k + NBUF) * kNW, st, bar0 + 8 * buf, pol);
        }
    }
    if (timed_out) {
        // let this warp's copies land before the CTA leaves or reuses the ring
        if (lane == 0) raise_status(p, kErrTimeout);
        for (int k = consumed; k < my_n && k < consumed + NBUF; ++k)
            mbar_wait(bar0 + 8 * (k % NBUF), (k / NBUF) & 1);
    }

    wp.reduce_l();
    __syncthreads();
    float* O = reinterpret_cast<float*>(smem);
    wp.store(O + warp * kStepRows * S::OSTRIDE, wm + warp * kStepRows, wl + warp * kStepRows, S::OSTRIDE, lane);
    __syncthreads();

    // ---- a warp per row: the warps' states joined, then written, or left as a partial
    // result that the last chunk's CTA to arrive merges by LSE
    constexpr int E = D / 32;
    const bool single = w.nsplit == 1;
    const long long slots = (static_cast<long long>(w.b) * a.Hkv + w.hk) * a.max_splits * d.M;  // [split][row] of the unit
    auto out_row = [&](int r) {
        const int i = r / a.G;
        return static_cast<long long>(q0 + i) * a.Hq + w.hk * a.G + (r - i * a.G);
    };
    for (int r = warp; r < M; r += kNW) {
        float mx = -INFINITY, lsum = 0.f, o[E];
#pragma unroll
        for (int k = 0; k < kNW; ++k) mx = fmaxf(mx, wm[k * kStepRows + r]);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        if (mx != -INFINITY) {
#pragma unroll
            for (int k = 0; k < kNW; ++k) {
                const float s = fast_exp2(wm[k * kStepRows + r] - mx);
                lsum += wl[k * kStepRows + r] * s;
                const float* src = O + (k * kStepRows + r) * S::OSTRIDE + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(src[e], s, o[e]);
            }
        }
        const float inv = lsum > 0.f ? 1.f / lsum : 0.f, l2 = lsum > 0.f ? mx + __log2f(lsum) : -INFINITY;
        if (single) {
            store_row<D>(d.out, out_row(r), o, inv * a.v_scale, lane, d.out_dtype);
            if (lane == 0 && d.lse) d.lse[out_row(r)] = l2 * kLn2;
        } else {
            const long long slot = slots + static_cast<long long>(w.split) * d.M + r;
#pragma unroll
            for (int e = 0; e < E; ++e) __stcg(d.part_out + slot * D + lane * E + e, o[e] * inv);
            if (lane == 0) __stcg(d.part_lse + slot, l2);
        }
    }
    if (single) return;
    __syncthreads();
    const long long unit = static_cast<long long>(w.b) * a.Hkv + w.hk;
    if (tid == 0) {
        const int last = atom_add_acq_rel_gpu(a.counters + unit) == w.nsplit - 1;
        if (last) a.counters[unit] = 0;  // every part has arrived: ready for the next call
        *flag = last;
    }
    __syncthreads();
    if (!*flag) return;
    for (int r = warp; r < M; r += kNW) {
        float acc[E], mx, ws;
        merge_row<D>(d.part_lse + slots + r, d.part_out + (slots + r) * D, d.M, w.nsplit, lane, acc, mx, ws);
        store_row<D>(d.out, out_row(r), acc, ws > 0.f ? a.v_scale / ws : 0.f, lane, d.out_dtype);
        if (lane == 0 && d.lse) d.lse[out_row(r)] = ws > 0.f ? (mx + __log2f(ws)) * kLn2 : -INFINITY;
    }
}

// kMin: CTAs per SM that the register budget aims for
template <class W, int D, int ELT, int NBUF, int kMin>
__global__ void __launch_bounds__(kNW * 32, kMin)
attend_step_kernel(const __grid_constant__ CUtensorMap tmap, const AttendParams a, const DecodeParams d) {
    launch_dependents();
    attend_step<W, D, ELT, NBUF>(tmap, a, d);
    wait_dependency();  // its own end implies that of the launch it overlaps
}

}  // namespace pkd
