// Ragged paged attention on the 5th-generation tensor cores: query blocks of
// any length against the paged cache, accumulators in tensor memory (TMEM).
//
// The query rows of one (request, kv head) are its tokens times the heads of the
// kv head, packed token-major: row i * G + g.  A work item is two tiles of up
// to 128 rows (TOK = 128 / G whole tokens each) against a range of keys, walked
// in tiles of 128 keys.  Per key tile and row tile:
//   S = Q K^T     tcgen05.mma, M = 128 rows, N = 128 keys: both operands in
//                 shared memory, K-major, 128-byte swizzle, as TMA lands them
//   softmax       one row per thread (TMEM lane = row): no shuffles.  The
//                 reference maximum moves only when a row's maximum grows by more
//                 than 2^8 (O and l are then rescaled by the row's own warp)
//   O += P V      P in TMEM over the spent S (A operand from tensor memory),
//                 V in shared memory read MN-major
// Two row tiles share every K/V tile, and while the softmax of one runs, the
// tensor cores work on the other's products: a key tile of both costs
// 2 x (S + O) = 4 products of 128x128xD against one softmax pass per tile.
//
// Warp roles (384 threads): warps 0-3 and 4-7 the softmax of tile 0 and 1 and, at an
// item's end, its epilogue (O out of TMEM, normalised, written -- or a partial
// result when the keys are split), warp 8 loads (work items, Q, K, V by TMA), warp
// 9 issues the products; for e4m3 caches S is an e4m3 product and warps 10-11 widen
// V to fp16 in shared memory ahead of the O product (P is rounded to fp16 then).
// Registers follow the roles (setmaxnreg).  (An epilogue group of its own left the
// softmax 176 registers and spills: 8192-token prompt 523 us.)
// Work items are handed out by an atomic counter in the workspace, the longest of
// a request first, so CTAs finish together whatever the lengths; results do not
// depend on who computes an item.  Every wait is bounded.
#pragma once

#include <type_traits>

#include "attend.cuh"
#include "tc05.cuh"

namespace pkd {

constexpr int kPtKeys = 128;       // keys per tile
constexpr int kPtRows = 128;       // rows per tile (TMEM lanes)
constexpr int kPtThreads = 384;
constexpr int kPtItems = 4;        // work-item ring
constexpr int kPtMaxBatch = 2048;  // requests whose tile prefix the CTA keeps in shared memory
constexpr int kPtL2Bytes = 64 << 20;  // keys and values walked together
// A row's reference moves when its maximum has grown by more than this (log2
// units).  The weights only must not overflow the operand type: bf16 has fp32's
// range, fp16 ends at 2^16.  (With 2^8 for both, half of the key tiles of scores
// with a spread of 3 made some warp repeat its pass.)
constexpr float kPtRescaleBF16 = 40.f, kPtRescaleFP16 = 14.f;

struct PtItem {
    int b, hk, q0, n, L, prefix;   // request, kv head, first query token, query tokens, length, prefix keys
    int tok0;                      // first token (of the request) of the item's rows
    int t0, t1, ntiles;            // keys of this item, tiles of 128 from t0
    int lo_all, hi_all;            // keys outside are seen by no row of the unit
    int split, nsplit, unit;
    int jb[2], je[2];              // key tiles [jb, je) of row tile t (empty: none)
    int bad, end;                  // bad: some page lies outside the pool
    int pad[2];
};

// Types of q and the cache.
enum PtType { kPtBF16 = 0, kPtFP16 = 1, kPtFP8 = 2 };

// NU K/V units; K and V of a key tile are one unit each (units of K have even
// numbers, NU is even, so a slot always holds the one or the other).  e4m3: the
// raw V units are widened to fp16 into two buffers of their own.
template <int D, int kType>
struct PtShape {
    static constexpr bool FP8 = kType == kPtFP8;
    static constexpr int ROWB = D * (FP8 ? 1 : 2);
    static constexpr int REGIONS = ROWB / 128;           // 128-byte regions of a row
    static constexpr int GROUP = 8 * ROWB;               // 8 keys: REGIONS regions of 8 x 128 bytes
    static constexpr int UNIT = kPtKeys / 8 * GROUP;     // 32 KB at D = 128, 16-bit
    static constexpr int NU = FP8 ? 6 : D == 128 ? 4 : 8;
    static constexpr int NV = FP8 ? 2 : 0;               // widened V tiles
    static constexpr int VGROUP = 8 * D * 2;             // 8 keys of V as the O product reads them
    static constexpr int VUNIT = kPtKeys / 8 * VGROUP;
    static constexpr int QTILE = kPtRows * ROWB;
    static constexpr int OFF_KV = 0;
    static constexpr int OFF_V = NU * UNIT;
    static constexpr int OFF_Q = OFF_V + NV * VUNIT;
    static_assert(NU % 2 == 0 && (!FP8 || D == 128), "unit parity; e4m3 rows are one region");
    static constexpr int OFF_STAGE = OFF_Q + 2 * QTILE;  // 2 KB per softmax warp: 64 bytes of 32 rows
    static constexpr int OFF_ITEM = OFF_STAGE + 8 * 2048;
    static constexpr int OFF_PREF = OFF_ITEM + kPtItems * static_cast<int>(sizeof(PtItem));
    static constexpr int OFF_SCAN = OFF_PREF + (kPtMaxBatch + 4) * 4;  // 16 warp sums, an arrival flag
    static constexpr int OFF_BAR = (OFF_SCAN + 128 + 7) & ~7;
    // units full/empty, Q full/empty, S full, P full, O step done, O full/drained, item full/empty, widened V, drain
    static constexpr int B_UF = 0, B_UE = B_UF + NU, B_QF = B_UE + NU, B_QE = B_QF + 1, B_SF = B_QE + 1;
    static constexpr int B_PF = B_SF + 2, B_OD = B_PF + 2, B_OF = B_OD + 2, B_OE = B_OF + 2, B_IF = B_OE + 2;
    static constexpr int B_IE = B_IF + kPtItems, B_VF = B_IE + kPtItems, B_VE = B_VF + NV, B_DR = B_VE + NV;
    static constexpr int NBAR = B_DR + 1;
    static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_TMEM + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
    static_assert(SMEM > 114 * 1024, "one CTA per SM: all 512 TMEM columns are its own");
};

// 16-key stages of the tile from key tk whose page lies in the pool (items with a bad page only).
__device__ __forceinline__ unsigned pt_stages(const AttendParams& p, const PtItem& I, int tk) {
    const int32_t* table = p.block_table + static_cast<long long>(I.b) * p.bt_stride;
    unsigned stages = 0;
#pragma unroll 1
    for (int s = 0; s < kPtKeys / kStageTok; ++s) {
        const int k = tk + kStageTok * s;
        const int pg = k < I.t1 ? table[page_div(k, p.pmagic, p.pmshift)] : -1;
        if (pg >= 0 && pg < p.num_pages) stages |= 1u << s;
    }
    return stages;
}

__device__ __forceinline__ bool pt_wait(uint32_t bar, uint32_t parity, const AttendParams& p) {
    return __all_sync(kFull, mbar_wait(bar, parity, p.status));
}

// a*b + c on two floats at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// What a softmax thread needs to turn its row's products into weights.
struct PtScore {
    float scale2, cap_in, cap_log2;
    float slope, base;   // bias: slope in log2 units; position - first key of the tile
    int c0, c1;          // keys [c0, c1) of the tile are seen
    unsigned stages;     // 16-key stages whose page is in the pool
};

template <bool kMasked>
__device__ __forceinline__ bool pt_seen(const PtScore& w, int k) {
    return !kMasked || (k >= w.c0 && k < w.c1 && (w.stages >> (k >> 4) & 1));
}

// The reference a row starts from: the largest logit among 32 keys.
template <bool kBias, bool kCap, bool kMasked>
__device__ __forceinline__ float pt_top(const uint32_t (&s)[32], int k0, const PtScore& w, float top) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float a = __uint_as_float(s[c]), b = __uint_as_float(s[c + 1]);
        if constexpr (kBias) {
            // (capped logits are below q.k scaled by as much as the reference may lie off,
            // so with a bias the cap counts)
            a = kCap ? capped(a, w.cap_in, w.cap_log2) : a * w.scale2;
            b = kCap ? capped(b, w.cap_in, w.cap_log2) : b * w.scale2;
            a = fmaf(-w.slope, fabsf(w.base - static_cast<float>(k0 + c)), a);
            b = fmaf(-w.slope, fabsf(w.base - static_cast<float>(k0 + c + 1)), b);
        }
        top = max3(top, pt_seen<kMasked>(w, k0 + c) ? a : -INFINITY, pt_seen<kMasked>(w, k0 + c + 1) ? b : -INFINITY);
    }
    return top;
}

// The weights 2^(x - m) of 32 keys (k0 .. k0 + 31 of the tile) from their
// products s, packed to the operand type, with their fp32 sum and the running
// maximum: of q.k (the logit rises with it), with a bias of x - m.
// Capped logits, kPoly: q.k times a polynomial in its square (cap_c), on packed
// FMAs; `far` keeps the largest |q.k|, and a tile beyond the polynomial's range is
// done again by exponential and reciprocal (capped(): three special-function
// results per key instead of one).
// A bias is linear in the key where no key lies behind its row's position
// (unmasked tiles); masked tiles take the distance's magnitude.
template <bool kBF16, bool kCap, bool kPoly, bool kBias, bool kMasked>
__device__ __forceinline__ void pt_weights(const uint32_t (&s)[32], uint32_t* pk, int k0, const PtScore& w,
                                           const float (&cc)[5], float m, float2 (&sum)[2], float& top, float& far) {
    const float nb = kBias ? -w.slope * w.base - m : 0.f;
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const int k = k0 + c;
        const float2 qk = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        float2 add = both(-m), x;  // what the scaled score needs to be the exponent
        if constexpr (kBias) {
            if constexpr (kMasked)
                add = make_float2(fmaf(-w.slope, fabsf(w.base - static_cast<float>(k)), -m),
                                  fmaf(-w.slope, fabsf(w.base - static_cast<float>(k + 1)), -m));
            else
                add = make_float2(fmaf(w.slope, static_cast<float>(k), nb), fmaf(w.slope, static_cast<float>(k + 1), nb));
        }
        if constexpr (kCap && kPoly) {
            const float2 z = mul2(qk, qk);
            float2 t = fma2(z, both(cc[4]), both(cc[3]));
            t = fma2(z, t, both(cc[2]));
            t = fma2(z, t, both(cc[1]));
            t = fma2(z, t, both(cc[0]));
            x = fma2(t, qk, add);
            far = max3(far, fabsf(qk.x), fabsf(qk.y));
        } else if constexpr (kCap) {
            x = add2(make_float2(capped(qk.x, w.cap_in, w.cap_log2), capped(qk.y, w.cap_in, w.cap_log2)), add);
        } else {
            x = fma2(qk, both(w.scale2), add);
        }
        if constexpr (kMasked) {
            x.x = pt_seen<kMasked>(w, k) ? x.x : -INFINITY;
            x.y = pt_seen<kMasked>(w, k + 1) ? x.y : -INFINITY;
        }
        if constexpr (kBias)
            top = max3(top, x.x, x.y);
        else if constexpr (kMasked)
            top = max3(top, pt_seen<kMasked>(w, k) ? qk.x : -INFINITY, pt_seen<kMasked>(w, k + 1) ? qk.y : -INFINITY);
        else
            top = max3(top, qk.x, qk.y);
        x.x = fast_exp2(x.x);
        x.y = fast_exp2(x.y);
        // l sums the fp32 weights; the product takes them rounded to the operand type
        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], x);
        pk[c >> 1] = pack2<kBF16>(x.x, x.y);
    }
}

template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Merge the partial results of one row by LSE (log2 units): a warp per row,
// lane l holds dims l * D/32 ...; parts s at part_lse[s * lse_step] and
// part_out[s * lse_step * D].  Partials come from other CTAs: L2 loads.
template <int D>
__device__ __forceinline__ void pt_merge_row(const float* pl, const float* po, long long step, int np, int lane,
                                             float (&acc)[D / 32], float& mx, float& ws) {
    constexpr int E = D / 32;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    mx = -INFINITY;
    ws = 0.f;
    for (int s = lane; s < np; s += 32) mx = fmaxf(mx, __ldcg(pl + s * step));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    if (mx == -INFINITY) return;
    for (int s0 = 0; s0 < np; s0 += 32) {
        const float l = s0 + lane < np ? __ldcg(pl + (s0 + lane) * step) : -INFINITY;
        const float wl = l == -INFINITY ? 0.f : fast_exp2(l - mx);
        ws += wl;
        const int m = min(32, np - s0);
#pragma unroll 4
        for (int j = 0; j < m; ++j) {
            const float w = __shfl_sync(kFull, wl, j);
            if (w == 0.f) continue;  // an empty part is never read
            const float* src = po + (s0 + j) * step * D + lane * E;
            if constexpr (E == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                acc[0] = fmaf(w, v.x, acc[0]);
                acc[1] = fmaf(w, v.y, acc[1]);
                acc[2] = fmaf(w, v.z, acc[2]);
                acc[3] = fmaf(w, v.w, acc[3]);
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                acc[0] = fmaf(w, v.x, acc[0]);
                acc[1] = fmaf(w, v.y, acc[1]);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kFull, ws, o);
}

// kPartials: every result is left as a partial one (for a merge that follows)
template <int D, int kType, bool kCap, bool kBias>
__global__ void __launch_bounds__(kPtThreads, 1)
attend_prompt_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                     const AttendParams p, const int partials) {
    using S = PtShape<D, kType>;
    constexpr bool kFp8 = kType == kPtFP8, kBF16 = kType == kPtBF16;  // e4m3: P and V in fp16
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb0 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    PtItem* items = reinterpret_cast<PtItem*>(smem + S::OFF_ITEM);
    int* pref = reinterpret_cast<int*>(smem + S::OFF_PREF);
    int* scan = reinterpret_cast<int*>(smem + S::OFF_SCAN);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::OFF_TMEM);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.G, TOK = kPtRows / G;  // whole tokens per row tile
    auto bar = [&](int i) { return smem_u32(bars + i); };

    // ------------------------------------------------------------ set-up
    if (tid == 0) {
        for (int i = 0; i < S::NU; ++i) {
            mbar_init(bar(S::B_UF + i), 1);
            mbar_init(bar(S::B_UE + i), kFp8 && (i & 1) ? 2 : 1);  // raw V: both widening warps
        }
        for (int i = 0; i < S::NV; ++i) {
            mbar_init(bar(S::B_VF + i), 2);
            mbar_init(bar(S::B_VE + i), 1);
        }
        mbar_init(bar(S::B_QF), 1);
        mbar_init(bar(S::B_QE), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(S::B_SF + i), 1);
            mbar_init(bar(S::B_PF + i), 4);
            mbar_init(bar(S::B_OD + i), 1);
            mbar_init(bar(S::B_OF + i), 1);
            mbar_init(bar(S::B_OE + i), 4);
        }
        for (int i = 0; i < kPtItems; ++i) {
            mbar_init(bar(S::B_IF + i), 1);
            mbar_init(bar(S::B_IE + i), 1 + 8 + (kFp8 ? 2 : 0));  // the issuing, softmax and widening warps
        }
        mbar_init(bar(S::B_DR), 1);
        fence_barrier_init();
    }
    if (warp == 9) {
        tc05::alloc(smem_u32(tslot), 512);  // S/P: columns 0-255, O: 256 + D * tile
        tc05::relinquish_alloc_permit();
    }
    // prefix of the requests' row-tile pairs (units of one kv head)
    {
        int run = 0;
        for (int b0 = 0; b0 < p.B; b0 += kPtThreads) {
            const int b = b0 + tid;
            int v = 0;
            if (b < p.B) {
                int q0, n;
                request_tokens(p, b, q0, n, blockIdx.x == 0);
                v = (n + 2 * TOK - 1) / (2 * TOK);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, v, o);
                if (lane >= o) v += y;
            }
            if (lane == 31) scan[warp] = v;
            __syncthreads();
            int before = run;
            for (int k = 0; k < kPtThreads / 32; ++k) {
                const int s = scan[k];
                if (k < warp) before += s;
                run += s;
            }
            if (b < p.B) pref[b + 1] = before + v;
            __syncthreads();
        }
        if (tid == 0) pref[0] = 0;
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = *tslot;
    constexpr uint32_t kIdS = kFp8 ? tc05::idesc_e4m3(kPtRows, kPtKeys)
                                   : tc05::idesc_f16(kBF16, kPtRows, kPtKeys, false, false);  // S = Q K^T
    constexpr uint32_t kIdO = tc05::idesc_f16(kBF16, kPtRows, D, false, true);         // O += P V

    if (warp >= 8) {
        reg_dec<88>();
        if (warp == 8) {
            // ------------------------------------------------------ loads
            if (lane == 0) {
                prefetch_tmap(&kvmap);
                prefetch_tmap(&qmap);
            }
            const uint64_t pol = policy_evict_first();
            uint64_t keep;
            asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
            const int total = pref[p.B] * p.Hkv * p.max_splits;
            int idx = blockIdx.x;
            int u = 0, nq = 0, npub = 0;
            bool ok = true;
            // Decode and publish the next item (or the end).  Called one item ahead, once
            // the ring is full of the current item's tiles, so that its chain of loads
            // (lengths, table) is hidden.
            auto publish = [&]() {
                for (;;) {
                    const int slot = npub % kPtItems;
                    if (idx >= total) {
                        if (npub >= kPtItems && !pt_wait(bar(S::B_IE + slot), ((npub / kPtItems) - 1) & 1, p)) return false;
                        if (lane == 0) {
                            items[slot].end = 1;
                            mbar_arrive(bar(S::B_IF + slot));
                        }
                        __syncwarp();
                        ++npub;
                        return true;
                    }
                    int next = 0;
                    if (lane == 0) next = static_cast<int>(gridDim.x) + atomicAdd(p.queue, 1);
                    // item idx: splits innermost; within a request groups of kv heads
                    // whose keys and values fit half of L2 together, in each the row tiles
                    // from the last (the longest, causal) to the first, all heads of the
                    // group per tile -- the short items come last
                    const int split = idx % p.max_splits, r1 = idx / p.max_splits;
                    int lo_b = 0, hi_b = p.B;
                    while (hi_b - lo_b > 1) {
                        const int mid = (lo_b + hi_b) >> 1;
                        if (static_cast<long long>(pref[mid]) * p.Hkv <= r1) lo_b = mid; else hi_b = mid;
                    }
                    const int b = lo_b, npair = pref[b + 1] - pref[b], r2 = r1 - pref[b] * p.Hkv;
                    int q0, n;
                    request_tokens(p, b, q0, n, false);
                    const int L = request_len(p, b, r2 == 0 && split == 0 && lane == 0);
                    const int prefix = p.prefix_lens ? p.prefix_lens[b] : 0;
                    const int group = max(1, min(p.Hkv, kPtL2Bytes / (2 * S::ROWB) / max(L, 1)));
                    const int g = r2 / (npair * group), width = min(group, p.Hkv - g * group), r3 = r2 - g * npair * group;
                    const int pair = npair - 1 - r3 / width, hk = g * group + r3 % width;
                    const int tok0 = pair * 2 * TOK;
                    int lo[2], hi[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int a0 = tok0 + t * TOK, a1 = min(a0 + TOK, n);
                        int l = 0x7fffffff, h = 0;
                        for (int i = a0 + lane; i < a1; i += 32) {
                            int x, y;
                            token_keys(p, q0, n, L, prefix, i, x, y);
                            if (x < y) {
                                l = min(l, x);
                                h = max(h, y);
                            }
                        }
                        lo[t] = __reduce_min_sync(kFull, l);
                        hi[t] = __reduce_max_sync(kFull, h);
                    }
                    const int lo_all = min(lo[0], lo[1]), hi_all = max(hi[0], hi[1]);
                    const int begin = lo_all & ~(kStageTok - 1);  // 16-key stages never cross a page
                    int nsplit = hi_all > 0 ? (hi_all - begin + p.chunk - 1) / p.chunk : 0;
                    if (nsplit > p.max_splits) {
                        if (lane == 0) atomicOr(p.status, kErrBounds);
                        nsplit = p.max_splits;
                    }
                    if (split >= max(nsplit, 1)) {  // nothing here
                        idx = __shfl_sync(kFull, next, 0);
                        continue;
                    }
                    const int t0 = nsplit ? begin + split * p.chunk : 0;
                    const int t1 = nsplit ? min(t0 + p.chunk, hi_all) : 0;
                    const int ntiles = (t1 - t0 + kPtKeys - 1) / kPtKeys;
                    // a page outside the pool anywhere in the item: the softmax checks its keys
                    const int32_t* row = p.block_table + static_cast<long long>(b) * p.bt_stride;
                    int bad = 0;
                    if (ntiles) {
                        const int c1 = page_div(t1 - 1, p.pmagic, p.pmshift);
                        for (int c = page_div(t0, p.pmagic, p.pmshift) + lane; c <= c1; c += 32)
                            bad |= row[c] < 0 || row[c] >= p.num_pages;
                        bad = __any_sync(kFull, bad);
                        if (bad && lane == 0) atomicOr(p.status, kErrBounds);
                    }
                    if (npub >= kPtItems && !pt_wait(bar(S::B_IE + slot), ((npub / kPtItems) - 1) & 1, p)) return false;
                    if (lane == 0) {
                        PtItem& I = items[slot];
                        I.b = b; I.hk = hk; I.q0 = q0; I.n = n; I.L = L; I.prefix = prefix; I.tok0 = tok0;
                        I.t0 = t0; I.t1 = t1; I.ntiles = ntiles; I.lo_all = lo_all; I.hi_all = hi_all;
                        I.split = split; I.nsplit = nsplit; I.unit = (pref[b] + pair) * p.Hkv + hk;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int a = max(lo[t], t0), z = min(hi[t], t1);
                            I.jb[t] = a < z ? (a - t0) / kPtKeys : 0;
                            I.je[t] = a < z ? (z - t0 + kPtKeys - 1) / kPtKeys : 0;
                        }
                        I.bad = bad; I.end = 0;
                        mbar_arrive(bar(S::B_IF + slot));
                    }
                    __syncwarp();
                    ++npub;
                    idx = __shfl_sync(kFull, next, 0);
                    return true;
                }
            };
            ok = publish();
            for (int it = 0; ok; ++it) {
                // the item's slot is not reused before this warp publishes four items on
                const PtItem& I = items[it % kPtItems];
                if (I.end) break;
                const int hk = I.hk, t0 = I.t0, t1 = I.t1, ntiles = I.ntiles;
                const int32_t* row = p.block_table + static_cast<long long>(I.b) * p.bt_stride;
                if (!ntiles) {
                    ok = publish();
                    continue;
                }
                // Q of the item's tiles (128-byte regions), once the last item's products have read theirs
                if (nq >= 1 && !pt_wait(bar(S::B_QE), (nq - 1) & 1, p)) { ok = false; break; }
                if (lane == 0) {
                    const int tiles = I.tok0 + TOK < I.n ? 2 : 1;
                    mbar_arrive_expect_tx(bar(S::B_QF), tiles * S::REGIONS * TOK * G * 128);
                    for (int t = 0; t < tiles; ++t)
                        for (int h = 0; h < S::REGIONS; ++h)
                            tma_load_3d(sb0 + S::OFF_Q + t * S::QTILE + h * kPtRows * 128, &qmap, 64 * h, hk * G,
                                        I.q0 + I.tok0 + t * TOK, bar(S::B_QF), pol);
                }
                __syncwarp();
                ++nq;
                auto entry = [&](int j) {
                    const int tok = t0 + j * kPtKeys + lane * kStageTok;
                    return lane < kPtKeys / kStageTok && tok < t1 ? row[page_div(tok, p.pmagic, p.pmshift)] : -1;
                };
                int pg = entry(0);
                const int ahead = min(ntiles, S::NU / 2) - 1;  // the ring is full behind this tile
                for (int j = 0; j < ntiles && ok; ++j) {
                    const int pg_next = j + 1 < ntiles ? entry(j + 1) : -1;
                    const int tok = t0 + j * kPtKeys + lane * kStageTok;
                    const bool load = pg >= 0 && pg < p.num_pages;
                    const int bytes = __popc(__ballot_sync(kFull, load)) * 2 * S::GROUP;
                    const int krow = load ? (pg * p.Hkv + hk) * p.P + (tok - page_div(tok, p.pmagic, p.pmshift) * p.P) : 0;
#pragma unroll 1
                    for (int v = 0; v < 2; ++v, ++u) {
                        const int us = u % S::NU;
                        if (u >= S::NU && !pt_wait(bar(S::B_UE + us), ((u / S::NU) - 1) & 1, p)) { ok = false; break; }
                        if (lane == 0) mbar_arrive_expect_tx(bar(S::B_UF + us), bytes);
                        __syncwarp();
                        if (load)
                            tma_load_4d(sb0 + S::OFF_KV + us * S::UNIT + 2 * lane * S::GROUP, &kvmap, 0, 0,
                                        v * S::REGIONS, krow >> 3, bar(S::B_UF + us), keep);
                    }
                    if (ok && j == ahead) ok = publish();
                    pg = pg_next;
                }
            }
            if (!ok) {
                // let every issued copy land before the CTA leaves
                if (lane == 0) atomicOr(p.status, kErrTimeout);
                for (int j = max(0, u - S::NU); j < u; ++j) mbar_wait(bar(S::B_UF + j % S::NU), (j / S::NU) & 1);
                if (nq) mbar_wait(bar(S::B_QF), (nq - 1) & 1);
            }
        } else if (warp == 9) {
            // --------------------------------------------------- products
            // The whole warp walks the items, converged, so that descriptors stay in
            // uniform registers; one elected lane issues (with the loop under a lane
            // test instead, a product took 115 cycles to issue, twice its run time).
            const bool one = tc05::elect_one();
            bool ok = true;
            int u = 0, nq = 0, nv = 0;  // nv: widened V tiles
            int np[2] = {0, 0}, no[2] = {0, 0};  // P tiles consumed, accumulations begun
            for (int it = 0; ok; ++it) {
                const int slot = it % kPtItems;
                if (!pt_wait(bar(S::B_IF + slot), (it / kPtItems) & 1, p)) { ok = false; break; }
                const PtItem& I = items[slot];
                if (I.end) break;
                const int ntiles = I.ntiles;
                const int jb[2] = {I.jb[0], I.jb[1]}, je[2] = {I.je[0], I.je[1]};
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::B_IE + slot));
                if (!ntiles) continue;
                if (!pt_wait(bar(S::B_QF), nq & 1, p)) { ok = false; break; }
                ++nq;
                auto k_ready = [&](int j) {
                    const int x = u + 2 * j;
                    return pt_wait(bar(S::B_UF + x % S::NU), (x / S::NU) & 1, p);
                };
                auto qk = [&](int t, int j) {
                    const uint64_t qd = tc05::smem_desc(sb0 + S::OFF_Q + t * S::QTILE, 16, 1024);
                    const uint64_t kd = tc05::smem_desc(sb0 + S::OFF_KV + ((u + 2 * j) % S::NU) * S::UNIT, 16, S::GROUP);
#pragma unroll
                    for (int kk = 0; kk < S::ROWB / 32; ++kk) {
                        const uint64_t qk_ = qd + (((kk >> 2) * kPtRows * 128 + (kk & 3) * 32) >> 4);
                        const uint64_t kk_ = kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4);
                        if (!one) continue;
                        if constexpr (kFp8)
                            tc05::mma_e4m3(tmem + kPtKeys * t, qk_, kk_, kIdS, kk > 0);
                        else
                            tc05::mma_f16(tmem + kPtKeys * t, qk_, kk_, kIdS, kk > 0);
                    }
                    if (one) tc05::commit(bar(S::B_SF + t));
                };
                ok = k_ready(0);
                tc05::fence_after_sync();
                for (int t = 0; ok && t < 2; ++t)
                    if (jb[t] == 0 && je[t] > 0) qk(t, 0);
                if (one) tc05::commit(bar(S::B_UE + u % S::NU));
                if (one && ntiles == 1) tc05::commit(bar(S::B_QE));
                for (int j = 0; ok && j < ntiles; ++j) {
                    const int vu = u + 2 * j + 1, vb = kFp8 ? (nv + j) % 2 : 0;
                    ok = kFp8 ? pt_wait(bar(S::B_VF + vb), ((nv + j) >> 1) & 1, p)
                              : pt_wait(bar(S::B_UF + vu % S::NU), (vu / S::NU) & 1, p);
                    const uint64_t vd = tc05::smem_desc(
                        sb0 + (kFp8 ? S::OFF_V + vb * S::VUNIT : S::OFF_KV + (vu % S::NU) * S::UNIT), 1024, S::VGROUP);
                    const uint32_t v_free = kFp8 ? bar(S::B_VE + vb) : bar(S::B_UE + vu % S::NU);
                    bool have_k = false;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok) break;
                        if (j >= jb[t] && j < je[t]) {
                            ok = pt_wait(bar(S::B_PF + t), np[t] & 1, p);
                            ++np[t];
                            if (ok && j == jb[t]) {
                                // a new accumulation: the epilogue has drained the last one
                                if (no[t] >= 1) ok = pt_wait(bar(S::B_OE + t), (no[t] - 1) & 1, p);
                                ++no[t];
                            }
                            if (!ok) break;
                            tc05::fence_after_sync();
                            const bool more = j > jb[t];
#pragma unroll
                            for (int kk = 0; kk < kPtKeys / 16; ++kk)
                                if (one)
                                    tc05::mma_f16_ts(tmem + 256 + D * t, tmem + kPtKeys * t + 8 * kk,
                                                     vd + ((2 * kk * S::VGROUP) >> 4), kIdO, more || kk > 0);
                            if (one) {
                                tc05::commit(bar(S::B_OD + t));
                                if (j == je[t] - 1) tc05::commit(bar(S::B_OF + t));
                            }
                        }
                        if (t == 1 && one) tc05::commit(v_free);
                        if (j + 1 < ntiles) {
                            if (!have_k) {
                                ok = k_ready(j + 1);
                                have_k = true;
                                if (!ok) break;
                                tc05::fence_after_sync();
                            }
                            // in issue order behind this tile's O product, which has read the P under S
                            if (j + 1 >= jb[t] && j + 1 < je[t]) qk(t, j + 1);
                            if (t == 1 && one) {
                                tc05::commit(bar(S::B_UE + (u + 2 * (j + 1)) % S::NU));
                                if (j + 1 == ntiles - 1) tc05::commit(bar(S::B_QE));  // Q is spent
                            }
                        }
                    }
                }
                u += 2 * ntiles;
                nv += ntiles;
            }
            if (!ok && one) atomicOr(p.status, kErrTimeout);
            // every product issued has completed before TMEM is freed
            if (one) {
                tc05::commit(bar(S::B_DR));
                mbar_wait(bar(S::B_DR), 0);
            }
            __syncwarp();
        } else if constexpr (kFp8) {
            // ---------------------------------- V of e4m3 caches, widened
            // every e4m3 value is exact in fp16; the 16-bit tile has the layout of a
            // 16-bit cache's.  A thread widens two key rows; rows that no query row
            // of the unit sees become zeros (their weight 0 must not meet a NaN)
            const int x = (warp - 10) * 32 + lane;
            int u = 0, nv = 0;
            bool ok = true;
            for (int it = 0; ok; ++it) {
                const int slot = it % kPtItems;
                if (!pt_wait(bar(S::B_IF + slot), (it / kPtItems) & 1, p)) { ok = false; break; }
                const PtItem& I = items[slot];
                if (I.end) break;
                const int ntiles = I.ntiles, t0 = I.t0, lo_all = I.lo_all, hi_all = min(I.hi_all, I.t1), bad = I.bad;
                const int32_t* table = p.block_table + static_cast<long long>(I.b) * p.bt_stride;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::B_IE + slot));
                for (int j = 0; j < ntiles; ++j, ++nv) {
                    const int vu = u + 2 * j + 1, vb = nv & 1;
                    if (!pt_wait(bar(S::B_UF + vu % S::NU), (vu / S::NU) & 1, p)) { ok = false; break; }
                    if (nv >= 2 && !pt_wait(bar(S::B_VE + vb), ((nv >> 1) - 1) & 1, p)) { ok = false; break; }
                    const uint8_t* raw = smem + S::OFF_KV + (vu % S::NU) * S::UNIT;
                    uint8_t* wide = smem + S::OFF_V + vb * S::VUNIT;
#pragma unroll 1
                    for (int r = x; r < kPtKeys; r += 64) {
                        const int key = t0 + j * kPtKeys + r, sw = r & 7;
                        bool seen = key >= lo_all && key < hi_all;
                        if (bad && seen) {
                            const int pg = table[page_div(key, p.pmagic, p.pmshift)];
                            seen = pg >= 0 && pg < p.num_pages;
                        }
                        const uint8_t* src = raw + (r >> 3) * S::GROUP + sw * 128;
                        uint8_t* dst = wide + (r >> 3) * S::VGROUP + sw * 128;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint4 e = *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4));
                            uint4 a = make_uint4(0, 0, 0, 0), b = a;
                            if (seen) {
                                a = make_uint4(e4m3x2_to_f16x2(e.x), e4m3x2_to_f16x2(e.x >> 16), e4m3x2_to_f16x2(e.y),
                                               e4m3x2_to_f16x2(e.y >> 16));
                                b = make_uint4(e4m3x2_to_f16x2(e.z), e4m3x2_to_f16x2(e.z >> 16), e4m3x2_to_f16x2(e.w),
                                               e4m3x2_to_f16x2(e.w >> 16));
                            }
                            uint8_t* half = dst + (c >> 2) * 1024;
                            *reinterpret_cast<uint4*>(half + (((2 * (c & 3)) ^ sw) << 4)) = a;
                            *reinterpret_cast<uint4*>(half + (((2 * (c & 3) + 1) ^ sw) << 4)) = b;
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(S::B_VF + vb));
                        mbar_arrive(bar(S::B_UE + vu % S::NU));
                    }
                }
                u += 2 * ntiles;
            }
            if (!ok && lane == 0) atomicOr(p.status, kErrTimeout);
        }
    } else {
        // ------------------------------------------ softmax and epilogue
        reg_inc<208>();
        const int t = warp >> 2, q4 = warp & 3, r = 32 * q4 + lane;  // row of tile t = TMEM lane
        const uint32_t lane_addr = static_cast<uint32_t>(32 * q4) << 16;
        const uint32_t s_addr = tmem + lane_addr + kPtKeys * t, o_addr = tmem + lane_addr + 256 + D * t;
        const int ri = r / G, rg = r - ri * G;
        int ns = 0, no = 0, u = 0;  // key tiles walked, accumulations drained; K/V units before the item
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int slot = it % kPtItems;
            if (!pt_wait(bar(S::B_IF + slot), (it / kPtItems) & 1, p)) { ok = false; break; }
            const PtItem& I = items[slot];
            if (I.end) break;
            const int jb = I.jb[t], je = I.je[t], t0 = I.t0, ntiles = I.ntiles;
            float m_used = -INFINITY, l = 0.f;
            if (jb < je) {
                const int tok = I.tok0 + t * TOK + ri;
                const bool valid = ri < TOK && tok < I.n;
                const bool warp_on = __any_sync(kFull, valid);
                int lo = 0, hi = 0x7fffffff;
                if (valid) token_keys(p, I.q0, I.n, I.L, I.prefix, tok, lo, hi);
                float slope = 0.f;
                const int pos = I.L - I.n + tok;
                if constexpr (kBias)
                    if (valid) slope = p.slopes[I.hk * G + rg] * kLog2e;
                const int bad = I.bad, lo_all = I.lo_all, hi_all = min(I.hi_all, I.t1);
                // key tiles [zl, zh) need no V row zeroed by this tile, [ml, mh) no mask
                // (bias: and lie before every row's position)
                const bool lead = t == 0 || !(I.jb[0] < I.je[0]);  // zeroes V rows of tiles that both walk
                const int jb0 = I.jb[0], je0 = I.je[0];
                const int zl = lo_all > t0 ? 1 : 0, zh = bad ? 0 : (hi_all - t0) / kPtKeys;
                int ml, mh;
                {
                    int l0 = valid ? lo : 0, h0 = valid ? min(hi, hi_all) : 0x7fffffff;
                    if (kBias && valid) h0 = min(h0, pos + 1);
                    ml = (__reduce_max_sync(kFull, l0) - t0 + kPtKeys - 1) / kPtKeys;
                    mh = bad ? 0 : (__reduce_min_sync(kFull, h0) - t0) / kPtKeys;  // below 0: rounded up, still masked
                    if (__reduce_min_sync(kFull, h0) < t0) mh = 0;
                }
                // capped scores beyond the polynomial's range: two tiles in a row make the
                // warp take the special functions for the next four
                int wide = kCap && p.cap_far < 0.f ? 1 << 30 : 0;
                for (int j = jb; j < je; ++j, ++ns) {
                    const int tk = t0 + j * kPtKeys;
                    if (!pt_wait(bar(S::B_SF + t), ns & 1, p)) { ok = false; break; }
                    if (warp_on) {
                        tc05::fence_after_sync();
                        PtScore w{p.scale_log2, p.cap_in, p.cap_log2, slope, static_cast<float>(pos - tk),
                                  lo - tk, min(hi, hi_all) - tk, bad ? pt_stages(p, I, tk) : 0xffu};
                        const bool masked = j < ml || j >= mh;
                        uint32_t a[32], b[32];
                        if (j == jb) {
                            // the row's first reference: its maximum over the tile
                            float top = -INFINITY;
                            auto tops = [&](auto mask) {
                                constexpr bool kMasked = decltype(mask)::value;
                                tc05::ld_32x32b_x32(s_addr, a);
                                tc05::wait_ld(a);
                                tc05::ld_32x32b_x32(s_addr + 32, b);
                                top = pt_top<kBias, kCap, kMasked>(a, 0, w, top);
                                tc05::wait_ld(b);
                                tc05::ld_32x32b_x32(s_addr + 64, a);
                                top = pt_top<kBias, kCap, kMasked>(b, 32, w, top);
                                tc05::wait_ld(a);
                                tc05::ld_32x32b_x32(s_addr + 96, b);
                                top = pt_top<kBias, kCap, kMasked>(a, 64, w, top);
                                tc05::wait_ld(b);
                                top = pt_top<kBias, kCap, kMasked>(b, 96, w, top);
                            };
                            if (masked)
                                tops(std::true_type{});
                            else
                                tops(std::false_type{});
                            m_used = kBias || top == -INFINITY ? top
                                     : kCap ? capped(top, p.cap_in, p.cap_log2) : top * p.scale_log2;
                        }
                        // one pass: weights against the reference, the tile's maximum beside
                        // them.  Where a row's maximum has outgrown the reference (or a capped
                        // score the polynomial) the pass is repeated, O and l rescaled.
                        uint32_t pk[64];
                        float2 sum[2];
#pragma unroll 1
                        for (;;) {
                            const float m = m_used == -INFINITY ? 0.f : m_used;
                            float top = -INFINITY, far = 0.f;
                            sum[0] = sum[1] = make_float2(0.f, 0.f);
                            auto pass = [&](auto poly, auto mask) {
                                constexpr bool kPoly = decltype(poly)::value, kMasked = decltype(mask)::value;
                                tc05::ld_32x32b_x32(s_addr, a);
                                tc05::wait_ld(a);
                                tc05::ld_32x32b_x32(s_addr + 32, b);
                                pt_weights<kBF16, kCap, kPoly, kBias, kMasked>(a, pk, 0, w, p.cap_c, m, sum, top, far);
                                tc05::wait_ld(b);
                                tc05::ld_32x32b_x32(s_addr + 64, a);
                                pt_weights<kBF16, kCap, kPoly, kBias, kMasked>(b, pk + 16, 32, w, p.cap_c, m, sum, top, far);
                                tc05::wait_ld(a);
                                tc05::ld_32x32b_x32(s_addr + 96, b);
                                pt_weights<kBF16, kCap, kPoly, kBias, kMasked>(a, pk + 32, 64, w, p.cap_c, m, sum, top, far);
                                tc05::wait_ld(b);
                                pt_weights<kBF16, kCap, kPoly, kBias, kMasked>(b, pk + 48, 96, w, p.cap_c, m, sum, top, far);
                            };
                            if (kCap && wide > 4)
                                pass(std::false_type{}, std::true_type{});
                            else if (masked)
                                pass(std::true_type{}, std::true_type{});
                            else
                                pass(std::true_type{}, std::false_type{});
                            if constexpr (kCap) {
                                // (far stays 0 in a pass that does not depend on it)
                                if (__any_sync(kFull, far > p.cap_far) && wide <= 4) {
                                    wide = 8;
                                    continue;
                                }
                            }
                            top = kBias ? top + m
                                  : top == -INFINITY ? top : kCap ? capped(top, p.cap_in, p.cap_log2) : top * p.scale_log2;
                            const bool need = top > m_used + (kBF16 ? kPtRescaleBF16 : kPtRescaleFP16);
                            if (!__any_sync(kFull, need)) break;
                            const float alpha = need ? fast_exp2(m_used - top) : 1.f;
                            if (need) m_used = top;
                            l *= alpha;
                            if (j > jb) {
                                if (!pt_wait(bar(S::B_OD + t), (ns - 1) & 1, p)) { ok = false; break; }
                                tc05::fence_after_sync();
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    uint32_t o[16];
                                    tc05::ld_32x32b_x16(o_addr + c, o);
                                    tc05::wait_ld();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tc05::st_32x32b_x16(o_addr + c, o);
                                }
                                tc05::wait_st();
                            }
                        }
                        if (!ok) break;
                        if (kCap && wide > 0) --wide;
                        tc05::st_32x32b_x32(s_addr, reinterpret_cast<const uint32_t(&)[32]>(pk[0]));
                        tc05::st_32x32b_x32(s_addr + 32, reinterpret_cast<const uint32_t(&)[32]>(pk[32]));
                        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                        tc05::wait_st();
                    }
                    // V rows that no row of the unit sees (stale slots, skipped pages)
                    // are zeroed: their weight 0 must not meet a NaN
                    if (!kFp8 && (j < zl || j >= zh) && (lead || j < jb0 || j >= je0)) {
                        const int vu = u + 2 * j + 1, key = tk + r;
                        if (!pt_wait(bar(S::B_UF + vu % S::NU), (vu / S::NU) & 1, p)) { ok = false; break; }
                        if (key < lo_all || key >= hi_all || (bad && !(pt_stages(p, I, tk) >> (r >> 4) & 1))) {
                            uint8_t* vrow = smem + S::OFF_KV + (vu % S::NU) * S::UNIT + (r >> 3) * S::GROUP + (r & 7) * 128;
#pragma unroll
                            for (int h = 0; h < S::REGIONS; ++h)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    *reinterpret_cast<uint4*>(vrow + h * 1024 + ((e + lane) & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async();
                    }
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(S::B_PF + t));
                }
                if (!ok) break;
            }
            // ---- the item's result (a tile without keys in it: nothing, or zeros)
            const int n = I.n, tok = I.tok0 + t * TOK + ri;
            if (I.tok0 + t * TOK < n) {
                const bool valid = ri < TOK && tok < n, live = jb < je;
                const int nsplit = I.nsplit, row = (I.q0 + tok) * p.Hq + I.hk * G + rg;  // below T * Hq < 2^31
                const bool whole = nsplit <= 1 && !partials;
                const long long part0 = whole ? 0 : static_cast<long long>(I.split) * p.T * p.Hq;
                const float inv = l > 0.f ? (whole ? p.v_scale : 1.f) / l : 0.f;
                if (live) {
                    if (!pt_wait(bar(S::B_OF + t), no & 1, p)) { ok = false; break; }
                    ++no;
                    tc05::fence_after_sync();
                }
                // 64 output bytes of every row at a time through the warp's staging area, so
                // that a store instruction covers 64 consecutive bytes of eight rows
                const int kind = whole ? p.out_dtype : 3, elt = kind == 3 ? 4 : 2;
                const int dst_row = valid && (whole || l > 0.f) ? row : -1;
                uint8_t* dst0 = whole ? static_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(p.part_out + part0 * D);
                uint8_t* stage = smem + S::OFF_STAGE + warp * 2048;
                auto flush = [&](const uint32_t (&h)[16], int byte) {
                    const int sw = (lane >> 1) & 3;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ sw) << 4)) =
                            make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = 8 * i + (lane >> 2);
                        const int dr = __shfl_sync(kFull, dst_row, rr);
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
                        if (dr >= 0)
                            __stcg(reinterpret_cast<uint4*>(dst0 + static_cast<long long>(dr) * (D * elt) + byte + (lane & 3) * 16), v);
                    }
                    __syncwarp();
                };
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    if (live) {
                        tc05::ld_32x32b_x32(o_addr + c, o);
                        tc05::wait_ld(o);
                        if (c == D - 32) {
                            // drained: the next item's O product may begin
                            tc05::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(S::B_OE + t));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = l > 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
                    uint32_t h[16];
                    if (kind == 3) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) h[e] = o[16 * half + e];
                            flush(h, 4 * c + 64 * half);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = __uint_as_float(o[2 * e]), y = __uint_as_float(o[2 * e + 1]);
                            h[e] = kind == 0 ? pack2<true>(x, y) : pack2<false>(x, y);
                        }
                        flush(h, 2 * c);
                    }
                }
                if (valid) {
                    const float l2 = l > 0.f ? m_used + __log2f(l) : -INFINITY;
                    if (!whole)
                        __stcg(p.part_lse + part0 + row, l2);
                    else if (p.lse)
                        p.lse[row] = l2 * kLn2;
                }
                if (!partials && nsplit > 1) {
                    // publish this tile's part (the group's barrier, then one arrival with
                    // release semantics); the arrival that completes the unit merges its rows
                    const int tok_end = min(I.tok0 + 2 * TOK, n), tiles = I.tok0 + TOK < n ? 2 : 1;
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
                    if ((tid & 127) == 0) scan[24 + t] = atom_add_acq_rel_gpu(p.counters + I.unit);
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
                    if (scan[24 + t] == nsplit * tiles - 1) {
                        const int rows = (tok_end - I.tok0) * G;
                        const long long step = static_cast<long long>(p.T) * p.Hq;
#pragma unroll 1
                        for (int x = q4; x < rows; x += 4) {
                            const long long mrow = static_cast<long long>(I.q0 + I.tok0 + x / G) * p.Hq + I.hk * G + x % G;
                            float acc[D / 32], mx, ws;
                            pt_merge_row<D>(p.part_lse + mrow, p.part_out + mrow * D, step, nsplit, lane, acc, mx, ws);
                            const float sc = ws > 0.f ? p.v_scale / ws : 0.f;
#pragma unroll
                            for (int e = 0; e < D / 32; ++e)
                                store_out(p.out, mrow * D + lane * (D / 32) + e, acc[e] * sc, p.out_dtype);
                            if (lane == 0 && p.lse) p.lse[mrow] = ws > 0.f ? (mx + __log2f(ws)) * kLn2 : -INFINITY;
                        }
                        if ((tid & 127) == 0) p.counters[I.unit] = 0;  // every part has arrived: ready for the next call
                    }
                }
            }
            u += 2 * ntiles;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S::B_IE + slot));
        }
        if (!ok && lane == 0) atomicOr(p.status, kErrTimeout);
    }

    // ---------------------------------------------------------- tear-down
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc05::fence_after_sync();
        tc05::dealloc(tmem, 512);
    }
    // the last CTA to leave resets the item counter for the next call
    if (tid == 0) {
        const int prev = atom_add_acq_rel_gpu(p.queue + 1);
        if (prev == static_cast<int>(gridDim.x) - 1) {
            p.queue[0] = 0;
            p.queue[1] = 0;
        }
    }
}

}  // namespace pkd
