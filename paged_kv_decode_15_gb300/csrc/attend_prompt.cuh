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
//                 reference of its weights moves only when a row's maximum outgrows it by
//                 2^14 or so (O and l are then rescaled by the row's own warp; how far, and
//                 from where, is the plan's choice: AttendParams::ref_up)
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
// softmax 176 registers and spills: 8192-token prompt 523 us, not 416.)
//
// What bounds it, D = 128 (32768-token prompt, 32 heads: 6.1 ms a call, 1440 TFLOP/s,
// 0.77 of a dense library product; 8192 tokens 414 us): per row tile a loop of the softmax
// (1540 cycles a key tile: 940 of exponentials and packing, the rest TMEM loads and
// stores and the arrival), the issuing warp's wake-up (270), the products (1120) and
// the softmax's (300).  Two row tiles run interleaved, so the tensor cores, 2050
// cycles a pair, are busy two thirds of its 3200; TMEM has no columns for a third
// tile or a second S.  An item costs another 6000 cycles or so between its last tile
// and the next one's first, a launch 15000 before its first tile (set-up, the item's
// chain of loads, Q and K) and as many for its first two tiles, whose code comes
// from memory: what bounds short launches.
// Work items are handed out by an atomic counter in the workspace, the longest of
// a request first, so CTAs finish together whatever the lengths; results do not
// depend on who computes an item.  Every wait is bounded.
#pragma once

#include <type_traits>

#include "attend.cuh"
#include "packed.cuh"
#include "tc05.cuh"

namespace pkd {

constexpr int kPtKeys = 128;       // keys per tile
constexpr int kPtRows = 128;       // rows per tile (TMEM lanes)
constexpr int kPtThreads = 384;
constexpr int kPtItems = 4;        // work-item ring
constexpr int kPtMaxBatch = 2048;  // requests whose tile prefix the CTA keeps in shared memory
constexpr int kPtL2Bytes = 64 << 20;  // keys and values walked together
// Row-tile pairs that a launch orders by weight, and items per CTA up to which it does.
constexpr int kPtMaxOrder = 512, kPtOrderItems = 16;
// A row's reference m moves when its maximum exceeds m by this (log2 units): its weights
// 2^(logit - m) must not overflow the operand type, which for fp16 ends at 2^16, and with
// bf16, whose V has fp32's range, they stay at 1 or below, so that O does not leave it.
// Where the reference lies to begin with is the plan's choice (AttendParams::ref_up).
// (Taken from the difference: a sum m + 15 of large logits would round up to m + 16.)
constexpr float kPtRoomBF16 = 0.f, kPtRoomFP16 = 15.f;

// Key tiles after which a row's O is folded away into the workspace and begun anew.
// The tensor cores cut an accumulation off to fp32 after every 16 keys, so that n keys
// of alike weight came out low by 0.85 n / 16 ulps: 2e-4 at 32768 keys, 3.2e-3 at
// 524288, more than six half steps of fp16.  Folded every 32768 keys, no sum loses
// more than 2048 x 2^-23 = 2^-12.  (4096 tokens on 131072 keys: 6.83 -> 6.82 ms, in fp16
// at D = 64 5.15 -> 5.23 ms.)
constexpr int kPtFold = 256;

struct PtItem {
    int b, hk, q0, n, L, prefix;   // request, kv head, first query token, query tokens, length, prefix keys
    int tok0;                      // first token (of the request) of the item's rows
    int t0, t1, ntiles;            // keys of this item, tiles of 128 from t0
    int lo_all, hi_all;            // keys outside are seen by no row of the unit
    int split, nsplit, unit;
    int jb[2], je[2];              // steps [jb, je) of row tile t (empty: none); step j is key tile pt_tile(j)
    int bad, end;                  // bad: some page lies outside the pool
};

// Types of q and the cache.
enum PtType { kPtBF16 = 0, kPtFP16 = 1, kPtFP8 = 2 };

// Key tile of step j.  With a distance bias the walk runs from the last tile to the
// first: a row meets its largest logits first, and its reference stays (rising,
// slopes near 1 moved it at every tile: 8192-token prompt 992 us).
template <bool kBias>
__device__ __forceinline__ int pt_tile(int j, int ntiles) { return kBias ? ntiles - 1 - j : j; }

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
    static constexpr int OFF_SCAN = OFF_PREF + (kPtMaxBatch + 4) * 4;  // 16 warp sums, arrival flags
    static constexpr int OFF_ORDER = OFF_SCAN + 128;     // uint16 [kPtMaxOrder]: row-tile pairs, longest first
    static constexpr int OFF_BAR = (OFF_ORDER + kPtMaxOrder * 2 + 7) & ~7;
    static_assert(8 * 2048 >= kPtMaxOrder * 2, "weights fit the staging area");
    // units full/empty, Q full/empty, S full, P full, O step done, O full/drained, item full/empty, widened V,
    // a split item's part stored/counted, drain
    static constexpr int B_UF = 0, B_UE = B_UF + NU, B_QF = B_UE + NU, B_QE = B_QF + 1, B_SF = B_QE + 1;
    static constexpr int B_PF = B_SF + 2, B_OD = B_PF + 2, B_OF = B_OD + 2, B_OE = B_OF + 2, B_IF = B_OE + 2;
    static constexpr int B_IE = B_IF + kPtItems, B_VF = B_IE + kPtItems, B_VE = B_VF + NV, B_JA = B_VE + NV;
    static constexpr int B_JD = B_JA + 2, B_DR = B_JD + 2, NBAR = B_DR + 1;
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

// The request whose units (row-tile pairs times `mul`) hold unit r; pref: prefix of the pairs.
__device__ __forceinline__ int pt_request(const int* pref, int B, int mul, int r) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(pref[mid]) * mul <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// Every lane of the warp waits, with a warp-uniform result: false after kWaitNs of
// wall time, or once another role or CTA has reported a timeout.
__device__ __forceinline__ bool pt_wait(uint32_t bar, uint32_t parity, const AttendParams& p) {
    uint64_t t0 = 0;
    bool done = true;
#pragma unroll 1
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (i & 255u) continue;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitNs || (*reinterpret_cast<const volatile int32_t*>(p.status) & kErrTimeout)) {
            done = false;
            break;
        }
    }
    return __all_sync(kFull, done);
}

// The issuing warp's wait for the queries of its CTA's item `it`.  With p.wait_ns = 0
// (diagnostic) a single test of the barrier: every second CTA gives up on its first
// item so, the others on a later one, between an epilogue and its join.  (The same in
// the waits for keys and values cost packed documents 2%.)
__device__ __forceinline__ bool pt_wait_queries(uint32_t bar, uint32_t parity, const AttendParams& p, int it) {
    if (p.wait_ns || (it == 0 && (blockIdx.x & 1))) return pt_wait(bar, parity, p);
    return __all_sync(kFull, mbar_test_wait(bar, parity));
}

// A chunk is 32 keys of a row's tile, k0 .. k0 + 31 from the tile's first: their
// products q.k as loaded, turned in place into what the exponential takes.

// c tanh(scale q.k / c) in log2 units.  kPoly: q.k times a polynomial in its square
// (for |q.k| <= cap_far) on packed FMAs; else by exponential and reciprocal
// (capped(): two more special-function results per key).
template <bool kPoly>
__device__ __forceinline__ void pt_cap(uint32_t (&v)[32], const AttendParams& p) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float2 x = make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1]));
        if constexpr (kPoly) {
            const float2 z = mul2(x, x);
            float2 t = fma2(z, both(p.cap_c[4]), both(p.cap_c[3]));
            t = fma2(z, t, both(p.cap_c[2]));
            t = fma2(z, t, both(p.cap_c[1]));
            t = fma2(z, t, both(p.cap_c[0]));
            x = mul2(t, x);
        } else {
            x = make_float2(capped(x.x, p.cap_in, p.cap_log2), capped(x.y, p.cap_in, p.cap_log2));
        }
        v[c] = __float_as_uint(x.x);
        v[c + 1] = __float_as_uint(x.y);
    }
}

// scale x - slope |dist - c|, dist: position minus the chunk's first key.  kBehind: no
// key lies behind the position, the distance is linear in c.
template <bool kBehind>
__device__ __forceinline__ void pt_bias(uint32_t (&v)[32], float scale, float slope, float dist) {
    const float nb = -slope * dist;
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float2 x = make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), add;
        if constexpr (kBehind)
            add = make_float2(fmaf(slope, static_cast<float>(c), nb), fmaf(slope, static_cast<float>(c + 1), nb));
        else
            add = make_float2(-slope * fabsf(dist - static_cast<float>(c)), -slope * fabsf(dist - static_cast<float>(c + 1)));
        x = fma2(x, both(scale), add);
        v[c] = __float_as_uint(x.x);
        v[c + 1] = __float_as_uint(x.y);
    }
}

// -inf where the row does not see the key: keys [c0, c1) of the chunk are seen, and
// of its two 16-key stages those whose bit is set.
__device__ __forceinline__ void pt_mask(uint32_t (&v)[32], int c0, int c1, unsigned stages) {
    const int a = max(c0, 0), b = min(c1, 32);
    uint32_t seen = a < b ? (0xffffffffu >> (32 - (b - a))) << a : 0u;
    if (!(stages & 1)) seen &= 0xffff0000u;
    if (!(stages & 2)) seen &= 0x0000ffffu;
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (!(seen >> c & 1)) v[c] = 0xff800000u;
}

// The largest |x| (kAbs) or x of a chunk.
template <bool kAbs>
__device__ __forceinline__ float pt_max(const uint32_t (&v)[32]) {
    float top[2] = {kAbs ? 0.f : -INFINITY, kAbs ? 0.f : -INFINITY};
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const float x = __uint_as_float(v[c]), y = __uint_as_float(v[c + 1]);
        float& m = top[(c >> 1) & 1];
        m = kAbs ? max3(m, fabsf(x), fabsf(y)) : max3(m, x, y);
    }
    return fmaxf(top[0], top[1]);
}

// The weights 2^(scale x - m) of a chunk, packed to the operand type, and their sum:
// l sums the fp32 weights, the product takes them rounded.
template <bool kBF16>
__device__ __forceinline__ float pt_weights(const uint32_t (&v)[32], uint32_t (&pk)[16], float scale, float m) {
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float2 x = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), both(scale), both(-m));
        x.x = fast_exp2(x.x);
        x.y = fast_exp2(x.y);
        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], x);
        pk[c >> 1] = pack2<kBF16>(x.x, x.y);
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// o += f times the N folded sums at `fold` (its row's, four dims every kPtRows vectors).
template <int N>
__device__ __forceinline__ void pt_add_folded(uint32_t (&o)[N], const float4* fold, float f) {
#pragma unroll
    for (int e = 0; e < N / 4; ++e) {
        const float4 x = __ldcg(fold + e * kPtRows);
        o[4 * e] = __float_as_uint(fmaf(f, x.x, __uint_as_float(o[4 * e])));
        o[4 * e + 1] = __float_as_uint(fmaf(f, x.y, __uint_as_float(o[4 * e + 1])));
        o[4 * e + 2] = __float_as_uint(fmaf(f, x.z, __uint_as_float(o[4 * e + 2])));
        o[4 * e + 3] = __float_as_uint(fmaf(f, x.w, __uint_as_float(o[4 * e + 3])));
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

// partials: every result is left as a partial one (for a merge that follows)
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
    uint16_t* order = reinterpret_cast<uint16_t*>(smem + S::OFF_ORDER);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::OFF_TMEM);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.G, TOK = kPtRows / G;  // whole tokens per row tile
    auto bar = [&](int i) { return smem_u32(bars + i); };

    // ------------------------------------------------------------ set-up
    launch_dependents();  // the next launch may fill SMs that this one leaves
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
            mbar_init(bar(S::B_JA + i), 4);
            mbar_init(bar(S::B_JD + i), 1);
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
        // (unsigned: at most 384 x 2^23 pairs at a time, should requests overlap)
        const unsigned room = p.max_pairs;
        unsigned run = 0;
        for (int b0 = 0; b0 < p.B; b0 += kPtThreads) {
            const int b = b0 + tid;
            unsigned v = 0;
            if (b < p.B) {
                int q0, n;
                request_tokens(p, b, q0, n, blockIdx.x == 0);
                v = (n + 2 * TOK - 1) / (2 * TOK);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(kFull, v, o);
                if (lane >= o) v += y;
            }
            if (lane == 31) scan[warp] = v;
            __syncthreads();
            unsigned before = run;
            for (int k = 0; k < kPtThreads / 32; ++k) {
                const unsigned s = scan[k];
                if (k < warp) before += s;
                run += s;
            }
            // requests of a bad query_start may overlap: pairs past the plan's are dropped
            run = min(run, room);
            if (b < p.B) pref[b + 1] = min(before + v, room);
            __syncthreads();
        }
        if (tid == 0) pref[0] = 0;
        __syncthreads();
    }
    // Few items per CTA: the longest are handed out first, whatever the lengths and
    // masks.  Every CTA ranks the pairs alike, by key tiles and then by number
    // (packed documents, 416 items on 152 CTAs: the last CTA ended after twice the mean time).
    const int npairs = pref[p.B];
    const bool ordered = npairs > 1 && npairs <= kPtMaxOrder && npairs * p.Hkv > static_cast<int>(gridDim.x) &&
                         npairs * p.Hkv <= kPtOrderItems * static_cast<int>(gridDim.x);
    if (ordered) {
        uint16_t* weight = reinterpret_cast<uint16_t*>(smem + S::OFF_STAGE);
        // A pair's weight: the keys from its first token's to its last token's.  (Only the
        // order depends on it: a look at every token's document took 10k cycles.)
        for (int x = tid; x < npairs; x += kPtThreads) {
            const int b = pt_request(pref, p.B, 1, x);
            int q0, n, lo = 0x7fffffff, hi = 0;
            request_tokens(p, b, q0, n, false);
            const int L = request_len(p, b, false), prefix = p.prefix_lens ? p.prefix_lens[b] : 0;
            const int a0 = (x - pref[b]) * 2 * TOK, a1 = min(a0 + 2 * TOK, n) - 1;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                int k0, k1;
                token_keys(p, q0, n, L, prefix, e ? a1 : a0, k0, k1);
                if (k0 < k1) lo = min(lo, k0), hi = max(hi, k1);
            }
            weight[x] = static_cast<uint16_t>(min(65535, hi > lo ? (hi - lo + kPtKeys - 1) / kPtKeys : 0));
        }
        __syncthreads();
        for (int x = tid; x < npairs; x += kPtThreads) {
            const int mine = weight[x];
            int rank = 0;
#pragma unroll 4
            for (int y = 0; y < npairs; ++y) rank += weight[y] > mine || (weight[y] == mine && y < x);
            order[rank] = static_cast<uint16_t>(x);
        }
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = *tslot;
    constexpr uint32_t kIdS = kFp8 ? tc05::idesc_e4m3(kPtRows, kPtKeys)
                                   : tc05::idesc_f16(kBF16, kPtRows, kPtKeys, false, false);  // S = Q K^T
    constexpr uint32_t kIdO = tc05::idesc_f16(kBF16, kPtRows, D, false, true);         // O += P V

    if (warp >= 8) {
        reg_dec<104>();
        if (warp == 8) {
            // ------------------------------------------------------ loads
            if (lane == 0) {
                prefetch_tmap(&kvmap);
                prefetch_tmap(&qmap);
            }
            const uint64_t pol = policy_evict_first();
            uint64_t keep;  // other row tiles read the same keys and values
            asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
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
                    // item idx: splits innermost, then the kv heads of a pair, by `order`; or
                    // request by request groups of kv heads whose keys and values fit half of
                    // L2 together, in each the row tiles from the last (the longest, causal) to
                    // the first, all heads of the group per tile
                    const int split = idx % p.max_splits, r1 = idx / p.max_splits;
                    int b, pair, hk;
                    if (ordered) {
                        hk = r1 % p.Hkv;
                        pair = order[r1 / p.Hkv];
                        b = pt_request(pref, p.B, 1, pair);
                        pair -= pref[b];
                    } else {
                        b = pt_request(pref, p.B, p.Hkv, r1);
                    }
                    int q0, n;
                    request_tokens(p, b, q0, n, false);
                    if (!ordered) {
                        const int npair = pref[b + 1] - pref[b], r2 = r1 - pref[b] * p.Hkv;
                        const int group = max(1, min(p.Hkv, kPtL2Bytes / (2 * S::ROWB) / max(request_len(p, b, false), 1)));
                        const int g = r2 / (npair * group), width = min(group, p.Hkv - g * group), r3 = r2 - g * npair * group;
                        pair = npair - 1 - r3 / width;
                        hk = g * group + r3 % width;
                    }
                    const int L = request_len(p, b, pair == 0 && hk == 0 && split == 0 && lane == 0);
                    const int prefix = p.prefix_lens ? p.prefix_lens[b] : 0;
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
                            const int first = (a - t0) / kPtKeys, past = (z - t0 + kPtKeys - 1) / kPtKeys;
                            I.jb[t] = a >= z ? 0 : kBias ? ntiles - past : first;
                            I.je[t] = a >= z ? 0 : kBias ? ntiles - first : past;
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
            // Round r publishes item r, loads the rest of item r - 1's tiles, then Q and the
            // first tiles of item r.  (An item's slot is not reused before this warp
            // publishes four items on.)
            int hk = 0, t0 = 0, t1 = 0, ntiles = 0, j = 0, pg = -1;
            const int32_t* row = p.block_table;
            auto entry = [&](int x) {
                const int tok = t0 + pt_tile<kBias>(x, ntiles) * kPtKeys + lane * kStageTok;
                return lane < kPtKeys / kStageTok && tok < t1 ? row[page_div(tok, p.pmagic, p.pmshift)] : -1;
            };
            for (int r = 0; ok; ++r) {
                ok = publish();
                bool end = false;
#pragma unroll 1
                for (int part = 0; ok && part < 2; ++part) {
                    int stop = ntiles;
                    if (part == 1) {
                        const PtItem& I = items[r % kPtItems];
                        end = I.end;
                        if (end) break;
                        hk = I.hk;
                        t0 = I.t0;
                        t1 = I.t1;
                        ntiles = I.ntiles;
                        row = p.block_table + static_cast<long long>(I.b) * p.bt_stride;
                        j = 0;
                        stop = min(ntiles, S::NU / 2);  // the ring is full behind them
                        if (!ntiles) break;
                        pg = entry(0);
                        // Q (128-byte regions), once the last item's products have read theirs
                        if (nq >= 1 && !pt_wait(bar(S::B_QE), (nq - 1) & 1, p)) { ok = false; break; }
                        if (lane == 0) {
                            const int tiles = I.tok0 + TOK < I.n ? 2 : 1;
                            mbar_arrive_expect_tx(bar(S::B_QF), tiles * S::REGIONS * TOK * G * 128);
                            for (int x = 0; x < tiles * S::REGIONS; ++x) {
                                const int t = x / S::REGIONS, h = x % S::REGIONS;
                                tma_load_3d(sb0 + S::OFF_Q + t * S::QTILE + h * kPtRows * 128, &qmap, 64 * h, hk * G,
                                            I.q0 + I.tok0 + t * TOK, bar(S::B_QF), pol);
                            }
                        }
                        __syncwarp();
                        ++nq;
                    }
#pragma unroll 1
                    for (; j < stop && ok; ++j) {
                        const int pg_next = j + 1 < ntiles ? entry(j + 1) : -1;
                        const int tok = t0 + pt_tile<kBias>(j, ntiles) * kPtKeys + lane * kStageTok;
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
                        pg = pg_next;
                    }
                }
                if (end) break;
            }
            // Let every issued copy land before the CTA leaves, also where this warp was done
            // and the ones that read the copies have given up: what lands later would land
            // in the shared memory of another CTA.
            for (int j = max(0, u - S::NU); j < u; ++j) mbar_wait(bar(S::B_UF + j % S::NU), (j / S::NU) & 1);
            if (nq) mbar_wait(bar(S::B_QF), (nq - 1) & 1);
            if (!ok && lane == 0) atomicOr(p.status, kErrTimeout);
        } else if (warp == 9) {
            // --------------------------------------------------- products
            // The whole warp walks the items, converged, and one elected lane issues (with
            // the loop under a lane test instead, a product took 115 cycles to issue, more
            // than the 75 it takes to run).
            const bool one = tc05::elect_one();
            const uint32_t tm = tc05::uniform(tmem), qlo = tc05::uniform(tc05::desc_lo(sb0 + S::OFF_Q, 16));
            bool ok = true;
            int u = 0, nq = 0, nv = 0;      // K/V units, Q loads, widened V tiles before the item
            int np[2] = {0, 0}, no[2] = {0, 0};  // per tile: P tiles consumed, accumulations begun
            for (int it = 0; ok; ++it) {
                const int slot = it % kPtItems;
                if (!pt_wait(bar(S::B_IF + slot), (it / kPtItems) & 1, p)) { ok = false; break; }
                const PtItem& I = items[slot];
                if (I.end) break;
                const int ntiles = I.ntiles, jbs[2] = {I.jb[0], I.jb[1]}, jes[2] = {I.je[0], I.je[1]};
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(S::B_IE + slot));
                if (!ntiles) continue;
                if (!pt_wait_queries(bar(S::B_QF), nq & 1, p, it)) { ok = false; break; }
                ++nq;
                // round j: the O products of key tile j, the S products of key tile j + 1.  A tile's
                // S product goes in issue order behind its O product, which has read the P under S.
#pragma unroll 1
                for (int j = -1; ok && j < ntiles; ++j) {
                    const int ku = u + 2 * (j + 1), vu = u + 2 * j + 1, vb = kFp8 ? (nv + j) & 1 : 0;
                    if (j >= 0)
                        ok = kFp8 ? pt_wait(bar(S::B_VF + vb), ((nv + j) >> 1) & 1, p)
                                  : pt_wait(bar(S::B_UF + vu % S::NU), (vu / S::NU) & 1, p);
                    const uint32_t vlo = tc05::uniform(tc05::desc_lo(
                        sb0 + (kFp8 ? S::OFF_V + vb * S::VUNIT : S::OFF_KV + ((vu + S::NU) % S::NU) * S::UNIT), 1024));
                    const uint32_t klo = tc05::uniform(tc05::desc_lo(sb0 + S::OFF_KV + (ku % S::NU) * S::UNIT, 16));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok) break;
                        const int jb = jbs[t], je = jes[t];
                        const uint32_t s_addr = tm + kPtKeys * t, o_addr = tm + 256 + D * t;
                        if (j >= jb && j < je) {
                            ok = pt_wait(bar(S::B_PF + t), np[t] & 1, p);
                            ++np[t];
                            if (ok && j == jb) {
                                // a new accumulation: the last one has been read out
                                if (no[t] >= 1) ok = pt_wait(bar(S::B_OE + t), (no[t] - 1) & 1, p);
                                ++no[t];
                            }
                            if (!ok) break;
                            tc05::fence_after_sync();
                            const bool more = (j - jb) % kPtFold != 0;  // (a fresh sum behind a fold)
#pragma unroll
                            for (int kk = 0; kk < kPtKeys / 16; ++kk)
                                if (one)
                                    tc05::mma_ts(o_addr, s_addr + 8 * kk, vlo + ((2 * kk * S::VGROUP) >> 4),
                                                 tc05::desc_hi(S::VGROUP), kIdO, more || kk > 0);
                            if (one) {
                                tc05::commit(bar(S::B_OD + t));
                                if (j == je - 1) tc05::commit(bar(S::B_OF + t));
                            }
                        }
                        if (j >= 0 && t == 1 && one) tc05::commit(kFp8 ? bar(S::B_VE + vb) : bar(S::B_UE + vu % S::NU));
                        if (j + 1 < ntiles) {
                            if (t == 0) {
                                ok = pt_wait(bar(S::B_UF + ku % S::NU), (ku / S::NU) & 1, p);
                                if (!ok) break;
                                tc05::fence_after_sync();
                            }
                            if (j + 1 >= jb && j + 1 < je) {
#pragma unroll
                                for (int kk = 0; kk < S::ROWB / 32; ++kk)
                                    if (one)
                                        tc05::mma_ss<kFp8>(s_addr,
                                                           qlo + ((t * S::QTILE + (kk >> 2) * kPtRows * 128 + (kk & 3) * 32) >> 4),
                                                           tc05::desc_hi(1024), klo + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                                                           tc05::desc_hi(S::GROUP), kIdS, kk > 0);
                                if (one) tc05::commit(bar(S::B_SF + t));
                            }
                            if (t == 1 && one) {
                                tc05::commit(bar(S::B_UE + ku % S::NU));
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
                        const int key = t0 + pt_tile<kBias>(j, ntiles) * kPtKeys + r, sw = r & 7;
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
        reg_inc<200>();
        const int t = warp >> 2, q4 = warp & 3, r = 32 * q4 + lane;  // row of tile t = TMEM lane
        const uint32_t lane_addr = static_cast<uint32_t>(32 * q4) << 16;
        const uint32_t s_addr = tmem + lane_addr + kPtKeys * t, o_addr = tmem + lane_addr + 256 + D * t;
        const int ri = r / G, rg = r - ri * G;
        int ns = 0, u = 0;  // key tiles walked; K/V units before the item
        int no = 0;         // twice the accumulations drained, plus the parity of the parts published (a register less)
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int slot = it % kPtItems;
            if (!pt_wait(bar(S::B_IF + slot), (it / kPtItems) & 1, p)) { ok = false; break; }
            const PtItem& I = items[slot];
            if (I.end) break;
            const int jb = I.jb[t], je = I.je[t], t0 = I.t0, ntiles = I.ntiles;
            float m_used = -INFINITY, l = 0.f;
            // where the row's O is folded away to, and behind it the reference it had then
            auto fold_row = [&]() { return p.fold + (static_cast<int>(blockIdx.x) * 2 + t) * (D / 4 + 1) * kPtRows + r; };
            auto fold_factor = [&](const float4* fold) {
                const float m = __ldcg(&fold[D / 4 * kPtRows].x);
                return m == -INFINITY ? 0.f : fast_exp2(m - m_used);
            };
            if (jb < je) {
                const int tok = I.tok0 + t * TOK + ri;
                const bool valid = ri < TOK && tok < I.n;
                const bool warp_on = __any_sync(kFull, valid);
                int lo = 0, hi = 0x7fffffff;
                if (valid) token_keys(p, I.q0, I.n, I.L, I.prefix, tok, lo, hi);
                // lanes without a row hold what was left in shared memory: they have no say in the
                // warp's votes, or the roundings of its rows would depend on the CTA's last item
                if (!valid) m_used = INFINITY;
                const float cap_far = valid ? p.cap_far : INFINITY;
                float slope = 0.f;
                const int pos = I.L - I.n + tok;
                if constexpr (kBias)
                    if (valid) slope = p.slopes[I.hk * G + rg] * kLog2e;
                const int bad = I.bad, lo_all = I.lo_all, hi_all = min(I.hi_all, I.t1);
                // key tiles [zl, zh) need no V row zeroed by this tile; keys [ml, mh) need no mask
                const bool lead = t == 0 || !(I.jb[0] < I.je[0]);  // zeroes V rows of tiles that both walk
                const int jb0 = I.jb[0], je0 = I.je[0];
                const int zl = lo_all > t0 ? 1 : 0, zh = bad ? 0 : (hi_all - t0) / kPtKeys;
                const int ml = __reduce_max_sync(kFull, valid ? lo : 0);
                // (with a bias no key from there on lies behind some row's position)
                const int mh = bad ? 0 : __reduce_min_sync(kFull, valid ? min(min(hi, hi_all), kBias ? pos + 1 : hi_all) : 0x7fffffff);
                int wide = 0;  // tiles left before a capped score out of the polynomial's range counts no more
                constexpr float kRoom = kBF16 ? kPtRoomBF16 : kPtRoomFP16;
                for (int j = jb; j < je; ++j, ++ns) {
                    const int kt = pt_tile<kBias>(j, ntiles), tk = t0 + kt * kPtKeys;
                    if (j > jb && (j - jb) % kPtFold == 0 && warp_on) {
                        // O so far, with what was folded before, to the workspace; the product
                        // of this tile, which waits for its P, begins a new one
                        if (!pt_wait(bar(S::B_OD + t), (ns - 1) & 1, p)) { ok = false; break; }
                        tc05::fence_after_sync();
                        float4* fold = fold_row();
                        const bool any = j - jb > kPtFold;
                        const float f = any ? fold_factor(fold) : 0.f;
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tc05::ld_32x32b_x16(o_addr + c, o);
                            tc05::wait_ld();
                            if (any) pt_add_folded<16>(o, fold + c / 4 * kPtRows, f);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                __stcg(fold + (c / 4 + e) * kPtRows,
                                       make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3])));
                        }
                        __stcg(&fold[D / 4 * kPtRows].x, m_used);
                    }
                    if (!pt_wait(bar(S::B_SF + t), ns & 1, p)) { ok = false; break; }
                    if (warp_on) {
                        tc05::fence_after_sync();
                        uint32_t v[2][32];
                        tc05::ld_32x32b_x32(s_addr, v[0]);
                        const bool masked = tk < ml || tk + kPtKeys > mh;
                        const float scale = (kCap || kBias) ? 1.f : p.scale_log2;
                        bool done = false;
                        const int c0 = lo - tk, c1 = min(hi, hi_all) - tk;
                        auto straight = [&](auto masked_tile) {
                            constexpr bool kMasked = decltype(masked_tile)::value;
                            // One pass of straight-line code against the reference of the tiles
                            // before.  The tile's maximum comes out beside the weights: they count
                            // only if no row has outgrown its reference (and no capped score the
                            // polynomial).  (Decided chunk by chunk, the pass took 1460 cycles, not
                            // 950.)  Tiles with masked keys have a copy of it where neither a cap nor
                            // a bias needs its registers (packed documents 99 -> 72 us, 8192-token
                            // prompt 419 -> 415; with them it spills: capped prompts with a window
                            // 179 -> 192, biased 8192-token prompt 440 -> 455).
                            const float m = m_used == -INFINITY ? 0.f : m_used;
                            uint32_t pk[4][16];
                            float sum = 0.f, top = -INFINITY, far = 0.f;
                            tc05::wait_ld(v[0]);
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint32_t (&x)[32] = v[c & 1];
                                if (c < 3) tc05::ld_32x32b_x32(s_addr + 32 * (c + 1), v[(c + 1) & 1]);
                                if constexpr (kCap) {
                                    far = fmaxf(far, pt_max<true>(x));
                                    pt_cap<true>(x, p);
                                }
                                if constexpr (kBias) {
                                    const float dist = static_cast<float>(pos - tk - 32 * c);
                                    pt_bias<true>(x, kCap ? 1.f : p.scale_log2, slope, dist);
                                }
                                if constexpr (kMasked) pt_mask(x, c0 - 32 * c, c1 - 32 * c, 3u);
                                top = fmaxf(top, pt_max<false>(x));
                                sum += pt_weights<kBF16>(x, pk[c], scale, m);
                                if (c < 3) tc05::wait_ld(v[(c + 1) & 1]);
                            }
                            const bool grown = fmaf(top, scale, -m_used) > kRoom, out = kCap && far > cap_far;
                            done = !__any_sync(kFull, grown || out);
                            if (done) {
                                l += sum;
#pragma unroll
                                for (int c = 0; c < 4; ++c) tc05::st_32x32b_x16(s_addr + 16 * c, pk[c]);
                            } else {
                                if (kCap && __any_sync(kFull, out)) wide = 8;
                                tc05::ld_32x32b_x32(s_addr, v[0]);
                            }
                        };
                        if (j > jb && !(kCap && wide > 0)) {
                            if (!masked)
                                straight(std::false_type{});
                            else if constexpr (!kCap && !kBias)
                                if (!bad) straight(std::true_type{});
                        }
                        if (!done) {
                            // Any other tile, in two rolled passes: the maximum, with which the
                            // references move (O and l follow), then the weights, written over
                            // products that are spent
                            const unsigned stages = bad ? pt_stages(p, I, tk) : 0xffu;
                            const unsigned loaded = stages & (0xffu >> max(0, 8 - (hi_all - tk + kStageTok - 1) / kStageTok));
                            auto logits = [&](uint32_t (&x)[32], int c) {
                                if constexpr (kCap) {
                                    // (nor have keys that were not loaded)
                                    const unsigned here = loaded >> (2 * c);
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (!(here >> e & 1)) {
#pragma unroll
                                            for (int i = 0; i < 16; ++i) x[16 * e + i] = 0u;
                                        }
                                    if (__any_sync(kFull, pt_max<true>(x) > cap_far))
                                        pt_cap<false>(x, p);
                                    else
                                        pt_cap<true>(x, p);
                                }
                                if constexpr (kBias) pt_bias<false>(x, kCap ? 1.f : p.scale_log2, slope, static_cast<float>(pos - tk - 32 * c));
                                if (masked) pt_mask(x, c0 - 32 * c, c1 - 32 * c, stages >> (2 * c));
                            };
                            // (without a bias the logit rises with q.k: the largest product gives the largest)
                            auto tops = [&](uint32_t (&x)[32], int c) {
                                if constexpr (kBias)
                                    logits(x, c);
                                else if (masked)
                                    pt_mask(x, c0 - 32 * c, c1 - 32 * c, stages >> (2 * c));
                                return pt_max<false>(x);
                            };
                            float top = -INFINITY;
                            tc05::wait_ld(v[0]);
#pragma unroll 1
                            for (int c = 0; c < 4; c += 2) {
                                tc05::ld_32x32b_x32(s_addr + 32 * c + 32, v[1]);
                                top = fmaxf(top, tops(v[0], c));
                                tc05::wait_ld(v[1]);
                                tc05::ld_32x32b_x32(s_addr + (c ? 0 : 64), v[0]);  // then the first chunk again
                                top = fmaxf(top, tops(v[1], c + 1));
                                tc05::wait_ld(v[0]);
                            }
                            if constexpr (!kBias)
                                top = top == -INFINITY ? top : kCap ? capped(top, p.cap_in, p.cap_log2) : top * p.scale_log2;
                            const bool need = top - m_used > kRoom;
                            if (__any_sync(kFull, need)) {
                                const float m_new = top + p.ref_up;
                                const float alpha = need ? fast_exp2(m_used - m_new) : 1.f;
                                if (need) m_used = m_new;
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
                            const float m = m_used == -INFINITY ? 0.f : m_used;
#pragma unroll 1
                            for (int c = 0; c < 4; c += 2) {
                                uint32_t pk[16];
                                tc05::ld_32x32b_x32(s_addr + 32 * c + 32, v[1]);
                                logits(v[0], c);
                                l += pt_weights<kBF16>(v[0], pk, scale, m);
                                tc05::wait_ld(v[1]);
                                if (c == 0) tc05::ld_32x32b_x32(s_addr + 64, v[0]);
                                tc05::st_32x32b_x16(s_addr + 16 * c, pk);
                                logits(v[1], c + 1);
                                l += pt_weights<kBF16>(v[1], pk, scale, m);
                                tc05::wait_ld(v[0]);
                                tc05::st_32x32b_x16(s_addr + 16 * c + 16, pk);
                            }
                            if (kCap && wide > 0) --wide;
                        }
                        tc05::wait_st();
                        if (!ok) break;
                    }
                    // V rows that no row of the unit sees (stale slots, skipped pages)
                    // are zeroed: their weight 0 must not meet a NaN
                    if (!kFp8 && (kt < zl || kt >= zh) && (lead || j < jb0 || j >= je0)) {
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
                const bool long_sum = je - jb > kPtFold;
                const float folded = long_sum ? fold_factor(fold_row()) : 0.f;
                if (live) {
                    if (!pt_wait(bar(S::B_OF + t), no >> 1 & 1, p)) { ok = false; break; }
                    no += 2;
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
                        if (long_sum) pt_add_folded<32>(o, fold_row() + c / 4 * kPtRows, folded);
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
                    // (both shifts are exact: l's logarithm is taken near 1)
                    const float l2 = l > 0.f ? (m_used - p.ref_up) + __log2f(l * p.ref_pow) : -INFINITY;
                    if (!whole)
                        __stcg(p.part_lse + part0 + row, l2);
                    else if (p.lse)
                        p.lse[row] = l2 * kLn2;
                }
                if (!partials && nsplit > 1) {
                    // publish this tile's part: the four warps' arrivals, one arrival at the unit's
                    // counter with release semantics (cumulative over the stores they ordered before
                    // it), its result back to the four; the arrival that completes the unit merges
                    // its rows.  Bounded waits, as everywhere: a warp that gives up leaves its
                    // siblings no barrier to hang on.
                    const int tok_end = min(I.tok0 + 2 * TOK, n), tiles = I.tok0 + TOK < n ? 2 : 1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(S::B_JA + t));
                    if (q4 == 0) {
                        if (!pt_wait(bar(S::B_JA + t), no & 1, p)) { ok = false; break; }
                        if (lane == 0) {
                            scan[24 + t] = atom_add_acq_rel_gpu(p.counters + I.unit);
                            mbar_arrive(bar(S::B_JD + t));
                        }
                        __syncwarp();
                    }
                    if (!pt_wait(bar(S::B_JD + t), no & 1, p)) { ok = false; break; }
                    no ^= 1;
                    if (scan[24 + t] == nsplit * tiles - 1) {
                        const int rows = (tok_end - I.tok0) * G;
                        const long long step = static_cast<long long>(p.T) * p.Hq;
#pragma unroll 1
                        for (int x = q4; x < rows; x += 4) {
                            const long long mrow = static_cast<long long>(I.q0 + I.tok0 + x / G) * p.Hq + I.hk * G + x % G;
                            float acc[D / 32], mx, ws;
                            merge_row<D>(p.part_lse + mrow, p.part_out + mrow * D, step, nsplit, lane, acc, mx, ws);
                            const float sc = ws > 0.f ? p.v_scale / ws : 0.f;
                            store_row<D>(p.out, mrow, acc, sc, lane, p.out_dtype);
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
    wait_dependency();  // its own end implies that of the launch it overlaps
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
