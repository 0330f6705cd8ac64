// pkd_key_weights on the 5th-generation tensor cores: prompts, whose products bind.
//
// A work item is 256 keys of one (request, kv head) -- two tiles of 128 -- against the
// query rows that see any of them, in tiles of up to 128 rows (TOK = 128 / G whole tokens,
// packed token-major as in the attention kernel).  Per query tile and key tile
//   S^T = K Q^T   tcgen05.mma, M = 128 keys, N = 128 rows, operands K-major as TMA lands them
//   sum           2^(scale s - lse), summed over the columns in registers.  TMEM is read in
//                 pieces of 16 keys x 32 rows whose lanes hold two of every eight rows, for
//                 two keys each: a lane keeps the LSEs of 32 rows, alike for all keys, and
//                 the quad's sums meet at the item's end.  (With a key per lane every lane
//                 needed all LSEs: their loads shared the pipe that TMEM's values come by,
//                 which bound the kernel: 1005 us for 16384 tokens)
// K stays for the whole item and both key tiles share every query tile, so a 128x128
// product costs 16 KB out of L2.  Sums: fp32, of a tile's columns first, in an order fixed by
// the sizes: no atomics on results.
//
// Warp roles (640 threads): warps 0-3 and 4-7 the exponentials of key tile 0 and 1 at even
// steps, 8-15 at odd ones (two S^T buffers a key tile, one for each; all warps at every step,
// on 64 rows each, spent more on waits: 896 us
// for 16384 tokens, not 849 then); warp 16
// loads (items, K, Q), warps 17 and 19 issue the products of key tile 0 and 1 (one warp for
// both left the tensor cores idle between them: its waits and the issue of a product take
// as long as the product), warp 18 lays out the LSEs.  K and Q
// tiles share NU slots: a slot goes to the next tile in the order in which slots become
// free, which is the same for the warp that fills them and the one that reads them (both
// keep the queue of free slots), so short items have all slots in flight and long ones
// NU - 2 query tiles.  Registers follow the roles (640 x 96 at launch = 512 x 104 + 128 x 64).
// Every wait is bounded.
//
// What bounds it, D = 128 (16384-token prompt, 32 heads: 876 us, 1255 TFLOP/s, 0.66 of a dense
// library product): per step of two 128x128 products (1024 cycles) the exponentials take the
// special-function units 1024 cycles, and a warp that is done with an S^T buffer meets
// its next one 650 cycles later -- waits on barriers that answer in 200 to 300 cycles while
// the units' queue is full -- so that neither is busy more than two thirds of the time.
// Products alone ran at 600 us, without exponentials 747.
//
// Few query tiles (two at most) stay in their slots instead, and an item is a run of key
// blocks that stream past them: bound by reading K then (the last 64 of 32768 tokens, four
// heads to a kv head: 34 us with items of one block).
// The exponent is one fused product, scale S - lse log2 e, with the second term rounded to fp32
// once per row, and 2^x the hardware's: off by 2^-24 of |lse log2 e| and by 2^-22.  The tensor
// cores' sums lie towards zero by more than that; the attention kernel's LSE, of the same sums, is
// low by as much (1.1e-6 on average for the last 64 of 32768 tokens), so that beside it the weights
// are off by 7e-7 of their norm, beside an LSE of 64 bits by 1.6e-6.  A row of LSE -inf weighs
// nothing: tiles with one take the masked pass.
// A request's query rows are split between items where its key blocks alone leave SMs
// idle; the sums of the parts are joined in order by the last to arrive.
#pragma once

#include "attend_prompt.cuh"
#include "key_weights.cuh"

namespace pkd {

constexpr int kWtKeys = 256, kWtThreads = 640, kWtItems = 4;
constexpr int kWtRegsExp = 104, kWtRegsOther = 64;  // registers of the exponential warps, of the others

constexpr int kWtStay = 2;        // query tiles that stay in their slots

struct WtItem {
    int b, hk, t0, blocks;        // key blocks from key t0 on
    int first, L, fresh, off;     // row of the first weighing token, whose position is off
    int i0, i1, steps, stay;      // weighing tokens [i0, i1), in tiles of TOK; stay: in their slots for all blocks
    int split, nsplit, unit;      // parts of the unit that hold any
    int end;
};

template <int D, int kType>
struct WtShape {
    static constexpr bool FP8 = kType == kPtFP8;
    static constexpr int ROWB = D * (FP8 ? 1 : 2), REGIONS = ROWB / 128, GROUP = 8 * ROWB;
    static constexpr int UNIT = 128 * ROWB;
    static constexpr int NU = UNIT == 32768 ? 6 : 12;
    static constexpr int OFF_LSE = NU * UNIT;
    static constexpr int OFF_SUM = OFF_LSE + 2 * 128 * 4;  // a block's sums of odd steps, for the warps of even ones
    static constexpr int OFF_NONE = OFF_SUM + kWtKeys * 4;  // per buffer of LSEs: some token's is -inf
    static constexpr int OFF_ITEM = OFF_NONE + 2 * 4;
    static constexpr int OFF_PREF = OFF_ITEM + kWtItems * static_cast<int>(sizeof(WtItem));
    static constexpr int OFF_SCAN = OFF_PREF + (kPtMaxBatch + 4) * 4;
    static constexpr int OFF_BAR = (OFF_SCAN + 128 + 7) & ~7;
    // slots full/empty, S full/empty [key tile][buffer], LSEs empty [buffer], items full/empty,
    // sums full/empty per 32 keys, drain
    static constexpr int B_UF = 0, B_UE = B_UF + NU, B_SF = B_UE + NU, B_SE = B_SF + 4, B_LE = B_SE + 4;
    static constexpr int B_IF = B_LE + 2, B_IE = B_IF + kWtItems, B_XF = B_IE + kWtItems;
    static constexpr int B_XE = B_XF + 8, B_DR = B_XE + 8;
    static constexpr int NBAR = B_DR + 2;
    static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_TMEM + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
    static_assert(SMEM > 114 * 1024, "one CTA per SM: all 512 TMEM columns are its own");
    static_assert(NU <= 15, "the queue of free slots holds 16 of four bits");
};

// Block k of an item: its first key, key tiles, and query tiles (none where no token sees a key).
struct WtBlock {
    int t0, nk, steps;
};
__device__ __forceinline__ WtBlock wt_block(const AttendParams& p, const WtItem& I, int k) {
    WtBlock x;
    x.t0 = I.t0 + k * kWtKeys;
    const int t1 = min(x.t0 + kWtKeys, I.L);
    x.nk = t1 - x.t0 > 128 ? 2 : 1;
    x.steps = I.steps;
    if (I.stay && ((p.causal && x.t0 - I.off >= I.i1) ||
                   (p.window > 0 && static_cast<long long>(t1 - 1) - I.off + p.window <= I.i0)))
        x.steps = 0;
    return x;
}

// The queue of free slots, four bits each, the next one lowest.
struct WtSlots {
    uint64_t queue;
    int n;
    __device__ __forceinline__ explicit WtSlots(int slots) : queue(0xfedcba9876543210ull), n(slots) {}
    __device__ __forceinline__ int take() {
        const int s = static_cast<int>(queue & 15);
        queue >>= 4;
        --n;
        return s;
    }
    __device__ __forceinline__ void give(int s) {
        queue = (queue & ~(15ull << (4 * n))) | static_cast<uint64_t>(s) << (4 * n);
        ++n;
    }
};

// 16 capped logits in log2 units: by the polynomial, or (far) by exponential and reciprocal.
__device__ __forceinline__ void wt_cap(uint32_t (&v)[16], const AttendParams& p, bool far) {
    if (far) {
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = __float_as_uint(capped(__uint_as_float(v[c]), p.cap_in, p.cap_log2));
        return;
    }
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
        const float2 x = make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), z = mul2(x, x);
        float2 t = fma2(z, both(p.cap_c[4]), both(p.cap_c[3]));
        t = fma2(z, t, both(p.cap_c[2]));
        t = fma2(z, t, both(p.cap_c[1]));
        t = mul2(fma2(z, t, both(p.cap_c[0])), x);
        v[c] = __float_as_uint(t.x);
        v[c + 1] = __float_as_uint(t.y);
    }
}

// 16 lanes x 32 columns of TMEM: lane i gets columns 8 k + 2 (i % 4) and the next of row
// i / 4 (r[4 k], r[4 k + 1]) and of row i / 4 + 8 (r[4 k + 2], r[4 k + 3]).
__device__ __forceinline__ void wt_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Wait for this warp's TMEM loads, with the loaded registers passed through.
__device__ __forceinline__ void wt_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

template <int D, int kType, bool kCap>
__global__ void __launch_bounds__(kWtThreads, 1)
key_weights_tc05_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                        const WeighParams w) {
    using S = WtShape<D, kType>;
    constexpr bool kFp8 = kType == kPtFP8;
    const AttendParams& p = w.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb0 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    WtItem* items = reinterpret_cast<WtItem*>(smem + S::OFF_ITEM);
    int* pref = reinterpret_cast<int*>(smem + S::OFF_PREF);
    int* scan = reinterpret_cast<int*>(smem + S::OFF_SCAN);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + S::OFF_TMEM);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.G, TOK = kPtRows / G;
    auto bar = [&](int i) { return smem_u32(bars + i); };

    // ------------------------------------------------------------ set-up
    if (tid == 0) {
        for (int i = 0; i < S::NU; ++i) {
            mbar_init(bar(S::B_UF + i), 1);
            mbar_init(bar(S::B_UE + i), 2);  // both issuing warps
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(S::B_SF + i), 2);  // the product, and the rows' LSEs
            mbar_init(bar(S::B_SE + i), 4);
        }
        for (int i = 0; i < 2; ++i) mbar_init(bar(S::B_LE + i), 8);
        for (int i = 0; i < kWtItems; ++i) {
            mbar_init(bar(S::B_IF + i), 1);
            mbar_init(bar(S::B_IE + i), 19);  // the issuing, LSE and sixteen exponential warps
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(bar(S::B_XF + i), 1);
            mbar_init(bar(S::B_XE + i), 1);
        }
        mbar_init(bar(S::B_DR), 1);
        mbar_init(bar(S::B_DR + 1), 1);
        fence_barrier_init();
    }
    if (warp == 17) {
        tc05::alloc(smem_u32(tslot), 512);  // S^T of (key tile, buffer): columns 128 * (2 * tile + buffer)
        tc05::relinquish_alloc_permit();
    }
    // prefix of the requests' runs of key blocks (units of one kv head)
    {
        int run = 0;
        for (int b0 = 0; b0 < p.B; b0 += kWtThreads) {
            const int b = b0 + tid;
            int v = b < p.B ? (request_len(p, b, blockIdx.x == 0) + kWtKeys - 1) / kWtKeys : 0;
            v = (v + w.run - 1) / w.run;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, v, o);
                if (lane >= o) v += y;
            }
            if (lane == 31) scan[warp] = v;
            __syncthreads();
            int before = run;
            for (int k = 0; k < kWtThreads / 32; ++k) {
                if (k < warp) before += scan[k];
                run += scan[k];
            }
            if (b < p.B) pref[b + 1] = before + v;
            __syncthreads();
        }
        if (tid == 0) pref[0] = scan[24] = 0;
    }
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tmem = *tslot;

    if (warp == 16) {
        reg_dec<kWtRegsOther>();
        // ---------------------------------------------------------- loads
        if (lane == 0) {
            prefetch_tmap(&kvmap);
            prefetch_tmap(&qmap);
        }
        const uint64_t pol = policy_evict_first();
        uint64_t keep;  // other items read the same queries
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
        const int units = pref[p.B] * p.Hkv, total = units * p.max_splits;
        WtSlots slots(S::NU);
        uint32_t phase = 0, used = 0;  // of each slot
        int idx = blockIdx.x, npub = 0;
        bool ok = true;
        // the slot of the next tile, empty
        auto take = [&]() {
            const int s = slots.take();
            ok = pt_wait(bar(S::B_UE + s), (phase >> s & 1) ^ 1, p);
            if (ok) phase ^= 1u << s, used |= 1u << s;
            return s;
        };
        const bool queued = total > static_cast<int>(gridDim.x);  // else: an item per CTA
        while (ok) {
            const int ring = npub % kWtItems;
            if (npub >= kWtItems && !pt_wait(bar(S::B_IE + ring), ((npub / kWtItems) - 1) & 1, p)) { ok = false; break; }
            if (idx >= total) {
                if (lane == 0) {
                    items[ring].end = 1;
                    mbar_arrive(bar(S::B_IF + ring));
                }
                __syncwarp();
                break;
            }
            int next = total;
            if (queued && lane == 0) next = static_cast<int>(gridDim.x) + atomicAdd(p.queue, 1);
            // item idx: parts innermost, then kv heads, the key blocks of a request from the
            // first (causal: seen by the most tokens)
            const int split = idx % p.max_splits, u = idx / p.max_splits;
            const int b = pt_request(pref, p.B, p.Hkv, u), r = u - pref[b] * p.Hkv;
            const int hk = r % p.Hkv, t0 = r / p.Hkv * w.run * kWtKeys;
            const WeighRequest q = weigh_request(w, b, r == 0 && split == 0 && lane == 0);
            const int t1 = min(t0 + w.run * kWtKeys, q.L), off = q.L - q.m;
            // tokens that see any of the keys: from the first key's position on, up to a
            // window behind the last key
            int i0 = p.causal ? max(0, t0 - off) : 0, i1 = q.m, nsplit = 0;
            if (p.window > 0) i1 = static_cast<int>(min(static_cast<long long>(q.m), static_cast<long long>(t1 - 1) - off + p.window));
            if (i0 < i1) {
                // parts begin at multiples of their size behind i0
                nsplit = min((i1 - i0 + p.chunk - 1) / p.chunk, p.max_splits);
                i0 += split * p.chunk;
                if (split + 1 < nsplit) i1 = min(i1, i0 + p.chunk);
            }
            if (split >= max(nsplit, 1)) {  // nothing here
                idx = __shfl_sync(kFull, next, 0);
                continue;
            }
            WtItem I;
            I.b = b; I.hk = hk; I.t0 = t0; I.blocks = (t1 - t0 + kWtKeys - 1) / kWtKeys;
            I.first = q.first; I.L = q.L; I.fresh = q.fresh; I.off = off;
            I.i0 = i0; I.i1 = i1; I.steps = nsplit ? (i1 - i0 + TOK - 1) / TOK : 0; I.stay = w.stay;
            I.split = split; I.nsplit = nsplit; I.unit = u; I.end = 0;
            if (lane == 0) {
                items[ring] = I;
                mbar_arrive(bar(S::B_IF + ring));
            }
            __syncwarp();
            ++npub;
            // the page of a block's 16-key stage, a lane each (asked for a block ahead, and looked
            // at where it is used), and its cache row; -1: no key, or none in the pool
            auto stage_key = [&](int k) { return t0 + k * kWtKeys + kStageTok * lane; };
            auto stage_page = [&](int k) {
                if (k >= I.blocks || lane >= kWtKeys / kStageTok || stage_key(k) >= t1) return 0;
                return p.block_table[static_cast<long long>(b) * p.bt_stride + page_div(stage_key(k), p.pmagic, p.pmshift)];
            };
            auto stage_row = [&](int k, int page) {
                const int t = stage_key(k);
                if (lane >= kWtKeys / kStageTok || t >= t1) return -1;
                if (page < 0 || page >= p.num_pages) {
                    atomicOr(p.status, kErrBounds);
                    scan[24] = 1;
                    return -1;
                }
                return (page * p.Hkv + hk) * p.P + (t - page_div(t, p.pmagic, p.pmshift) * p.P);
            };
            int page = stage_page(0), qs[kWtStay] = {0, 0};
            bool have = false;
#pragma unroll 1
            for (int k = 0; ok && k < I.blocks; ++k) {
                const int page_next = stage_page(k + 1);
                const WtBlock x = wt_block(p, I, k);
                if (x.steps) {
                    auto load_q = [&](int s, int j) {
                        if (lane == 0) mbar_arrive_expect_tx(bar(S::B_UF + s), S::REGIONS * TOK * G * 128);
                        __syncwarp();
                        if (lane < S::REGIONS)
                            tma_load_3d(sb0 + s * S::UNIT + lane * kPtRows * 128, &qmap, 64 * lane, hk * G, q.first + i0 + j * TOK,
                                        bar(S::B_UF + s), keep);
                    };
                    if (I.stay && !have) {
#pragma unroll
                        for (int j = 0; j < kWtStay; ++j) {
                            if (j >= x.steps || !ok) continue;
                            qs[j] = take();
                            if (ok) load_q(qs[j], j);
                        }
                        have = true;
                    }
                    const int krow = stage_row(k, page);
                    __syncwarp();  // scan[24] before lane 0's arrival
                    int ks[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e >= x.nk || !ok) continue;
                        ks[e] = take();
                        if (!ok) continue;
                        const bool load = krow >= 0 && (lane >> 3) == e;
                        const int bytes = __popc(__ballot_sync(kFull, load)) * 2 * S::GROUP;
                        if (lane == 0) mbar_arrive_expect_tx(bar(S::B_UF + ks[e]), bytes);
                        __syncwarp();
                        if (load)
                            tma_load_4d(sb0 + ks[e] * S::UNIT + 2 * (lane & 7) * S::GROUP, &kvmap, 0, 0, 0, krow >> 3,
                                        bar(S::B_UF + ks[e]), pol);
                    }
#pragma unroll 1
                    for (int j = 0; ok && !I.stay && j < x.steps; ++j) {
                        const int s = take();
                        if (!ok) break;
                        load_q(s, j);
                        slots.give(s);
                    }
                    slots.give(ks[0]);
                    if (x.nk > 1) slots.give(ks[1]);
                }
                page = page_next;
            }
            if (have)
#pragma unroll
                for (int j = 0; j < kWtStay; ++j)
                    if (j < I.steps) slots.give(qs[j]);
            idx = __shfl_sync(kFull, next, 0);
        }
        // let every issued copy land before the CTA leaves
        for (int s = 0; s < S::NU; ++s)
            if (used >> s & 1) mbar_wait(bar(S::B_UF + s), (phase >> s & 1) ^ 1);
        if (!ok && lane == 0) atomicOr(p.status, kErrTimeout);
    } else if (warp == 17 || warp == 19) {
        reg_dec<kWtRegsOther>();
        // ------------------------------------------- products of key tile t
        constexpr uint32_t kId = kFp8 ? tc05::idesc_e4m3(128, 128) : tc05::idesc_f16(kType == kPtBF16, 128, 128, false, false);
        const int t = (warp - 17) >> 1;
        const bool one = tc05::elect_one();
        const uint32_t tm = tc05::uniform(tmem + 256 * t), lo0 = tc05::uniform(tc05::desc_lo(sb0, 16));
        WtSlots slots(S::NU);
        uint32_t phase = 0, sphase = 0;  // of the slots, of the S^T buffers
        int step = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int ring = it % kWtItems;
            if (!pt_wait(bar(S::B_IF + ring), (it / kWtItems) & 1, p)) { ok = false; break; }
            const WtItem& I = items[ring];
            if (I.end) break;
            const int blocks = I.blocks, tiles = I.steps;
            const bool stay = I.stay;
            bool have = false;
            int qs[kWtStay] = {0, 0};
#pragma unroll 1
            for (int k = 0; ok && k < blocks; ++k) {
                const WtBlock x = wt_block(p, I, k);
                if (!x.steps) continue;
                const bool fresh = stay && !have;
                if (fresh) {
#pragma unroll
                    for (int j = 0; j < kWtStay; ++j)
                        if (j < tiles) qs[j] = slots.take();
                    have = true;
                }
                const int k0 = slots.take(), k1 = x.nk > 1 ? slots.take() : -1;
                const int mine = t == 0 ? k0 : k1;
                // both tiles: this warp releases both slots, and only what was filled may be released
                ok = pt_wait(bar(S::B_UF + k0), phase >> k0 & 1, p) && (k1 < 0 || pt_wait(bar(S::B_UF + k1), phase >> k1 & 1, p));
                const uint32_t klo = tc05::uniform(lo0 + ((mine < 0 ? 0 : mine) * S::UNIT >> 4));
                phase ^= 1u << k0;
                if (k1 >= 0) phase ^= 1u << k1;
#pragma unroll 1
                for (int j = 0; ok && j < x.steps; ++j, ++step) {
                    const int s = stay ? qs[j & 1] : slots.take(), buf = step & 1;
                    if (!stay || fresh) {
                        ok = pt_wait_queries(bar(S::B_UF + s), phase >> s & 1, p, it);
                        phase ^= 1u << s;
                    }
                    // (a block without a second key tile goes through all of the second one's
                    // barriers, with nothing in them: what its warps wait for is then always
                    // their own.  They once waited for the first tile's instead, whose phase of
                    // two steps before they could take for the one to come)
                    ok = ok && pt_wait(bar(S::B_SE + 2 * t + buf), (sphase >> buf & 1) ^ 1, p);
                    if (!ok) break;
                    sphase ^= 1u << buf;
                    if (mine >= 0) {
                        tc05::fence_after_sync();
                        const uint32_t qlo = tc05::uniform(lo0 + (s * S::UNIT >> 4)), d = tm + 128 * buf;
#pragma unroll
                        for (int kk = 0; kk < S::ROWB / 32; ++kk)
                            if (one)
                                tc05::mma_ss<kFp8>(d, klo + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), tc05::desc_hi(S::GROUP),
                                                   qlo + (((kk >> 2) * kPtRows * 128 + (kk & 3) * 32) >> 4), tc05::desc_hi(1024), kId,
                                                   kk > 0);
                    }
                    if (one) tc05::commit(bar(S::B_SF + 2 * t + buf));
                    if (!stay) {
                        if (one) tc05::commit(bar(S::B_UE + s));
                        slots.give(s);
                    }
                }
                if (ok && one) {
                    tc05::commit(bar(S::B_UE + k0));
                    if (k1 >= 0) tc05::commit(bar(S::B_UE + k1));
                }
                slots.give(k0);
                if (k1 >= 0) slots.give(k1);
            }
            if (have)
#pragma unroll
                for (int j = 0; j < kWtStay; ++j)
                    if (j < tiles) {
                        if (ok && one) tc05::commit(bar(S::B_UE + qs[j]));
                        slots.give(qs[j]);
                    }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S::B_IE + ring));
        }
        if (!ok && one) atomicOr(p.status, kErrTimeout);
        // every product issued has completed before TMEM is freed
        if (one) {
            tc05::commit(bar(S::B_DR + t));
            mbar_wait(bar(S::B_DR + t), 0);
        }
        __syncwarp();
    } else if (warp == 18) {
        reg_dec<kWtRegsOther>();
        // ------------------------------------- the rows' LSEs, as added to logits
        float* lse2 = reinterpret_cast<float*>(smem + S::OFF_LSE);
        int* none = reinterpret_cast<int*>(smem + S::OFF_NONE);
        int nl = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int ring = it % kWtItems;
            if (!pt_wait(bar(S::B_IF + ring), (it / kWtItems) & 1, p)) { ok = false; break; }
            const WtItem& I = items[ring];
            if (I.end) break;
            const int i0 = I.i0, i1 = I.i1;
            const float* lse = w.lse + static_cast<long long>(I.first) * p.Hq + I.hk * G;
            int tok[4], col[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = 4 * lane + e;
                tok[e] = c / G;
                col[e] = tok[e] < TOK ? c - tok[e] * G : -1;
            }
            auto load = [&](int j, float (&x)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + j * TOK + tok[e];
                    x[e] = col[e] >= 0 && i < i1 ? lse[static_cast<long long>(i) * p.Hq + col[e]] : -INFINITY;
                }
            };
            float x[4];
            if (I.steps) load(0, x);
#pragma unroll 1
            for (int k = 0; ok && k < I.blocks; ++k) {
                const int steps = wt_block(p, I, k).steps;
#pragma unroll 1
                for (int j = 0; j < steps; ++j, ++nl) {
                    const int buf = nl & 1;
                    bool dead = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) dead |= x[e] == -INFINITY && col[e] >= 0 && i0 + j * TOK + tok[e] < i1;
                    dead = __any_sync(kFull, dead);
                    float4 v;
                    v.x = x[0] == -INFINITY ? x[0] : -kLog2e * x[0];
                    v.y = x[1] == -INFINITY ? x[1] : -kLog2e * x[1];
                    v.z = x[2] == -INFINITY ? x[2] : -kLog2e * x[2];
                    v.w = x[3] == -INFINITY ? x[3] : -kLog2e * x[3];
                    if (steps > 1) load(j + 1 < steps ? j + 1 : 0, x);
                    if (!pt_wait(bar(S::B_LE + buf), ((nl >> 1) & 1) ^ 1, p)) { ok = false; break; }
                    *reinterpret_cast<float4*>(lse2 + 128 * buf + 4 * lane) = v;
                    if (lane == 0) none[buf] = dead;
                    __syncwarp();
                    // (the last step's with this buffer is over: all its readers have said so)
                    if (lane < 2) mbar_arrive(bar(S::B_SF + 2 * lane + buf));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S::B_IE + ring));
        }
        if (!ok && lane == 0) atomicOr(p.status, kErrTimeout);
    } else {
        reg_inc<kWtRegsExp>();
        // --------------------------------------------------- exponentials
        const int odd = warp >> 3, tile = (warp >> 2) & 1, q4 = warp & 3, pair = warp & 7, g = lane >> 2, c4 = lane & 3;
        const uint32_t s_addr = tmem + (static_cast<uint32_t>(32 * q4) << 16) + 128 * (2 * tile + odd);
        const float* lse2 = reinterpret_cast<const float*>(smem + S::OFF_LSE) + 128 * odd + 2 * c4;
        const int* none = reinterpret_cast<const int*>(smem + S::OFF_NONE) + odd;
        // lane (g, c4) ends up with the sum of key 8 c4 + g of its warp's 32
        float* sum = reinterpret_cast<float*>(smem + S::OFF_SUM) + 32 * pair + 8 * c4 + g;
        const float scale = kCap ? 1.f : p.scale_log2;
        const int rows = TOK * G;
        int step = 0;                 // steps before the item
        uint32_t phase = 0;           // of this key tile's S (bit 0), of the sums (bit 1)
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int ring = it % kWtItems;
            if (!pt_wait(bar(S::B_IF + ring), (it / kWtItems) & 1, p)) { ok = false; break; }
            const WtItem& I = items[ring];
            if (I.end) break;
            const int i0 = I.i0, i1 = I.i1, L = I.L, off = I.off;
#pragma unroll 1
            for (int kb = 0; ok && kb < I.blocks; ++kb) {
                const WtBlock x = wt_block(p, I, kb);
                const int steps = x.steps, k0 = x.t0 + 32 * pair;
                const bool active = tile < x.nk;
                // the earlier weight of this lane's key comes near while the block is weighed
                // (in a register all the while it cost a spill)
                const int key = k0 + 8 * c4 + g;
                if (!odd && w.prior && key < min(L, I.fresh))
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(w.prior + I.b * w.prior_b + I.hk * w.prior_h + key));
                // tokens [lo, hi) see a key
                auto lo_of = [&](int key) { return p.causal ? max(i0, key - off) : i0; };
                auto hi_of = [&](int key) {
                    return p.window > 0 ? static_cast<int>(min(static_cast<long long>(i1), static_cast<long long>(key) - off + p.window)) : i1;
                };
                // every key of the warp is seen by [wlo, whi)
                const int wlo = lo_of(min(k0 + 31, L - 1)), whi = hi_of(min(k0, L - 1));
                float total[2][2] = {};  // of 16 keys, 8 keys
#pragma unroll 1
                for (int j = (odd - step) & 1; j < steps; j += 2) {
                    const int a = i0 + j * TOK;
                    if (!pt_wait(bar(S::B_SF + 2 * tile + odd), phase & 1, p)) { ok = false; break; }
                    phase ^= 1u;
                    float2 n[16];  // LSEs of rows 8 k + 2 c4 and the next
#pragma unroll
                    for (int k = 0; k < 16; ++k) n[k] = *reinterpret_cast<const float2*>(lse2 + 8 * k);
                    const bool dead = *none;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(S::B_LE + odd));
                    if (active) {
                        tc05::fence_after_sync();
                        float2 acc[2][2] = {};  // of 16 keys, 8 keys
                        auto piece = [&](uint32_t (&x)[16], int hl, int cc, auto select) {
                            // columns [c0, c1) see the lane's two keys
                            int c0[2] = {0, 0}, c1[2] = {0, 0};
                            if constexpr (decltype(select)::value) {
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    const int key = k0 + 16 * hl + 8 * r + g;
                                    c0[r] = min(max(lo_of(key) - a, 0), TOK) * G;
                                    c1[r] = key < L ? min(max(hi_of(key) - a, 0), TOK) * G : c0[r];
                                }
                            }
                            // a token of LSE -inf weighs nothing, whatever its q holds (padding may hold
                            // NaN, which adding -inf would keep)
                            if constexpr (decltype(select)::value) {
                                if (dead) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const float2 m = n[4 * cc + (e >> 2)];
                                        if ((e & 1 ? m.y : m.x) == -INFINITY) x[e] = 0u;
                                    }
                                }
                            }
                            if constexpr (kCap) {
                                // products of keys behind the last, or of no row, hold what was left in
                                // shared memory: they have no say in the vote, or the roundings of the
                                // others would depend on it
                                if constexpr (decltype(select)::value) {
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const int r = (e >> 1) & 1, c = 32 * cc + 8 * (e >> 2) + 2 * c4 + (e & 1);
                                        if (c < c0[r] || c >= c1[r]) x[e] = 0u;
                                    }
                                }
                                float top = 0.f;
#pragma unroll
                                for (int e = 0; e < 16; e += 2) top = max3(top, fabsf(__uint_as_float(x[e])), fabsf(__uint_as_float(x[e + 1])));
                                wt_cap(x, p, __any_sync(kFull, top > p.cap_far));
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    float2 y = fma2(make_float2(__uint_as_float(x[4 * k + 2 * r]), __uint_as_float(x[4 * k + 2 * r + 1])),
                                                    both(scale), n[4 * cc + k]);
                                    y.x = fast_exp2(y.x);
                                    y.y = fast_exp2(y.y);
                                    if constexpr (decltype(select)::value) {
                                        const int c = 32 * cc + 8 * k + 2 * c4;
                                        y.x = c >= c0[r] && c < c1[r] ? y.x : 0.f;
                                        y.y = c + 1 >= c0[r] && c + 1 < c1[r] ? y.y : 0.f;
                                    }
                                    acc[hl][r] = add2(acc[hl][r], y);
                                }
                            }
                        };
                        // piece u: 16 keys (u & 1), 32 rows (u >> 1)
                        auto at = [&](int u) { return s_addr + (static_cast<uint32_t>(16 * (u & 1)) << 16) + 32 * (u >> 1); };
                        if (wlo <= a && whi >= a + TOK && rows == 128 && !dead && (!kCap || k0 + 32 <= L)) {
                            uint32_t v[2][16];
                            wt_ld(at(0), v[0]);
                            wt_wait_ld(v[0]);
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                if (u < 7) wt_ld(at(u + 1), v[(u + 1) & 1]);
                                piece(v[u & 1], u & 1, u >> 1, std::false_type{});
                                if (u < 7) wt_wait_ld(v[(u + 1) & 1]);
                            }
                        } else {
                            const int cols = min(TOK, i1 - a) * G;
#pragma unroll
                            for (int u = 0; u < 8; ++u) {
                                if (32 * (u >> 1) >= cols) continue;
                                uint32_t v[16];
                                wt_ld(at(u), v);
                                wt_wait_ld(v);
                                piece(v, u & 1, u >> 1, std::true_type{});
                            }
                        }
                        tc05::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(S::B_SE + 2 * tile + odd));
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                            for (int r = 0; r < 2; ++r) total[hl][r] += acc[hl][r].x + acc[hl][r].y;
                    } else if (lane == 0) {
                        mbar_arrive(bar(S::B_SE + 2 * tile + odd));
                    }
                }
                if (!ok) break;
                step += steps;
                if (active) {
#pragma unroll
                    for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            total[hl][r] += __shfl_xor_sync(kFull, total[hl][r], 1);
                            total[hl][r] += __shfl_xor_sync(kFull, total[hl][r], 2);
                        }
                    float mine = c4 == 0 ? total[0][0] : c4 == 1 ? total[0][1] : c4 == 2 ? total[1][0] : total[1][1];
                    if (steps && odd) {
                        if (!pt_wait(bar(S::B_XE + pair), (phase >> 1) ^ 1, p)) { ok = false; break; }
                        *sum = mine;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(S::B_XF + pair));
                    } else if (steps) {
                        if (!pt_wait(bar(S::B_XF + pair), phase >> 1, p)) { ok = false; break; }
                        mine += *sum;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(S::B_XE + pair));
                    }
                    if (steps) phase ^= 2u;
                    if (!odd) {
                        bool whole = true;
                        if (I.nsplit > 1) {
                            // the unit's parts, joined in order by the warp whose arrival is the last
                            float* part = p.part_out + static_cast<long long>(I.unit) * p.max_splits * kWtKeys + (key - x.t0);
                            __stcg(part + I.split * kWtKeys, mine);
                            __syncwarp();
                            int prev = 0;
                            if (lane == 0) prev = atom_add_acq_rel_gpu(p.counters + 8 * I.unit + pair);
                            prev = __shfl_sync(kFull, prev, 0);
                            __syncwarp();  // lane 0's acquire comes before all lanes' reads of the other parts
                            whole = prev == I.nsplit - 1;
                            if (whole) {
                                mine = 0.f;
                                for (int s = 0; s < I.nsplit; ++s) mine += __ldcg(part + s * kWtKeys);
                                if (lane == 0) p.counters[8 * I.unit + pair] = 0;  // ready for the next call
                            }
                        }
                        if (whole && key < L) {
                            if (scan[24]) {  // a page outside the pool was not loaded
                                const int page = p.block_table[static_cast<long long>(I.b) * p.bt_stride + page_div(key, p.pmagic, p.pmshift)];
                                if (page < 0 || page >= p.num_pages) mine = 0.f;
                            }
                            const float before = w.prior && key < I.fresh ? w.prior[I.b * w.prior_b + I.hk * w.prior_h + key] : 0.f;
                            w.weights[I.b * w.weights_b + I.hk * w.weights_h + key] = fmaf(w.decay, before, mine);
                        }
                    }
                }
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(S::B_IE + ring));
        }
        if (!ok && lane == 0) atomicOr(p.status, kErrTimeout);
    }

    // ---------------------------------------------------------- tear-down
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == 17) {
        tc05::fence_after_sync();
        tc05::dealloc(tmem, 512);
    }
    // the last CTA to leave resets the item counter for the next call
    if (tid == 0 && pref[p.B] * p.Hkv * p.max_splits > static_cast<int>(gridDim.x)) {
        const int prev = atom_add_acq_rel_gpu(p.queue + 1);
        if (prev == static_cast<int>(gridDim.x) - 1) {
            p.queue[0] = 0;
            p.queue[1] = 0;
        }
    }
}

}  // namespace pkd
