// pkd_key_weights on mma.sync: steps of few query rows per kv head, bound by reading K.
//
// A warp takes 16 keys of one kv head at a time: D[key, row] = K q^T on m16n8k16 (e4m3:
// m16n8k32) products, the keys as the A operand straight from global memory.  A dot
// product does not care for the order of its dims, so a lane loads 16 consecutive bytes
// of two key rows (a quad: 64, a load instruction 8 x 64 bytes, whole sectors) and takes
// its four words as the operands of two k-steps; q is loaded in the same order.  On their
// way the keys wait in a ring of kKwStages steps in shared memory (cp.async), where a lane
// finds the bytes that it copied itself: no barrier and no swizzle.  Then exp2(logit - lse),
// the sum over a lane's rows and over its quad, and one 4-byte store per key.
//
// What bounds it (64 requests of 1024 to 4096 keys, 8 kv heads, bf16: 54 us, 5.7 TB/s of the
// copy's 6.8; 4 contexts of up to 131072 keys, e4m3, 8 rows: 64 us, 5.5 TB/s): a warp's step
// is a chain of products, exponentials and votes of its quad, and a CTA's first keys wait
// for two trips to memory, so that warps in number count for more than bytes in flight:
// twenty warps of two stages each, not eight of six (78 us), with the table asked for
// before the lengths.  Keys in registers, two steps ahead: 54 and 70 us.  Earlier weights
// are asked for two steps ahead (loaded where they are added: 75 us in e4m3).
#include "attend_launch.h"
#include "key_weights.cuh"

namespace pkd {

constexpr int kKwWarps = 4;
constexpr int kKwStages = 2, kKwCtas = 5;  // steps of a warp's ring (4 KB each), CTAs of an SM
constexpr int kKwSmem = kKwWarps * kKwStages * 4096;

__device__ __forceinline__ void kw_copy(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int kType>
__device__ __forceinline__ void kw_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    const uint32_t a[4] = {a0, a1, a2, a3};
    if constexpr (kType == 2)
        mma16832_e4m3(d, a, b0, b1);
    else
        mma16816<kType == 0>(d, a, b0, b1);
}

// kType: 0 bf16, 1 fp16, 2 e4m3.  NT: tiles of 8 rows, whose q stays in registers.
template <int D, int kType, int NT, bool kCap>
__global__ void __launch_bounds__(32 * kKwWarps, kKwCtas) key_weights_kernel(const WeighParams w) {
    constexpr int ROWB = D * (kType == 2 ? 1 : 2), C = ROWB / 64;  // 64-byte chunks of a row
    constexpr int U = 256 / ROWB;                                  // 16-key groups of a step: 8 loads per lane
    const AttendParams& p = w.a;
    const int b = blockIdx.z, hk = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q4 = lane & 3;
    // a lane keeps the page of one 16-key group of its warp's share (at most 32).  Asked for
    // before the request's length is known (the table has a column for it): one trip to
    // memory less before the first keys
    const int k0 = blockIdx.x * p.chunk;
    const int32_t* table = p.block_table + static_cast<long long>(b) * p.bt_stride;
    const int my_key = k0 + 16 * ((lane / U) * kKwWarps * U + warp * U + lane % U);
    int my_page = -1;
    if (my_key < min(k0 + p.chunk, p.max_kv_len)) my_page = table[page_div(my_key, p.pmagic, p.pmshift)];
    const WeighRequest r = weigh_request(w, b, blockIdx.x == 0 && hk == 0 && threadIdx.x == 0);
    const int k1 = min(k0 + p.chunk, r.L);
    if (k0 >= k1) return;
    const int rows = r.m * p.G, steps = (k1 - k0 + 16 * U - 1) / (16 * U);
    if (my_key >= k1) {
        my_page = -1;
    } else if (my_page < 0 || my_page >= p.num_pages) {
        my_page = -1;
        atomicOr(p.status, kErrBounds);
    }

    // q of the rows, as B operands, with their LSE and the keys that they see
    uint32_t bq[NT][4 * C];
    float lse2[NT][2];
    int lo[NT][2], hi[NT][2];  // none where there is no row, or its LSE says so
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = 8 * n + g;
        const int i = c / p.G;
        const uint8_t* row = static_cast<const uint8_t*>(p.q) +
                             (static_cast<long long>(r.first + i) * p.q_stride + (hk * p.G + c - i * p.G) * D) *
                                 (ROWB / D);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (c < rows) x = __ldg(reinterpret_cast<const uint4*>(row + 64 * j + 16 * q4));
            bq[n][4 * j] = x.x; bq[n][4 * j + 1] = x.y; bq[n][4 * j + 2] = x.z; bq[n][4 * j + 3] = x.w;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = 8 * n + 2 * q4 + e, tok = col / p.G;
            const int pos = r.L - r.m + tok;
            float x = -INFINITY;
            if (col < rows) x = w.lse[static_cast<long long>(r.first + tok) * p.Hq + hk * p.G + col - tok * p.G];
            lse2[n][e] = x * kLog2e;
            lo[n][e] = p.window > 0 ? pos - p.window + 1 : 0;
            hi[n][e] = x == -INFINITY ? 0 : p.causal ? pos + 1 : r.L;
        }
    }

    extern __shared__ __align__(16) uint8_t ring[];
    const uint8_t* bytes = ring + warp * (kKwStages * 4096) + 16 * lane;  // this lane's bytes: every 512
    const uint32_t bytes_at = smem_u32(bytes);
    auto page_of = [&](int s, int u) { return __shfl_sync(kFull, my_page, (s / kKwWarps * U + u) & 31); };
    auto copy_keys = [&](int s, int slot) {
        if (s < steps)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = k0 + 16 * (s * U + u), page = page_of(s, u);
                if (page < 0) continue;
                const int in_page = t - page_div(t, p.pmagic, p.pmshift) * p.P;
                const uint8_t* row = w.cache + (static_cast<long long>(page * p.Hkv + hk) * p.P + in_page + g) * (2 * ROWB) + 16 * q4;
                const uint32_t dst = bytes_at + slot * 4096 + u * (4096 / U);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    kw_copy(dst + 1024 * j, row + 64 * j);
                    kw_copy(dst + 1024 * j + 512, row + 64 * j + 8 * 2 * ROWB);
                }
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto prior_of = [&](int s, float (&x)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = k0 + 16 * (s * U + u) + g + 8 * q4;
            x[u] = 0.f;
            if (w.prior && q4 < 2 && key < min(k1, r.fresh)) x[u] = w.prior[b * w.prior_b + hk * w.prior_h + key];
        }
    };
    auto weigh = [&](int s, int slot, const float (&before)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = k0 + 16 * (s * U + u);
            if (t >= k1) continue;
            // this lane stores key t + g + 8 * q4 (q4 < 2)
            const int mine = t + g + 8 * q4;
            const bool store = q4 < 2 && mine < k1;
            float sum[2] = {0.f, 0.f};
            if (page_of(s, u) >= 0) {
                uint4 ka[C][2];
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    ka[j][0] = *reinterpret_cast<const uint4*>(bytes + slot * 4096 + u * (4096 / U) + 1024 * j);
                    ka[j][1] = *reinterpret_cast<const uint4*>(bytes + slot * 4096 + u * (4096 / U) + 1024 * j + 512);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // two chains of products: one alone is as long as a step takes
                    float d[4] = {0.f, 0.f, 0.f, 0.f}, d2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        const uint4 x = ka[j][0], y = ka[j][1];
                        kw_mma<kType>(d, x.x, y.x, x.y, y.y, bq[n][4 * j], bq[n][4 * j + 1]);
                        kw_mma<kType>(d2, x.z, y.z, x.w, y.w, bq[n][4 * j + 2], bq[n][4 * j + 3]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        d[e] += d2[e];
                        const int key = t + g + 8 * (e >> 1);
                        const float x = kCap ? capped(d[e], p.cap_in, p.cap_log2) - lse2[n][e & 1]
                                             : fmaf(d[e], p.scale_log2, -lse2[n][e & 1]);
                        sum[e >> 1] += key >= lo[n][e & 1] && key < hi[n][e & 1] ? fast_exp2(x) : 0.f;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[e] += __shfl_xor_sync(kFull, sum[e], 1);
                sum[e] += __shfl_xor_sync(kFull, sum[e], 2);
            }
            if (store) w.weights[b * w.weights_b + hk * w.weights_h + mine] = fmaf(w.decay, before[u], q4 ? sum[1] : sum[0]);
        }
    };
#pragma unroll
    for (int i = 0; i < kKwStages - 1; ++i) copy_keys(warp + i * kKwWarps, i);
    int slot = 0;
    float a0[U], a1[U];
    prior_of(warp, a0);
    prior_of(warp + kKwWarps, a1);
#pragma unroll 1
    for (int s = warp; s < steps; s += kKwWarps) {
        copy_keys(s + (kKwStages - 1) * kKwWarps, slot == 0 ? kKwStages - 1 : slot - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kKwStages - 1) : "memory");
        float a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = a0[u], a0[u] = a1[u];
        prior_of(s + 2 * kKwWarps, a1);
        weigh(s, slot, a);
        slot = slot + 1 == kKwStages ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int kType, int NT>
static cudaError_t launch_one(const WeighParams& w, dim3 grid, cudaStream_t stream) {
    auto kern = w.a.cap_log2 > 0.f ? key_weights_kernel<D, kType, NT, true> : key_weights_kernel<D, kType, NT, false>;
    static PerDevice state[2];
    const cudaError_t e = kernel_setup(state[w.a.cap_log2 > 0.f], kern, 32 * kKwWarps, kKwSmem);
    if (e != cudaSuccess) return e;
    kern<<<grid, 32 * kKwWarps, kKwSmem, stream>>>(w);
    return cudaGetLastError();
}

// rows: query rows of a kv head and request, at most
cudaError_t launch_key_weights(int D, int kv_dtype, long long rows, const WeighParams& w, dim3 grid, cudaStream_t stream) {
    const bool two = rows > 8;
#define PKD_KW(d, t) \
    if (D == d && kv_dtype == t) return two ? launch_one<d, t, 2>(w, grid, stream) : launch_one<d, t, 1>(w, grid, stream);
    PKD_KW(128, 0) PKD_KW(128, 1) PKD_KW(128, 2) PKD_KW(64, 0) PKD_KW(64, 1)
#undef PKD_KW
    return cudaErrorInvalidValue;
}

}  // namespace pkd
