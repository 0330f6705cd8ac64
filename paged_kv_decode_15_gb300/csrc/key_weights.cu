// pkd_key_weights on mma.sync: steps of few query rows per kv head, bound by reading K.
//
// A warp takes 16 keys of one kv head at a time: D[key, row] = K q^T on m16n8k16 (e4m3:
// m16n8k32) products, the keys as the A operand straight from global memory.  A dot
// product does not care for the order of its dims, so a lane loads 16 consecutive bytes
// of two key rows (a quad: 64, a load instruction 8 x 64 bytes, whole sectors) and takes
// its four words as the operands of two k-steps; q is loaded in the same order.  No
// shared memory, no barrier.  Then exp2(logit - lse), the sum over a lane's rows and
// over its quad, and one 4-byte store per key.
#include "attend_launch.h"
#include "key_weights.cuh"

namespace pkd {

constexpr int kKwWarps = 4;

template <int kType>
__device__ __forceinline__ void kw_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    const uint32_t a[4] = {a0, a1, a2, a3};
    if constexpr (kType == 2)
        mma16832_e4m3(d, a, b0, b1);
    else
        mma16816<kType == 0>(d, a, b0, b1);
}

// kType: 0 bf16, 1 fp16, 2 e4m3.  NT: tiles of 8 rows whose q stays in registers; more
// rows than that are walked in groups, q from the L1 cache.
template <int D, int kType, int NT, bool kCap>
__global__ void __launch_bounds__(32 * kKwWarps, 4) key_weights_kernel(const WeighParams w) {
    constexpr int ROWB = D * (kType == 2 ? 1 : 2), C = ROWB / 64;  // 64-byte chunks of a row
    constexpr int U = 256 / ROWB;                                  // 16-key groups of a step: 8 loads per lane
    const AttendParams& p = w.a;
    const int b = blockIdx.z, hk = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q4 = lane & 3;
    const WeighRequest r = weigh_request(w, b, blockIdx.x == 0 && hk == 0 && threadIdx.x == 0);
    const int k0 = blockIdx.x * p.chunk, k1 = min(k0 + p.chunk, r.L);
    if (k0 >= k1) return;
    const int rows = r.m * p.G, steps = (k1 - k0 + 16 * U - 1) / (16 * U);
    const int32_t* table = p.block_table + static_cast<long long>(b) * p.bt_stride;

    // q of 8 * NT rows from row c0 on, as B operands, with the rows' LSE and positions
    uint32_t bq[NT][4 * C];
    float lse2[NT][2];
    int lo[NT][2], hi[NT][2];  // keys that a row sees: none where there is no row, or its LSE says so
    auto load_rows = [&](int c0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int c = c0 + 8 * n + g;
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
                const int col = c0 + 8 * n + 2 * q4 + e, tok = col / p.G;
                const int pos = r.L - r.m + tok;
                float x = -INFINITY;
                if (col < rows) x = w.lse[static_cast<long long>(r.first + tok) * p.Hq + hk * p.G + col - tok * p.G];
                lse2[n][e] = x * kLog2e;
                lo[n][e] = p.window > 0 ? pos - p.window + 1 : 0;
                hi[n][e] = x == -INFINITY ? 0 : p.causal ? pos + 1 : r.L;
            }
        }
    };
    const bool resident = rows <= 8 * NT;
    load_rows(0);

    uint4 ka[2][U][C][2];
    bool good[2][U];
    // a lane keeps the page of one 16-key group of its warp's share (at most 32)
    int my_page = -1;
    {
        const int group = (lane / U) * kKwWarps * U + warp * U + lane % U, t = k0 + 16 * group;
        if (t < k1) my_page = table[page_div(t, p.pmagic, p.pmshift)];
        if (t < k1 && (my_page < 0 || my_page >= p.num_pages)) {
            my_page = -1;
            atomicOr(p.status, kErrBounds);
        }
    }
    auto load_keys = [&](int s, int buf) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = s / kKwWarps;  // the warp's i-th step
            const int t = k0 + 16 * (s * U + u);
            const int page = __shfl_sync(kFull, my_page, (i * U + u) & 31);
            good[buf][u] = page >= 0;
            if (page < 0) continue;
            const int slot = t - page_div(t, p.pmagic, p.pmshift) * p.P;
            const uint8_t* row = w.cache + (static_cast<long long>(page * p.Hkv + hk) * p.P + slot + g) * (2 * ROWB) + 16 * q4;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                ka[buf][u][j][0] = __ldcs(reinterpret_cast<const uint4*>(row + 64 * j));
                ka[buf][u][j][1] = __ldcs(reinterpret_cast<const uint4*>(row + 64 * j + 8 * 2 * ROWB));
            }
        }
    };
    auto weigh = [&](int s, int buf) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = k0 + 16 * (s * U + u);
            if (t >= k1) continue;
            // this lane stores key t + g + 8 * q4 (q4 < 2)
            const int mine = t + g + 8 * q4;
            const bool store = q4 < 2 && mine < k1;
            float before = 0.f;
            if (store && w.prior && mine < r.fresh) before = w.prior[b * w.prior_b + hk * w.prior_h + mine];
            float sum[2] = {0.f, 0.f};
            if (good[buf][u]) {
                for (int c0 = 0; c0 < rows; c0 += 8 * NT) {
                    if (!resident) load_rows(c0);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            const uint4 x = ka[buf][u][j][0], y = ka[buf][u][j][1];
                            kw_mma<kType>(d, x.x, y.x, x.y, y.y, bq[n][4 * j], bq[n][4 * j + 1]);
                            kw_mma<kType>(d, x.z, y.z, x.w, y.w, bq[n][4 * j + 2], bq[n][4 * j + 3]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = t + g + 8 * (e >> 1);
                            const float x = kCap ? capped(d[e], p.cap_in, p.cap_log2) - lse2[n][e & 1]
                                                 : fmaf(d[e], p.scale_log2, -lse2[n][e & 1]);
                            sum[e >> 1] += key >= lo[n][e & 1] && key < hi[n][e & 1] ? fast_exp2(x) : 0.f;
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[e] += __shfl_xor_sync(kFull, sum[e], 1);
                sum[e] += __shfl_xor_sync(kFull, sum[e], 2);
            }
            if (store) w.weights[b * w.weights_b + hk * w.weights_h + mine] = fmaf(w.decay, before, q4 ? sum[1] : sum[0]);
        }
    };
    int s = warp;
    if (s < steps) load_keys(s, 0);
#pragma unroll 1
    for (; s < steps; s += 2 * kKwWarps) {
        if (s + kKwWarps < steps) load_keys(s + kKwWarps, 1);
        weigh(s, 0);
        if (s + kKwWarps >= steps) break;
        if (s + 2 * kKwWarps < steps) load_keys(s + 2 * kKwWarps, 0);
        weigh(s + kKwWarps, 1);
    }
}

template <int D, int kType, int NT>
static cudaError_t launch_one(const WeighParams& w, dim3 grid, cudaStream_t stream) {
    if (w.a.cap_log2 > 0.f)
        key_weights_kernel<D, kType, NT, true><<<grid, 32 * kKwWarps, 0, stream>>>(w);
    else
        key_weights_kernel<D, kType, NT, false><<<grid, 32 * kKwWarps, 0, stream>>>(w);
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
