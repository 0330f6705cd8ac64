// Rotary step of a layer: queries rotated, keys rotated and appended to the
// paged cache with their values, in one launch.
//
// For position p and pair j of a head, with c = cos_sin[p][j] and
// s = cos_sin[p][rd/2 + j] (rd = rotary_dim):
//   (x1, x2) -> (x1 c - x2 s, x2 c + x1 s)
// where the pair is (x[j], x[j + rd/2]), or (x[2j], x[2j+1]) interleaved; the
// dims from rd on are copied.  The rotation is computed in fp32 and rounded
// once: to the input type, or, for e4m3 storage, as e4m3(x / scale) with an
// IEEE division straight from the fp32 value.
//
// Memory moves bound it: every element is read once and written once, 16
// elements (two 16-byte chunks, the two halves of eight pairs) per thread and
// head.  One block per token: a thread keeps its place u in the head, so its
// 16 table entries are read once for all heads of the token, and the q, k and v
// loads (all heads, issued before any use) do not wait for the position that
// the table row depends on.
#include <cmath>

#include "launch.h"
#include "ptx.cuh"

namespace pkd {

struct RopeParams {
    const uint8_t* q;        // [T, Hq, D], token stride q_stride elements
    const uint8_t* key;      // [T, Hkv, D]
    const uint8_t* value;    // [T, Hkv, D]
    const int64_t* positions;  // [T]
    const float* table;        // [max_position, rd]: cos, then sin
    const int64_t* slots;      // [T]
    uint8_t* q_out;            // [T, Hq, D], token stride q_out_stride elements
    uint8_t* cache;            // [num_pages, Hkv, P, 2D]
    long long q_stride, k_stride, v_stride, q_out_stride, max_position, num_slots;
    int Hq, Hkv, P, rd;
    float q_scale, k_scale, v_scale;
    float q_inv, k_inv, v_inv;  // 1/scale where rope_divide holds, else 0
};

__device__ __forceinline__ uint32_t rope_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// x / scale, correctly rounded, from y = 1/scale correctly rounded: q = x y is
// within an ulp, the remainder x - q scale is exact in one fma, and q + r y
// rounds to the quotient (Markstein, 1990; y's significand not all ones, no
// underflow that e4m3 would see: the host checks the scale's range).  Beyond
// e4m3's range, where r may overflow, q itself saturates the same; a zero q
// keeps its sign.
// rope_prompt (32768 tokens, e4m3) takes this instead of a division per value.
__device__ __forceinline__ float rope_divide(float x, float scale, float y) {
    const float q = x * y;
    const float r = fmaf(-q, scale, x);
    const float a = fabsf(q);
    return a > 0.f && a < 1024.f ? fmaf(r, y, q) : q;
}

template <bool kBF16>
__device__ __forceinline__ void rope_widen(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBF16)
            bf16x2_to_f32(w[i], f[2 * i], f[2 * i + 1]);
        else
            f16x2_to_f32(w[i], f[2 * i], f[2 * i + 1]);
    }
}

// Eight values to `dst`: rounded to the 16-bit type, or as e4m3(x / scale).
template <bool kBF16>
__device__ __forceinline__ void rope_store(uint8_t* dst, const float (&f)[8], bool fp8, float scale, float inv) {
    if (!fp8) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<kBF16>(f[0], f[1]), pack2<kBF16>(f[2], f[3]),
                                                    pack2<kBF16>(f[4], f[5]), pack2<kBF16>(f[6], f[7]));
        return;
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = inv != 0.f ? rope_divide(f[2 * i], scale, inv) : __fdiv_rn(f[2 * i], scale);
        const float b = inv != 0.f ? rope_divide(f[2 * i + 1], scale, inv) : __fdiv_rn(f[2 * i + 1], scale);
        h[i] = rope_e4m3x2(a, b);
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

constexpr int kRopeThreads = 128;
constexpr int kRopeHeads = 3;  // heads in flight per thread

template <int D, bool kBF16, bool kQ8, bool kKV8, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeParams p) {
    constexpr int U = D / 16;                // threads per head
    constexpr int HS = kRopeThreads / U;     // heads side by side
    constexpr int KE = kKV8 ? 1 : 2, QE = kQ8 ? 1 : 2;
    const long long t = blockIdx.x;
    const int u = threadIdx.x % U, hs = threadIdx.x / U;
    const int H = p.Hq + 2 * p.Hkv;
    // first elements of the thread's two chunks; rotated: the pairs lie in rd
    const bool turn = 16 * u < p.rd;
    const int e0 = !kInterleaved && turn ? 8 * u : 16 * u;
    const int e1 = !kInterleaved && turn ? p.rd / 2 + 8 * u : 16 * u + 8;

    const long long pos = __ldg(p.positions + t), slot = __ldg(p.slots + t);
    auto source = [&](int h) -> const uint8_t* {
        if (h < p.Hq) return p.q + 2 * (t * p.q_stride + h * D);
        if (h < p.Hq + p.Hkv) return p.key + 2 * (t * p.k_stride + (h - p.Hq) * D);
        return p.value + 2 * (t * p.v_stride + (h - p.Hq - p.Hkv) * D);
    };
    const bool known = pos >= 0 && pos < p.max_position;
    const bool cached = slot >= 0 && slot < p.num_slots;
    float c[8], s[8];
    for (int base = hs; base < H; base += kRopeHeads * HS) {
        uint4 a[kRopeHeads], b[kRopeHeads];
#pragma unroll
        for (int i = 0; i < kRopeHeads; ++i) {
            const int h = base + i * HS;
            if (h >= H) continue;
            // values keep their order: chunks 2u and 2u + 1
            const bool val = h >= p.Hq + p.Hkv;
            const uint8_t* src = source(h);
            a[i] = *reinterpret_cast<const uint4*>(src + 2 * (val ? 16 * u : e0));
            b[i] = *reinterpret_cast<const uint4*>(src + 2 * (val ? 16 * u + 8 : e1));
        }
        if (!known) return;  // a position outside the table: nothing of the token is written
        if (base == hs && turn) {
            const float4* row = reinterpret_cast<const float4*>(p.table + pos * p.rd) + 2 * u;
            const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row + p.rd / 8), s1 = __ldg(row + p.rd / 8 + 1);
            c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
            s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
        }
#pragma unroll
        for (int i = 0; i < kRopeHeads; ++i) {
            const int h = base + i * HS;
            if (h >= H) continue;
            const bool is_q = h < p.Hq, val = h >= p.Hq + p.Hkv;
            if (!is_q && !cached) continue;
            const int d0 = val ? 16 * u : e0, d1 = val ? 16 * u + 8 : e1;
            uint8_t* dst;
            if (is_q) {
                dst = p.q_out + QE * (t * p.q_out_stride + h * D);
            } else {
                const long long page = slot / p.P;
                const int off = static_cast<int>(slot - page * p.P), hk = val ? h - p.Hq - p.Hkv : h - p.Hq;
                dst = p.cache + KE * (((page * p.Hkv + hk) * p.P + off) * 2 * D + (val ? D : 0));
            }
            if ((val || !turn) && !(is_q ? kQ8 : kKV8)) {  // the input's bits
                *reinterpret_cast<uint4*>(dst + 2 * d0) = a[i];
                *reinterpret_cast<uint4*>(dst + 2 * d1) = b[i];
                continue;
            }
            float x[8], y[8];
            rope_widen<kBF16>(a[i], x);
            rope_widen<kBF16>(b[i], y);
            if (!val && turn) {
                if constexpr (kInterleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x1 = x[2 * j], x2 = x[2 * j + 1], y1 = y[2 * j], y2 = y[2 * j + 1];
                        x[2 * j] = x1 * c[j] - x2 * s[j];
                        x[2 * j + 1] = x2 * c[j] + x1 * s[j];
                        y[2 * j] = y1 * c[4 + j] - y2 * s[4 + j];
                        y[2 * j + 1] = y2 * c[4 + j] + y1 * s[4 + j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float x1 = x[j], x2 = y[j];
                        x[j] = x1 * c[j] - x2 * s[j];
                        y[j] = x2 * c[j] + x1 * s[j];
                    }
                }
            }
            const int elt = is_q ? QE : KE;
            const bool fp8 = is_q ? kQ8 : kKV8;
            const float scale = is_q ? p.q_scale : val ? p.v_scale : p.k_scale;
            const float inv = is_q ? p.q_inv : val ? p.v_inv : p.k_inv;
            rope_store<kBF16>(dst + elt * d0, x, fp8, scale, inv);
            rope_store<kBF16>(dst + elt * d1, y, fp8, scale, inv);
        }
    }
}

// 1/s, correctly rounded, where rope_divide is exact: s within 2^+-60 and its
// significand not all ones; else 0 (an IEEE division per value).
static float division_inverse(float s) {
    int e;
    const float m = frexpf(s, &e);
    return e > -60 && e < 60 && m != 1.0f - 0x1p-24f ? 1.0f / s : 0.0f;
}

template <int D>
static cudaError_t launch_rope(const RopeParams& p, long long T, bool bf16, bool q8, bool kv8, bool inter,
                               cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(T);
#define PKD_ROPE(b, q, k, i)                                                                       \
    if (bf16 == b && q8 == q && kv8 == k && inter == i)                                            \
        rope_write_kernel<D, b, q, k, i><<<grid, kRopeThreads, 0, stream>>>(p);
#define PKD_ROPE_T(b) \
    PKD_ROPE(b, false, false, false) PKD_ROPE(b, false, false, true) PKD_ROPE(b, false, true, false) \
    PKD_ROPE(b, false, true, true) PKD_ROPE(b, true, false, false) PKD_ROPE(b, true, false, true)    \
    PKD_ROPE(b, true, true, false) PKD_ROPE(b, true, true, true)
    PKD_ROPE_T(true) PKD_ROPE_T(false)
#undef PKD_ROPE_T
#undef PKD_ROPE
    return cudaGetLastError();
}

}  // namespace pkd

extern "C" pkd_status pkd_rope_cache_write(const void* q, int64_t q_stride, const void* key, int64_t key_stride,
                                           const void* value, int64_t value_stride, pkd_dtype in_dtype,
                                           const int64_t* positions, const float* cos_sin, int64_t max_position,
                                           int rotary_dim, int interleaved, const int64_t* slot_mapping,
                                           int64_t num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                           int page_size, int64_t num_pages, void* kv_cache, pkd_dtype kv_dtype,
                                           float k_scale, float v_scale, void* q_out, int64_t q_out_stride,
                                           pkd_dtype q_out_dtype, float q_scale, void* stream) {
    using pkd::report;
    if (num_tokens < 0 || num_heads < 0 || num_kv_heads < 1 || page_size < 1 || num_pages < 1 || max_position < 0)
        return report(PKD_EINVAL, "invalid shape: num_tokens=%lld num_heads=%d num_kv_heads=%d page_size=%d "
                      "num_pages=%lld max_position=%lld", (long long)num_tokens, num_heads, num_kv_heads, page_size,
                      (long long)num_pages, (long long)max_position);
    if (head_dim != 64 && head_dim != 128) return report(PKD_EUNSUPPORTED, "head_dim %d not supported (64 or 128)", head_dim);
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16)
        return report(PKD_EUNSUPPORTED, "rotary_dim %d must be a multiple of 16 between 16 and head_dim %d", rotary_dim,
                      head_dim);
    if (in_dtype != PKD_BF16 && in_dtype != PKD_FP16)
        return report(PKD_EUNSUPPORTED, "q/key/value dtype %d not supported (bf16, fp16)", (int)in_dtype);
    if (kv_dtype != in_dtype && kv_dtype != PKD_FP8_E4M3)
        return report(PKD_EUNSUPPORTED, "cache dtype %d must equal the input dtype or be fp8-e4m3", (int)kv_dtype);
    if (num_heads > 0 && q_out_dtype != in_dtype && q_out_dtype != PKD_FP8_E4M3)
        return report(PKD_EUNSUPPORTED, "q_out dtype %d must equal the input dtype or be fp8-e4m3", (int)q_out_dtype);
    const int64_t qrow = (int64_t)num_heads * head_dim, krow = (int64_t)num_kv_heads * head_dim;
    if (q_stride < qrow || q_out_stride < qrow || key_stride < krow || value_stride < krow || q_stride % 8 ||
        q_out_stride % 8 || key_stride % 8 || value_stride % 8)
        return report(PKD_EINVAL, "token strides must be >= heads*head_dim and multiples of 8 elements");
    if (kv_dtype == PKD_FP8_E4M3 && !(k_scale > 0.f && v_scale > 0.f && std::isfinite(k_scale) && std::isfinite(v_scale)))
        return report(PKD_EINVAL, "fp8 scales must be positive and finite");
    if (num_heads > 0 && q_out_dtype == PKD_FP8_E4M3 && !(q_scale > 0.f && std::isfinite(q_scale)))
        return report(PKD_EINVAL, "q_scale must be positive and finite");
    if (num_tokens == 0) return PKD_OK;
    if (num_tokens > 0x7fffffffll) return report(PKD_EUNSUPPORTED, "num_tokens must be < 2^31");
    if ((num_heads > 0 && (!q || !q_out)) || !key || !value || !positions || !cos_sin || !slot_mapping || !kv_cache)
        return report(PKD_EINVAL, "null pointer argument");
    auto aligned = [](const void* x, size_t a) { return reinterpret_cast<uintptr_t>(x) % a == 0; };
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(kv_cache, 16) ||
        !aligned(cos_sin, 16) || !aligned(positions, 8) || !aligned(slot_mapping, 8))
        return report(PKD_EINVAL, "q, key, value, q_out, cos_sin and kv_cache must be 16-byte aligned");
    if (num_heads > 0 && q == q_out && (q_out_dtype != in_dtype || (q_stride != q_out_stride && num_tokens > 1)))
        return report(PKD_EINVAL, "q_out may be q itself only with the same dtype and stride");
    pkd::RopeParams p{};
    p.q = static_cast<const uint8_t*>(q);
    p.key = static_cast<const uint8_t*>(key);
    p.value = static_cast<const uint8_t*>(value);
    p.positions = positions;
    p.table = cos_sin;
    p.slots = slot_mapping;
    p.q_out = static_cast<uint8_t*>(q_out);
    p.cache = static_cast<uint8_t*>(kv_cache);
    p.q_stride = q_stride;
    p.k_stride = key_stride;
    p.v_stride = value_stride;
    p.q_out_stride = q_out_stride;
    p.max_position = max_position;
    p.num_slots = num_pages * page_size;
    p.Hq = num_heads;
    p.Hkv = num_kv_heads;
    p.P = page_size;
    p.rd = rotary_dim;
    p.q_scale = q_scale;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.q_inv = pkd::division_inverse(q_scale);
    p.k_inv = pkd::division_inverse(k_scale);
    p.v_inv = pkd::division_inverse(v_scale);
    const bool q8 = num_heads > 0 && q_out_dtype == PKD_FP8_E4M3, kv8 = kv_dtype == PKD_FP8_E4M3;
    const cudaError_t e = head_dim == 128
        ? pkd::launch_rope<128>(p, num_tokens, in_dtype == PKD_BF16, q8, kv8, interleaved != 0, (cudaStream_t)stream)
        : pkd::launch_rope<64>(p, num_tokens, in_dtype == PKD_BF16, q8, kv8, interleaved != 0, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return report(PKD_ECUDA, "pkd_rope_cache_write launch: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
    return PKD_OK;
}
