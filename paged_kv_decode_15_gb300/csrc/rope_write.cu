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
// Memory moves bound it (32768 tokens, 32 + 8 heads, bf16 to e4m3: 122 us, 0.75 of the
// copy bandwidth with the ALU pipe 56% busy; 4099 tokens in fp16: 10 us, that
// bandwidth): every element is read once and written once, 16
// elements (two 16-byte chunks, the two halves of eight pairs) per thread and
// head.  One block per token: a thread keeps its place u in the head, so its
// 16 table entries are read once for all heads of the token, and the q, k and v
// loads (all heads, issued before any use) do not wait for the position that
// the table row depends on.
#include <cmath>

#include "launch.h"
#include "packed.cuh"
#include "page_math.h"
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
    float q_inv, k_inv, v_inv;  // 1/scale where rope_store8 takes it, else 0
    uint32_t pmagic;            // slot / P for slots below 2^31
    int pmshift;
};

__device__ __forceinline__ uint32_t rope_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool kBF16>
__device__ __forceinline__ void rope_widen(const uint4& v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBF16)
            bf16x2_to_f32(w[i], f[i].x, f[i].y);
        else
            f16x2_to_f32(w[i], f[i].x, f[i].y);
    }
}

template <bool kBF16>
__device__ __forceinline__ void rope_store16(uint8_t* dst, const float2 (&f)[4]) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<kBF16>(f[0].x, f[0].y), pack2<kBF16>(f[1].x, f[1].y),
                                                pack2<kBF16>(f[2].x, f[2].y), pack2<kBF16>(f[3].x, f[3].y));
}

// Eight values as e4m3(x / scale), the quotient correctly rounded, from their
// negatives n = -x.  With y = 1/scale correctly rounded, q = n (-y) is within an ulp
// of the quotient, the remainder r = q scale + n is exact in one fma, and q - r y
// rounds to the quotient (Markstein, 1990; y's significand not all ones, no
// underflow that e4m3 would see: the host checks the scale's range and passes
// y = 0 where a division is needed).  Taken from -x, a zero keeps its sign.  Eight
// with one far beyond e4m3's range, whose remainder could overflow, are divided.
// All on packed operations (with a division per value
// rope_prompt_fp8 took 207 us, with the correction in single ones 171 us).
__device__ __forceinline__ void rope_store8(uint8_t* dst, const float2 (&n)[4], float scale, float y) {
    float2 q[4];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = mul2(n[i], both(-y));
        top = max3(top, fabsf(q[i].x), fabsf(q[i].y));
    }
    uint32_t h[4];
    if (y != 0.f && top < 1073741824.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = fma2(fma2(q[i], both(scale), n[i]), both(-y), q[i]);
            h[i] = rope_e4m3x2(q[i].x, q[i].y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = rope_e4m3x2(__fdiv_rn(-n[i].x, scale), __fdiv_rn(-n[i].y, scale));
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

constexpr int kRopeThreads = 128;

// Heads in flight per thread and blocks per SM.  The e4m3 forms have the arithmetic
// to hide too and go by threads: rope_prompt_fp8 takes 122 us with one head and ten
// blocks, 151 us with three heads and the five blocks that their registers leave.
template <int D, bool kBF16, bool kQ8, bool kKV8, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kQ8 || kKV8 ? 10 : 7) rope_write_kernel(const RopeParams p) {
    constexpr int kRopeHeads = kQ8 || kKV8 ? 1 : 3;
    constexpr bool kNegTurn = kQ8 && kKV8;   // every turned value goes to e4m3: turned to its negative
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
    // cache row of the token's slot in head 0 (heads are P rows apart)
    long long row0 = 0;
    if (cached) {
        const long long page = p.num_slots <= 0x7fffffffll ? page_div(static_cast<int>(slot), p.pmagic, p.pmshift) : slot / p.P;
        row0 = page * p.Hkv * p.P + (slot - page * p.P);
    }
    float2 c[4], s[4];  // cosines and sines of the thread's eight pairs
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
            float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row + p.rd / 8), s1 = __ldg(row + p.rd / 8 + 1);
            if constexpr (kNegTurn) {
                c0 = make_float4(-c0.x, -c0.y, -c0.z, -c0.w); c1 = make_float4(-c1.x, -c1.y, -c1.z, -c1.w);
                s0 = make_float4(-s0.x, -s0.y, -s0.z, -s0.w); s1 = make_float4(-s1.x, -s1.y, -s1.z, -s1.w);
            }
            c[0] = make_float2(c0.x, c0.y); c[1] = make_float2(c0.z, c0.w); c[2] = make_float2(c1.x, c1.y); c[3] = make_float2(c1.z, c1.w);
            s[0] = make_float2(s0.x, s0.y); s[1] = make_float2(s0.z, s0.w); s[2] = make_float2(s1.x, s1.y); s[3] = make_float2(s1.z, s1.w);
        }
#pragma unroll
        for (int i = 0; i < kRopeHeads; ++i) {
            const int h = base + i * HS;
            if (h >= H) continue;
            const bool is_q = h < p.Hq, val = h >= p.Hq + p.Hkv;
            if (!is_q && !cached) continue;
            const int d0 = val ? 16 * u : e0, d1 = val ? 16 * u + 8 : e1;
            const bool fp8 = is_q ? kQ8 : kKV8;
            uint8_t* dst;
            if (is_q)
                dst = p.q_out + QE * (t * p.q_out_stride + h * D);
            else
                dst = p.cache + KE * ((row0 + static_cast<long long>(val ? h - p.Hq - p.Hkv : h - p.Hq) * p.P) * 2 * D + (val ? D : 0));
            if ((val || !turn) && !fp8) {  // the input's bits
                *reinterpret_cast<uint4*>(dst + 2 * d0) = a[i];
                *reinterpret_cast<uint4*>(dst + 2 * d1) = b[i];
                continue;
            }
            float2 x[4], y[4];
            if (fp8 && (val || !turn || !kNegTurn)) {  // rope_store8 takes negatives
                a[i] = make_uint4(a[i].x ^ 0x80008000u, a[i].y ^ 0x80008000u, a[i].z ^ 0x80008000u, a[i].w ^ 0x80008000u);
                b[i] = make_uint4(b[i].x ^ 0x80008000u, b[i].y ^ 0x80008000u, b[i].z ^ 0x80008000u, b[i].w ^ 0x80008000u);
            }
            rope_widen<kBF16>(a[i], x);
            rope_widen<kBF16>(b[i], y);
            if (!val && turn) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (kInterleaved) {
                        // pairs (x[j].x, x[j].y) and (y[j].x, y[j].y): table entries j and 4 + j
                        const float cx = j & 1 ? c[j >> 1].y : c[j >> 1].x, sx = j & 1 ? s[j >> 1].y : s[j >> 1].x;
                        const float cy = j & 1 ? c[2 + (j >> 1)].y : c[2 + (j >> 1)].x, sy = j & 1 ? s[2 + (j >> 1)].y : s[2 + (j >> 1)].x;
                        x[j] = fma2(x[j], both(cx), mul2(make_float2(x[j].y, x[j].x), make_float2(-sx, sx)));
                        y[j] = fma2(y[j], both(cy), mul2(make_float2(y[j].y, y[j].x), make_float2(-sy, sy)));
                    } else {
                        const float2 x1 = x[j], x2 = y[j];
                        x[j] = fma2(x1, c[j], mul2(x2, make_float2(-s[j].x, -s[j].y)));
                        y[j] = fma2(x2, c[j], mul2(x1, s[j]));
                    }
                }
            }
            if (fp8) {
                const float scale = is_q ? p.q_scale : val ? p.v_scale : p.k_scale;
                const float inv = is_q ? p.q_inv : val ? p.v_inv : p.k_inv;
                rope_store8(dst + d0, x, scale, inv);
                rope_store8(dst + d1, y, scale, inv);
            } else {
                rope_store16<kBF16>(dst + 2 * d0, x);
                rope_store16<kBF16>(dst + 2 * d1, y);
            }
        }
    }
}

// 1/s, correctly rounded, where rope_store8 is exact with it: s within 2^+-60 and its
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
    if (num_pages > ((int64_t)1 << 50) / ((int64_t)page_size * num_kv_heads))
        return report(PKD_EUNSUPPORTED, "cache too large: num_pages*num_kv_heads*page_size must be <= 2^50");
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
    pkd::page_magic(page_size, p.pmagic, p.pmshift);
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
