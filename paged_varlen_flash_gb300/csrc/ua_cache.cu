// ua_cache.cu -- writing K and V rows into the paged cache (bf16, fp8 e4m3 or
// 4-bit e2m1 with one e4m3 scale per 16 dims) and reading a quantised cache
// back as bf16 pages.
//
// Both are one pass over the rows, bound by HBM for prompts and by launch
// latency for decode steps.  A thread owns 16 consecutive dims of one (token,
// KV head) row: the 4-bit format's scale group, 32 bytes of bf16.  Threads run
// over the groups of a row first (256 contiguous bytes of bf16 at d = 128),
// then over tokens, whose 4-bit rows are adjacent in their page, so both sides
// touch whole sectors; a thread's groups are all loaded before the first is
// converted, so that a prompt chunk pays one memory round trip, not eight.
//
// Measured: 8 prompts of 8192 tokens, 8 KV heads, d = 128: store to 4 bits 65 us
// (5.3 TB/s), expand 57 us (6.1 TB/s); 64 tokens of a decode step 4.4 us.  The
// same prompts to fp8 87 us (a division per element), and to 4 bits with tensor
// scales that are no powers of two 230 us (a division and seven compares).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ua_cache.h"
#include "ua_fp4.cuh"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;   // groups per thread

struct Group {       // 16 bf16 values
    uint32_t w[8];
};

__device__ __forceinline__ Group load_group(const void* src) {
    const uint4 a = __ldg(static_cast<const uint4*>(src)), b = __ldg(static_cast<const uint4*>(src) + 1);
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ void store_group(void* dst, const Group& x) {
    static_cast<uint4*>(dst)[0] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
}

__device__ __forceinline__ float bf16_at(const Group& x, int e) {
    return (e & 1) ? bf16_hi(x.w[e >> 1]) : bf16_lo(x.w[e >> 1]);
}

// The low byte of an e4m3 pair as fp32.
__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
    float s;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}"
        : "=f"(s) : "r"(e4m3x2_to_f16(code)));
    return s;
}

// Two fp32 values to e4m3 (nearest even, magnitudes saturate at 448).
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// e4m3 of the exact quotient a / 6 (a >= 0): the fp32 quotient is rounded to
// odd (truncated, last bit set when inexact), so that rounding it to e4m3
// cannot land on a tie that the exact quotient is not on.
__device__ __forceinline__ uint32_t sixth_to_e4m3(float a) {
    if (a == INFINITY) return 0x7e;              // 448
    float q = __fdiv_rz(a, 6.f);
    if (fmaf(-q, 6.f, a) != 0.f) q = __uint_as_float(__float_as_uint(q) | 1u);
    return f32x2_to_e4m3(q, 0.f) & 0xffu;
}

// One group in the 4-bit format: 8 bytes of codes and the scale byte.
struct Fp4Group {
    uint32_t codes[2], s8;
};

// Any tensor scale: a magnitude's code is the number of midpoints below it; the
// midpoints times s are exact in fp32, and one that is met rounds to the even
// code.
__device__ __forceinline__ Fp4Group quantise_any(const Group& x, float scale) {
    float y[16];
    float amax = 0.f;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        y[e] = __fdiv_rn(bf16_at(x, e), scale);
        nan |= y[e] != y[e];
        amax = fmaxf(amax, fabsf(y[e]));
    }
    Fp4Group r{{0, 0}, nan ? 0x7fu : sixth_to_e4m3(amax)};
    if (nan || r.s8 == 0) return r;
    const float s = e4m3_to_f32(r.s8);
    const float t0 = 0.25f * s, t1 = 0.75f * s, t2 = 1.25f * s, t3 = 1.75f * s, t4 = 2.5f * s, t5 = 3.5f * s,
                t6 = 5.f * s;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float a = fabsf(y[e]);
        uint32_t c = (a > t0) + (a >= t1) + (a > t2) + (a >= t3) + (a > t4) + (a >= t5) + (a > t6);
        if (c) c |= (__float_as_uint(y[e]) >> 28) & 8u;
        r.codes[e >> 3] |= c << (4 * (e & 7));
    }
    return r;
}

// A tensor scale 2^k, |k| <= 64 (inv = 2^-k), the usual case, with a quarter of
// the instructions (prompts of 8 x 8192 tokens: see store_kernel).  Here y = x inv
// has bf16's 8 significant bits and s four, so a quotient that is not a midpoint
// (of two e2m1 or e4m3 values: at most 7 bits after the product with s or 6) is
// at least 2^-9 of itself away from one.  Quotients computed to 2^-22 are
// therefore rounded to 11 bits (the scale, through f16) or to multiples of
// 2^-16 (the codes: adding 192 does that) first, which puts every midpoint
// exactly on itself and moves nothing else across one; the hardware's
// conversions then round ties to even.
__device__ __forceinline__ Fp4Group quantise_pow2(const Group& x, float inv) {
    // Magnitudes as 16-bit integers: ordered like the values, NaN above 0x7f80.
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = __vmaxu2(top, x.w[k] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    const bool nan = top > 0x7f80u;
    const float sixth = fminf(__uint_as_float(top << 16) * inv * (1.f / 6.f), 448.f);
    Fp4Group r;
    uint16_t s8;
    asm("{\n\t.reg .b32 h;\n\tcvt.rn.f16x2.f32 h, %1, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 %0, h;\n\t}"
        : "=h"(s8) : "f"(sixth));
    r.s8 = nan ? 0x7fu : s8 & 0xffu;
    const float s = e4m3_to_f32(r.s8);
    const float f = nan || s == 0.f ? 0.f : __fdividef(inv, s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = fmaf(bf16_at(x, 8 * h + e), f, 192.f) - 192.f;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\tmov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(r.codes[h])
            : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
        // The conversion keeps the sign of what it rounds to 0; code 8 becomes 0.
        const uint32_t c = r.codes[h], some = (c | c >> 1 | c >> 2) & 0x11111111u;
        r.codes[h] = nan ? 0u : c & (0x77777777u | some << 3);
    }
    return r;
}

// Element index of (block, slot, head) in a bf16 or fp8 cache.
__device__ __forceinline__ int64_t row_at(const CacheParams& c, int64_t block, int slot, int h) {
    return ((block * c.b + slot) * c.hk + h) * c.d;
}

// A CTA's items, in order group, row (token or key), KV head, operand.
struct Place {
    int grp, row, h;
    bool v;
};

// x / n for x < 2^16, n < 2^8, with m = 2^32 / n rounded up.
__device__ __forceinline__ int div_by(int x, uint32_t m) { return (int)__umulhi((uint32_t)x, m); }

__device__ __forceinline__ Place place_of(int e, int group_log2, int rows, uint32_t rows_inv) {
    const int rest = e >> group_log2, x = rows == 1 ? rest : div_by(rest, rows_inv);
    return {e & ((1 << group_log2) - 1), rest - x * rows, x >> 1, (x & 1) != 0};
}

// POW2: both tensor scales are powers of two (k_inv, v_inv their inverses).
template <int KV, bool POW2>
__global__ void __launch_bounds__(kThreads) store_kernel(const StoreParams p, int tokens, float k_inv, float v_inv) {
    const CacheParams& c = p.c;
    const int s = blockIdx.y;
    const int32_t a = __ldg(p.cu_seqlens_q + s), z = __ldg(p.cu_seqlens_q + s + 1);
    const int32_t sk = __ldg(c.seqused_k + s);
    const int sq = z - a;
    uint32_t st = 0;
    if (a < 0 || z < a || (int64_t)z > p.total_q) {
        st = UA_DEVERR_CU_SEQLENS;
    } else {
        if (sk < sq) st |= UA_DEVERR_CONTEXT;
        if (sq > p.max_seqlen_q || sk > p.max_seqlen_k || (int64_t)sk > (int64_t)c.bt_stride * c.b)
            st |= UA_DEVERR_BOUNDS;
    }
    if (st) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(c.err, (int)st);
        return;
    }
    const int64_t first = (int64_t)blockIdx.x * tokens;
    if (first >= sq) return;
    const int n = (int)min((int64_t)tokens, sq - first);
    const int groups = c.d >> 4, group_log2 = 31 - __clz(groups), b_log2 = 31 - __clz(c.b);
    const uint32_t n_inv = n == 1 ? 0u : 0xffffffffu / (uint32_t)n + 1u;
    const int items = groups * n * c.hk * 2;
    for (int e0 = threadIdx.x; e0 < items; e0 += kThreads * kItems) {
        Group x[kItems];
        int32_t id[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int e = e0 + k * kThreads;
            if (e >= items) break;
            const Place at = place_of(e, group_log2, n, n_inv);
            const int64_t token = a + first + at.row;
            x[k] = load_group((at.v ? p.v_new : p.k_new) + token * p.stride + at.h * c.d + at.grp * 16);
            id[k] = __ldg(c.block_table + (int64_t)s * c.bt_stride + ((sk - sq + (int)first + at.row) >> b_log2));
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int e = e0 + k * kThreads;
            if (e >= items) break;
            if (id[k] < 0 || (int64_t)id[k] >= c.num_blocks) {
                atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
                continue;
            }
            const Place at = place_of(e, group_log2, n, n_inv);
            const int slot = (sk - sq + (int)first + at.row) & (c.b - 1);
            uint8_t* cache = at.v ? c.v_cache : c.k_cache;
            const float scale = at.v ? c.v_scale : c.k_scale;
            if constexpr (KV == UA_DTYPE_BF16) {
                store_group(cache + (row_at(c, id[k], slot, at.h) + at.grp * 16) * 2, x[k]);
            } else if constexpr (KV == UA_DTYPE_FP8_E4M3) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = f32x2_to_e4m3(__fdiv_rn(bf16_at(x[k], 4 * q), scale),
                                         __fdiv_rn(bf16_at(x[k], 4 * q + 1), scale)) |
                           (f32x2_to_e4m3(__fdiv_rn(bf16_at(x[k], 4 * q + 2), scale),
                                          __fdiv_rn(bf16_at(x[k], 4 * q + 3), scale)) << 16);
                *reinterpret_cast<uint4*>(cache + row_at(c, id[k], slot, at.h) + at.grp * 16) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                Fp4Group r;
                if constexpr (POW2) r = quantise_pow2(x[k], at.v ? v_inv : k_inv);
                else r = quantise_any(x[k], scale);
                uint8_t* page = cache + ((int64_t)id[k] * c.hk + at.h) * fp4_page_bytes(c.b, c.d);
                *reinterpret_cast<uint2*>(page + slot * (c.d / 2) + at.grp * 8) = make_uint2(r.codes[0], r.codes[1]);
                page[c.b * (c.d / 2) + slot * groups + at.grp] = (uint8_t)r.s8;
            }
        }
    }
}

// Two f16 values times s times `scale` in fp32, rounded once to bf16.
__device__ __forceinline__ uint32_t f16x2_to_bf16(uint32_t h, float s, float scale) {
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return pack_bf16x2(lo * s * scale, hi * s * scale);
}

template <int KV>
__global__ void __launch_bounds__(kThreads) expand_kernel(const ExpandParams p, int keys) {
    const CacheParams& c = p.c;
    const int s = blockIdx.y;
    const int sk = __ldg(c.seqused_k + s);
    const int beg = p.begin ? __ldg(p.begin + s) : 0;
    if (sk < 0 || beg < 0 || beg > sk || sk - beg > p.max_keys || (int64_t)sk > (int64_t)c.bt_stride * c.b ||
        (int64_t)sk > (int64_t)p.out_stride * c.b) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(c.err, (int)UA_DEVERR_BOUNDS);
        return;
    }
    const int64_t first = beg + (int64_t)blockIdx.x * keys;
    if (first >= sk) return;
    const int n = (int)min((int64_t)keys, sk - first);
    const int groups = c.d >> 4, group_log2 = 31 - __clz(groups), b_log2 = 31 - __clz(c.b);
    const uint32_t n_inv = n == 1 ? 0u : 0xffffffffu / (uint32_t)n + 1u;
    const int items = groups * n * c.hk * 2;
    for (int e0 = threadIdx.x; e0 < items; e0 += kThreads * kItems) {
        Group x[kItems];       // the stored bytes, then the values
        uint32_t s8[kItems];
        int32_t to[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int e = e0 + k * kThreads;
            if (e >= items) break;
            const Place at = place_of(e, group_log2, n, n_inv);
            const int pos = (int)first + at.row, slot = pos & (c.b - 1);
            const int32_t id = __ldg(c.block_table + (int64_t)s * c.bt_stride + (pos >> b_log2));
            to[k] = __ldg(p.out_table + (int64_t)s * p.out_stride + (pos >> b_log2));
            if (id < 0 || (int64_t)id >= c.num_blocks || to[k] < 0 || (int64_t)to[k] >= p.out_blocks) {
                atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
                to[k] = -1;
                continue;
            }
            const uint8_t* cache = at.v ? c.v_cache : c.k_cache;
            if constexpr (KV == UA_DTYPE_BF16) {
                x[k] = load_group(cache + (row_at(c, id, slot, at.h) + at.grp * 16) * 2);
            } else if constexpr (KV == UA_DTYPE_FP8_E4M3) {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(cache + row_at(c, id, slot, at.h) + at.grp * 16));
                x[k].w[0] = q.x; x[k].w[1] = q.y; x[k].w[2] = q.z; x[k].w[3] = q.w;
            } else {
                const uint8_t* page = cache + ((int64_t)id * c.hk + at.h) * fp4_page_bytes(c.b, c.d);
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(page + slot * (c.d / 2) + at.grp * 8));
                x[k].w[0] = q.x; x[k].w[1] = q.y;
                s8[k] = __ldg(page + c.b * (c.d / 2) + slot * groups + at.grp);
            }
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int e = e0 + k * kThreads;
            if (e >= items) break;
            if (to[k] < 0) continue;
            const Place at = place_of(e, group_log2, n, n_inv);
            const float scale = at.v ? c.v_scale : c.k_scale;
            if constexpr (KV == UA_DTYPE_FP8_E4M3) {
                const uint32_t q[4] = {x[k].w[0], x[k].w[1], x[k].w[2], x[k].w[3]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[k].w[2 * i] = f16x2_to_bf16(e4m3x2_to_f16(q[i] & 0xffffu), 1.f, scale);
                    x[k].w[2 * i + 1] = f16x2_to_bf16(e4m3x2_to_f16(q[i] >> 16), 1.f, scale);
                }
            } else if constexpr (KV == UA_DTYPE_FP4_E2M1) {
                const float sv = e4m3_to_f32(s8[k]);
                uint32_t h0[4], h1[4];
                e2m1x8_to_f16(x[k].w[0], h0);
                e2m1x8_to_f16(x[k].w[1], h1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[k].w[i] = f16x2_to_bf16(h0[i], sv, scale);
                    x[k].w[4 + i] = f16x2_to_bf16(h1[i], sv, scale);
                }
            }
            const int slot = ((int)first + at.row) & (c.b - 1);
            store_group((at.v ? p.v_out : p.k_out) + row_at(c, to[k], slot, at.h) + at.grp * 16, x[k]);
        }
    }
}

// 1 / scale where that is exact and safe to multiply by (a power of two), else 0.
float exact_inverse(float scale) {
    int e = 0;
    return std::frexp(scale, &e) == 0.5f && e >= -63 && e <= 65 ? 1.f / scale : 0.f;
}

// Rows (tokens or keys) per CTA: kItems groups per thread, at most 255 rows.
int rows_per_cta(const CacheParams& c) {
    return std::min(255, std::max(1, kThreads * kItems / (c.d / 16 * c.hk * 2)));
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, cudaStream_t stream) {
    const int tokens = rows_per_cta(p.c);
    dim3 grid((unsigned)((p.max_seqlen_q + (int64_t)tokens - 1) / tokens), (unsigned)p.c.num_seqs);
    const float k_inv = exact_inverse(p.c.k_scale), v_inv = exact_inverse(p.c.v_scale);
    auto kern = p.c.kv_dtype == UA_DTYPE_BF16       ? store_kernel<UA_DTYPE_BF16, false>
                : p.c.kv_dtype == UA_DTYPE_FP8_E4M3 ? store_kernel<UA_DTYPE_FP8_E4M3, false>
                : k_inv != 0.f && v_inv != 0.f      ? store_kernel<UA_DTYPE_FP4_E2M1, true>
                                                    : store_kernel<UA_DTYPE_FP4_E2M1, false>;
    kern<<<grid, kThreads, 0, stream>>>(p, tokens, k_inv, v_inv);
    return cudaGetLastError();
}

cudaError_t launch_expand(const ExpandParams& p, cudaStream_t stream) {
    const int keys = rows_per_cta(p.c);
    dim3 grid((unsigned)((p.max_keys + (int64_t)keys - 1) / keys), (unsigned)p.c.num_seqs);
    auto kern = p.c.kv_dtype == UA_DTYPE_BF16       ? expand_kernel<UA_DTYPE_BF16>
                : p.c.kv_dtype == UA_DTYPE_FP8_E4M3 ? expand_kernel<UA_DTYPE_FP8_E4M3>
                                                    : expand_kernel<UA_DTYPE_FP4_E2M1>;
    kern<<<grid, kThreads, 0, stream>>>(p, keys);
    return cudaGetLastError();
}

}  // namespace ua
