// ua_quant.cuh -- 16 consecutive dims of a cached row: loading them as bf16 and
// writing them in the cache's format (bf16, fp8 e4m3, or 4-bit e2m1 with one e4m3
// scale per 16 dims).  Shared by the kernels that write K and V rows.
#pragma once

#include <cmath>
#include <cstdint>

#include "ua_cache.h"
#include "ua_fp4.cuh"
#include "ua_ptx.cuh"

namespace ua {

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

// One group of a row in the cache's format.  POW2: the tensor scale is a power of
// two and inv its inverse.
template <int KV, bool POW2>
__device__ __forceinline__ void store_values(const CacheParams& c, uint8_t* cache, int64_t block, int slot, int h, int grp,
                                             const Group& x, float scale, float inv) {
    if constexpr (KV == UA_DTYPE_BF16) {
        store_group(cache + (row_at(c, block, slot, h) + grp * 16) * 2, x);
    } else if constexpr (KV == UA_DTYPE_FP8_E4M3) {
        // (The product with a power of two is the quotient; what underflows is 0 in e4m3 either way.)
        auto y = [&](int e) { return POW2 ? bf16_at(x, e) * inv : __fdiv_rn(bf16_at(x, e), scale); };
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = f32x2_to_e4m3(y(4 * q), y(4 * q + 1)) | (f32x2_to_e4m3(y(4 * q + 2), y(4 * q + 3)) << 16);
        *reinterpret_cast<uint4*>(cache + row_at(c, block, slot, h) + grp * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        Fp4Group r;
        if constexpr (POW2) r = quantise_pow2(x, inv);
        else r = quantise_any(x, scale);
        uint8_t* page = cache + (block * c.hk + h) * fp4_page_bytes(c.b, c.d);
        *reinterpret_cast<uint2*>(page + slot * (c.d / 2) + grp * 8) = make_uint2(r.codes[0], r.codes[1]);
        page[c.b * (c.d / 2) + slot * (c.d / 16) + grp] = (uint8_t)r.s8;
    }
}

// 1 / scale where that is exact and safe to multiply by (a power of two), else 0.
inline float exact_inverse(float scale) {
    int e = 0;
    return std::frexp(scale, &e) == 0.5f && e >= -63 && e <= 65 ? 1.f / scale : 0.f;
}

}  // namespace ua
