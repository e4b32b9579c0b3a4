// ua_fp4.cuh -- the 4-bit cache format: one page per (block, KV head) holding
// b rows of d / 2 bytes of e2m1 codes, then b rows of d / 16 e4m3 scales.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace ua {

// Bytes of one page.
__host__ __device__ constexpr int64_t fp4_page_bytes(int b, int d) {
    return (int64_t)b * (d / 2 + d / 16);
}

// The four bytes of `w` (two e2m1 codes each, low nibble first) as four f16x2
// words.  Every e2m1 value is exact in f16.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 codes (low byte first) as f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}

// The low or high half of an f16x2 word in both halves.
__device__ __forceinline__ uint32_t splat_lo(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t splat_hi(uint32_t h) { return __byte_perm(h, h, 0x3232); }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

}  // namespace ua
