// ua_fp4_tiles.cuh -- f16 operand tiles of the tcgen05 kernels over 4-bit caches:
// 128 query rows, or the keys of pages, in the 128-byte-swizzled layout that a
// TMA copy of a 16-bit tensor would have (panels of 64 dims, 128 bytes a row).
#pragma once

#include <cstdint>

#include "ua_common.cuh"
#include "ua_fp4.cuh"
#include "ua_ptx.cuh"

namespace ua {

// Rows of a tile: packed (position, head) pairs, positions first .. last, the g
// heads of one KV head.
struct TileRows {
    int64_t q0;        // the sequence's first row of q
    int hkv, g;
    int first, last;   // positions
    __device__ __forceinline__ int pos(int r) const { return first + r / g; }
    __device__ __forceinline__ bool real(int r) const { return r < 128 / g * g && pos(r) <= last; }
    __device__ __forceinline__ int head(int r) const { return hkv * g + r % g; }
    __device__ __forceinline__ int64_t row(const FwdParams& p, int r) const { return (q0 + pos(r)) * p.hq + head(r); }
};

// Q as f16, each row scaled by a power of two so that its largest magnitude
// lies in [1, 2) (f16 covers 2^-24 below that); the factors go to q_scale.  Eight
// threads a row; BATCH passes' loads are in flight together.
template <int D, int THREADS, int BATCH>
__device__ __forceinline__ void stage_q(const FwdParams& p, const TileRows& rows, int t, uint8_t* tile, float* q_scale) {
    constexpr int kPer = D / 8, kEach = THREADS / 8, kPasses = 128 / kEach, kPanel = 128 * 128;
    const int e0 = (t & 7) * kPer;
#pragma unroll 1
    for (int pass = 0; pass < kPasses; pass += BATCH) {
        uint4 x[BATCH][kPer / 8];
        const int r_0 = pass * kEach + (t >> 3);
#pragma unroll
        for (int a = 0; a < BATCH; ++a) {
            const int r = r_0 + kEach * a;
            const bool real = rows.real(r);
#pragma unroll
            for (int c = 0; c < kPer / 8; ++c)
                x[a][c] = real ? __ldg(reinterpret_cast<const uint4*>(p.q + rows.row(p, r) * D + e0) + c)
                               : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int a = 0; a < BATCH; ++a) {
            const int r = r_0 + kEach * a;
            uint32_t amax = 0;
#pragma unroll
            for (int c = 0; c < kPer / 8; ++c)
                amax = __vmaxu2(amax, __vmaxu2(__vmaxu2(x[a][c].x & 0x7fff7fffu, x[a][c].y & 0x7fff7fffu),
                                               __vmaxu2(x[a][c].z & 0x7fff7fffu, x[a][c].w & 0x7fff7fffu)));
            amax = max(amax & 0xffffu, amax >> 16);
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
            const int ef = (int)(amax >> 7);
            const int e = (amax == 0 || ef == 255) ? 0 : min(max(ef, 1), 253) - 127;
            const float down = __int_as_float((127 - e) << 23);
            if ((t & 7) == 0) q_scale[r] = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int c = 0; c < kPer / 8; ++c) {
                const uint32_t v[4] = {x[a][c].x, x[a][c].y, x[a][c].z, x[a][c].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                        : "=r"(h[k]) : "f"(bf16_hi(v[k]) * down), "f"(bf16_lo(v[k]) * down));
                const int dim = e0 + c * 8;
                *reinterpret_cast<uint4*>(tile + (dim >> 6) * kPanel + r * 128 + ((((dim & 63) >> 3) ^ (r & 7)) << 4)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    }
}

// 16 bytes of codes (dims 32 chunk .. + 31 of the tile's key k) and their two scales
// (e4m3, low byte first) to four 16-byte units of the key's row in one panel.
__device__ __forceinline__ void stage_codes(uint4 codes, uint32_t s8, int chunk, int k, uint8_t* panel) {
    const uint32_t sc = e4m3x2_to_f16(s8), s0 = splat_lo(sc), s1 = splat_hi(sc);
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t h[4];
        e2m1x8_to_f16(w[q], h);
        const uint32_t f = q < 2 ? s0 : s1;
        *reinterpret_cast<uint4*>(panel + k * 128 + ((((chunk & 1) * 4 + q) ^ (k & 7)) << 4)) =
            make_uint4(mul_f16x2(h[0], f), mul_f16x2(h[1], f), mul_f16x2(h[2], f), mul_f16x2(h[3], f));
    }
}

}  // namespace ua
