// ua_cache.cu -- writing K and V rows into the paged cache (bf16, fp8 e4m3 or
// 4-bit e2m1 with one e4m3 scale per 16 dims) and reading a quantised cache
// back as bf16 pages.
//
// Both are one pass over the rows, bound by HBM for prompts and by launch
// latency for decode steps.  A thread owns 16 consecutive dims of one (token,
// KV head) row: the 4-bit format's scale group, 32 bytes of bf16.  Threads run
// over the groups of a row first (256 contiguous bytes of bf16 at d = 128),
// then over tokens, whose 4-bit rows are adjacent in their page, so both sides
// touch whole sectors.
#include <algorithm>
#include <cstdint>

#include "ua_cache.h"
#include "ua_fp4.cuh"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kThreads = 256;

struct Group {       // 16 bf16 values
    uint4 a, b;
};

__device__ __forceinline__ float bf16_at(const Group& x, int e) {
    const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
    return (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
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
__device__ __forceinline__ void quantise_group(const Group& x, float scale, uint32_t (&codes)[2], uint32_t& s8) {
    float y[16];
    float amax = 0.f;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        y[e] = bf16_at(x, e);
        if (scale != 1.f) y[e] = __fdiv_rn(y[e], scale);
        nan |= y[e] != y[e];
        amax = fmaxf(amax, fabsf(y[e]));
    }
    s8 = nan ? 0x7fu : sixth_to_e4m3(amax);
    codes[0] = codes[1] = 0;
    if (nan || s8 == 0) return;
    uint32_t h = e4m3x2_to_f16(s8);
    float s;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(s) : "r"(h));
    // A magnitude's code is the number of midpoints below it; the midpoints
    // times s are exact in fp32, and one that is met rounds to the even code.
    const float t0 = 0.25f * s, t1 = 0.75f * s, t2 = 1.25f * s, t3 = 1.75f * s, t4 = 2.5f * s, t5 = 3.5f * s,
                t6 = 5.f * s;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float a = fabsf(y[e]);
        uint32_t c = (a > t0) + (a >= t1) + (a > t2) + (a >= t3) + (a > t4) + (a >= t5) + (a > t6);
        c |= (__float_as_uint(y[e]) >> 28) & 8u;
        codes[e >> 3] |= c << (4 * (e & 7));
    }
}

// Address of the 16-dim group `grp` of (block, slot, head): fp8 and bf16 rows,
// or the codes of a 4-bit page.
__device__ __forceinline__ int64_t row_at(const CacheParams& c, int64_t block, int slot, int h) {
    return ((block * c.b + slot) * c.hk + h) * c.d;
}

__global__ void __launch_bounds__(kThreads) store_kernel(const StoreParams p, int tokens) {
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
    const int groups = c.d / 16;
    const int items = groups * n * c.hk * 2;
    for (int e = threadIdx.x; e < items; e += kThreads) {
        const int grp = e % groups;
        int rest = e / groups;
        const int tok = (int)first + rest % n;
        rest /= n;
        const int h = rest >> 1;
        const bool v = rest & 1;
        const int pos = sk - sq + tok;
        const int32_t id = __ldg(c.block_table + (int64_t)s * c.bt_stride + pos / c.b);
        if (id < 0 || (int64_t)id >= c.num_blocks) {
            atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
            continue;
        }
        const int slot = pos % c.b;
        const uint4* src = reinterpret_cast<const uint4*>((v ? p.v_new : p.k_new) + (int64_t)(a + tok) * p.stride +
                                                          h * c.d + grp * 16);
        Group x;
        x.a = __ldg(src);
        x.b = __ldg(src + 1);
        uint8_t* cache = v ? c.v_cache : c.k_cache;
        const float scale = v ? c.v_scale : c.k_scale;
        if (c.kv_dtype == UA_DTYPE_BF16) {
            uint4* dst = reinterpret_cast<uint4*>(cache + (row_at(c, id, slot, h) + grp * 16) * 2);
            dst[0] = x.a;
            dst[1] = x.b;
        } else if (c.kv_dtype == UA_DTYPE_FP8_E4M3) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float y0 = __fdiv_rn(bf16_at(x, 4 * k), scale), y1 = __fdiv_rn(bf16_at(x, 4 * k + 1), scale);
                const float y2 = __fdiv_rn(bf16_at(x, 4 * k + 2), scale), y3 = __fdiv_rn(bf16_at(x, 4 * k + 3), scale);
                w[k] = f32x2_to_e4m3(y0, y1) | (f32x2_to_e4m3(y2, y3) << 16);
            }
            *reinterpret_cast<uint4*>(cache + row_at(c, id, slot, h) + grp * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            uint32_t codes[2], s8;
            quantise_group(x, scale, codes, s8);
            uint8_t* page = cache + ((int64_t)id * c.hk + h) * fp4_page_bytes(c.b, c.d);
            *reinterpret_cast<uint2*>(page + slot * (c.d / 2) + grp * 8) = make_uint2(codes[0], codes[1]);
            page[c.b * (c.d / 2) + slot * groups + grp] = (uint8_t)s8;
        }
    }
}

// Two f16 values times `scale` in fp32, rounded once to bf16.
__device__ __forceinline__ uint32_t f16x2_to_bf16(uint32_t h, float s, float scale) {
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return pack_bf16x2(lo * s * scale, hi * s * scale);
}

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
    const int groups = c.d / 16;
    const int items = groups * n * c.hk * 2;
    for (int e = threadIdx.x; e < items; e += kThreads) {
        const int grp = e % groups;
        int rest = e / groups;
        const int pos = (int)first + rest % n;
        rest /= n;
        const int h = rest >> 1;
        const bool v = rest & 1;
        const int32_t id = __ldg(c.block_table + (int64_t)s * c.bt_stride + pos / c.b);
        const int32_t to = __ldg(p.out_table + (int64_t)s * p.out_stride + pos / c.b);
        if (id < 0 || (int64_t)id >= c.num_blocks || to < 0 || (int64_t)to >= p.out_blocks) {
            atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
            continue;
        }
        const int slot = pos % c.b;
        const uint8_t* cache = v ? c.v_cache : c.k_cache;
        const float scale = v ? c.v_scale : c.k_scale;
        uint32_t w[8];
        if (c.kv_dtype == UA_DTYPE_BF16) {
            const uint4* src = reinterpret_cast<const uint4*>(cache + (row_at(c, id, slot, h) + grp * 16) * 2);
            const uint4 a = src[0], b = src[1];
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        } else if (c.kv_dtype == UA_DTYPE_FP8_E4M3) {
            const uint4 a = *reinterpret_cast<const uint4*>(cache + row_at(c, id, slot, h) + grp * 16);
            const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[2 * k] = f16x2_to_bf16(e4m3x2_to_f16(q[k] & 0xffffu), 1.f, scale);
                w[2 * k + 1] = f16x2_to_bf16(e4m3x2_to_f16(q[k] >> 16), 1.f, scale);
            }
        } else {
            const uint8_t* page = cache + ((int64_t)id * c.hk + h) * fp4_page_bytes(c.b, c.d);
            const uint2 a = *reinterpret_cast<const uint2*>(page + slot * (c.d / 2) + grp * 8);
            const uint32_t sh = e4m3x2_to_f16(page[c.b * (c.d / 2) + slot * groups + grp]);
            float sv;
            asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(sv) : "r"(sh));
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(a.x, h0);
            e2m1x8_to_f16(a.y, h1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = f16x2_to_bf16(h0[k], sv, scale);
                w[4 + k] = f16x2_to_bf16(h1[k], sv, scale);
            }
        }
        uint4* dst = reinterpret_cast<uint4*>((v ? p.v_out : p.k_out) + row_at(c, to, slot, h) + grp * 16);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Rows (tokens or keys) per CTA: about eight groups per thread.
int rows_per_cta(const CacheParams& c) {
    return std::max(1, kThreads * 8 / (c.d / 16 * c.hk * 2));
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, cudaStream_t stream) {
    const int tokens = rows_per_cta(p.c);
    dim3 grid((unsigned)((p.max_seqlen_q + (int64_t)tokens - 1) / tokens), (unsigned)p.c.num_seqs);
    store_kernel<<<grid, kThreads, 0, stream>>>(p, tokens);
    return cudaGetLastError();
}

cudaError_t launch_expand(const ExpandParams& p, cudaStream_t stream) {
    const int keys = rows_per_cta(p.c);
    dim3 grid((unsigned)((p.max_keys + (int64_t)keys - 1) / keys), (unsigned)p.c.num_seqs);
    expand_kernel<<<grid, kThreads, 0, stream>>>(p, keys);
    return cudaGetLastError();
}

}  // namespace ua
