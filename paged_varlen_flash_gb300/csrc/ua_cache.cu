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
#include "ua_quant.cuh"

namespace ua {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;   // groups per thread

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
            store_values<KV, POW2>(c, cache, id[k], slot, at.h, at.grp, x[k], scale, at.v ? v_inv : k_inv);
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
