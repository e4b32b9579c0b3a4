// ua_rope.cu -- q and k of a step's tokens rotated by their positions, k and v written
// to their slots of the paged cache.
//
// A pair (a, b) of a head's dims becomes
//     m (a cos(phi) - b sin(phi)),  m (a sin(phi) + b cos(phi)),   phi = pos * f_i.
// The angle is kept as a fraction of a turn in 64 bits: pos * round(2^64 f_i / 2 pi)
// modulo 2^64 drops the whole turns exactly, so that the fraction is off by at most
// |pos| 2^-65 turns wherever the position lies, where an fp32 product would be off by
// |pos f| 2^-24.  Its upper 32 bits go to sincospi.
//
// One CTA per token: the token's n angles are computed once (one per thread) and used
// by all H_q + H_k rotated heads; a thread owns 16 dims of a row.
#include <algorithm>
#include <cstdint>

#include "ua_ptx.cuh"
#include "ua_quant.cuh"
#include "ua_rope.h"

namespace ua {
namespace {

constexpr int kThreads = 128;

// Eight bf16 values: x * c - y * s with (c, s) from cs[0 .. 7], or x * c + y * s.
__device__ __forceinline__ uint4 turn8(uint4 x, uint4 y, const float2* cs, float sign) {
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 u = cs[2 * k], v = cs[2 * k + 1];
        r[k] = pack_bf16x2(bf16_lo(a[k]) * u.x + sign * (bf16_lo(b[k]) * u.y),
                           bf16_hi(a[k]) * v.x + sign * (bf16_hi(b[k]) * v.y));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// Four neighbouring pairs in eight values.
__device__ __forceinline__ uint4 turn_pairs(uint4 x, const float2* cs) {
    const uint32_t a[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 u = cs[k];
        const float lo = bf16_lo(a[k]), hi = bf16_hi(a[k]);
        r[k] = pack_bf16x2(lo * u.x - hi * u.y, lo * u.y + hi * u.x);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int KV, bool POW2, bool PAIRS>
__global__ void __launch_bounds__(kThreads)
rope_store_kernel(const RopeParams p, const __grid_constant__ RopeTable table, float k_inv, float v_inv) {
    __shared__ float2 cs[kMaxFreq];
    const CacheParams& c = p.c;
    const int64_t token = blockIdx.x;
    const int tid = threadIdx.x, n = table.n;
    const int64_t slot = __ldg(p.slots + token);
    if (tid < n) {
        const uint64_t phase = (uint64_t)(int64_t)__ldg(p.positions + token) * table.turn[tid];
        float s, co;
        sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &co);
        cs[tid] = make_float2(co * table.magnitude, s * table.magnitude);
    }
    __syncthreads();
    const int64_t block = slot >> (31 - __clz(c.b));
    const bool store = slot >= 0 && block < c.num_blocks;
    if (slot >= 0 && !store && tid == 0) atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
    const int groups = c.d >> 4, group_log2 = 31 - __clz(groups);
    const int items = (p.hq + 2 * c.hk) << group_log2;
    for (int e0 = 0; e0 < items; e0 += kThreads) {
        const int e = e0 + tid;
        const int grp = e & (groups - 1), row = e >> group_log2;
        const bool live = e < items;
        const bool is_q = row < p.hq, is_v = row >= p.hq + c.hk;
        const int h = is_q ? row : (row - p.hq) % c.hk;
        const __nv_bfloat16* src = is_q ? p.q + token * p.q_stride
                                        : (is_v ? p.v_new : p.k_new) + token * p.kv_stride;
        src += h * c.d;
        Group x;
        if (live) {
            uint4 own[2], other[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = grp * 16 + 8 * k;
                own[k] = *reinterpret_cast<const uint4*>(src + j);
                if (!PAIRS && !is_v && j < 2 * n) other[k] = *reinterpret_cast<const uint4*>(src + (j < n ? j + n : j - n));
            }
            if (!is_v) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int j = grp * 16 + 8 * k;
                    if (j >= 2 * n) continue;
                    if constexpr (PAIRS) own[k] = turn_pairs(own[k], cs + j / 2);
                    else own[k] = turn8(own[k], other[k], cs + (j < n ? j : j - n), j < n ? -1.f : 1.f);
                }
            }
            x = {{own[0].x, own[0].y, own[0].z, own[0].w, own[1].x, own[1].y, own[1].z, own[1].w}};
        }
        __syncwarp();            // q_out may be q: a row is read by one warp before it is written
        if (!live) continue;
        if (is_q)
            store_group(p.q_out + token * p.out_stride + h * c.d + grp * 16, x);
        else if (store)
            store_values<KV, POW2>(c, is_v ? c.v_cache : c.k_cache, block, (int)(slot & (c.b - 1)), h, grp, x,
                                   is_v ? c.v_scale : c.k_scale, is_v ? v_inv : k_inv);
    }
}

template <bool PAIRS>
cudaError_t launch_layout(const RopeParams& p, const RopeTable& t, cudaStream_t stream) {
    const float k_inv = exact_inverse(p.c.k_scale), v_inv = exact_inverse(p.c.v_scale);
    const bool pow2 = k_inv != 0.f && v_inv != 0.f;
    auto kern = p.c.kv_dtype == UA_DTYPE_BF16 ? rope_store_kernel<UA_DTYPE_BF16, false, PAIRS>
                : p.c.kv_dtype == UA_DTYPE_FP8_E4M3
                    ? (pow2 ? rope_store_kernel<UA_DTYPE_FP8_E4M3, true, PAIRS>
                            : rope_store_kernel<UA_DTYPE_FP8_E4M3, false, PAIRS>)
                    : (pow2 ? rope_store_kernel<UA_DTYPE_FP4_E2M1, true, PAIRS>
                            : rope_store_kernel<UA_DTYPE_FP4_E2M1, false, PAIRS>);
    kern<<<(unsigned)p.total_q, kThreads, 0, stream>>>(p, t, k_inv, v_inv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_store(const RopeParams& p, const RopeTable& t, cudaStream_t stream) {
    return t.pairs ? launch_layout<true>(p, t, stream) : launch_layout<false>(p, t, stream);
}

}  // namespace ua
