// ua_rope.cu -- q and k of a step's tokens rotated by their positions, k and v written
// to their slots of the paged cache.
//
// A pair (a, b) of a head's dims becomes
//     m (a cos(phi) - b sin(phi)),  m (a sin(phi) + b cos(phi)),   phi = pos * f_i.
// The angle is kept as a fraction of a turn in 64 bits: pos * round(2^64 f_i / 2 pi)
// modulo 2^64 drops the whole turns exactly, so that the fraction is off by at most
// |pos| 2^-65 turns (2^-34 at the last position), where an fp32 product would be off by
// |pos f| 2^-24.  Its upper 32 bits go to sincospi as an fp32 number: 2^-32 of a turn cut
// off, and 2^-26 rounded away at most, at any position.
//
// One CTA per token, bound by HBM for prompts.  A thread owns two runs of 8 dims of every
// 16th (8th, 32nd) row: (j ..) and (j + n ..) where halves are paired, so that a pair is
// in one thread, its cos and sin stay in registers over all H_q + H_k rotated heads, and
// q may be rotated in place.  The rows' loads are issued before the angles are computed
// and hide them.
//
// Measured: 65536 tokens, 32 + 2 x 8 heads, d = 128: 229 us (7.0 TB/s of q, k, v read and
// q, k, v written; 409 us when a thread owned 16 neighbouring dims and read the other half
// again), into an fp8 cache 216; 64 tokens of a decode step 3.0 us.  Into a 4-bit cache
// (rope_store_fp4_kernel, which reads the other half again) 328 us, 4.3 TB/s.
#include <algorithm>
#include <cstdint>

#include "ua_launch.h"
#include "ua_ptx.cuh"
#include "ua_quant.cuh"
#include "ua_rope.h"

namespace ua {
namespace {

constexpr int kThreads = 128;       // at most
constexpr int kRows = 3;            // rows in flight per thread

// Angles of one token: (cos, sin) of pair i at cs[turn_at(i)], so that the threads of a row
// read neighbouring words.
__device__ __forceinline__ int turn_at(int i, int run, int n) { return i % run * (n / run) + i / run; }

__device__ __forceinline__ void token_turns(const RopeTable& table, int32_t pos, float2* cs, int run) {
    for (int i = threadIdx.x; i < table.n; i += blockDim.x) {
        const uint64_t phase = (uint64_t)(int64_t)pos * table.turn[i];
        float s, c;
        sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
        cs[turn_at(i, run, table.n)] = make_float2(c * table.magnitude, s * table.magnitude);
    }
}

// Rows of a token: the heads of q, of k, of v.
struct RowPlace {
    const RopeParams& p;
    int64_t token;
    __device__ __forceinline__ const __nv_bfloat16* operator()(int row) const {
        const int d = p.c.d, hk = p.c.hk;
        return row < p.hq ? p.q + token * p.q_stride + row * d
               : row < p.hq + hk ? p.k_new + token * p.kv_stride + (row - p.hq) * d
                                 : p.v_new + token * p.kv_stride + (row - p.hq - hk) * d;
    }
};

// Eight values in an e4m3 cache's format.
template <bool POW2>
__device__ __forceinline__ uint2 to_e4m3(uint4 x, float scale, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
        r[i] = POW2 ? f32x2_to_e4m3(lo * inv, hi * inv) : f32x2_to_e4m3(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale));
    }
    return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}

// bf16 and fp8 caches.
template <int KV, bool POW2, bool PAIRS>
__global__ void __launch_bounds__(kThreads)
rope_store_kernel(const RopeParams p, const __grid_constant__ RopeTable table, float k_inv, float v_inv) {
    __shared__ float2 cs[kMaxFreq];
    const CacheParams& c = p.c;
    const int64_t token = blockIdx.x;
    griddep_wait();
    const int n = table.n, units = c.d >> 4, unit_log2 = 31 - __clz(units);
    const int unit = threadIdx.x & (units - 1), row0 = threadIdx.x >> unit_log2, step = blockDim.x >> unit_log2;
    const int rows = p.hq + 2 * c.hk, turned = p.hq + c.hk;
    const int64_t slot = p.slots[token];
    const int32_t pos = p.positions[token];
    // The thread's runs: both of rotated dims, or (with neighbours paired: each for itself) not.
    const bool half = !PAIRS && unit < n / 8;
    const int a = PAIRS || half ? 8 * unit : 2 * n + 16 * (unit - n / 8);
    const int b = PAIRS ? a + c.d / 2 : half ? a + n : a + 8;
    const bool rot_a = PAIRS ? a < 2 * n : half, rot_b = PAIRS ? b < 2 * n : half;

    const RowPlace place{p, token};
    uint4 x[kRows], y[kRows];
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int row = base + k * step;
            if (row >= rows) break;
            const __nv_bfloat16* src = place(row);
            x[k] = *reinterpret_cast<const uint4*>(src + a);
            y[k] = *reinterpret_cast<const uint4*>(src + b);
        }
    };
    int base = row0;
    load(base);
    token_turns(table, pos, cs, PAIRS ? 4 : 8);
    __syncthreads();
    float2 t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const bool rot = PAIRS && k >= 4 ? rot_b : rot_a;
        const int i = PAIRS ? (k < 4 ? a : b) / 2 + (k & 3) : a + k;
        t[k] = rot ? cs[turn_at(i, PAIRS ? 4 : 8, n)] : make_float2(1.f, 0.f);
    }
    const int64_t block = slot >> (31 - __clz(c.b));
    const bool store = slot >= 0 && block < c.num_blocks;
    if (slot >= 0 && !store && threadIdx.x == 0) atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
    for (;;) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int row = base + k * step;
            if (row >= rows) break;
            if (row < turned && (rot_a || rot_b)) {
                uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, v[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u0 = bf16_lo(u[i]), u1 = bf16_hi(u[i]), v0 = bf16_lo(v[i]), v1 = bf16_hi(v[i]);
                    if constexpr (PAIRS) {
                        if (rot_a) u[i] = pack_bf16x2(u0 * t[i].x - u1 * t[i].y, u0 * t[i].y + u1 * t[i].x);
                        if (rot_b) v[i] = pack_bf16x2(v0 * t[4 + i].x - v1 * t[4 + i].y, v0 * t[4 + i].y + v1 * t[4 + i].x);
                    } else {
                        const float2 t0 = t[2 * i], t1 = t[2 * i + 1];
                        u[i] = pack_bf16x2(u0 * t0.x - v0 * t0.y, u1 * t1.x - v1 * t1.y);
                        v[i] = pack_bf16x2(u0 * t0.y + v0 * t0.x, u1 * t1.y + v1 * t1.x);
                    }
                }
                x[k] = make_uint4(u[0], u[1], u[2], u[3]);
                y[k] = make_uint4(v[0], v[1], v[2], v[3]);
            }
            if (row < p.hq) {
                __nv_bfloat16* dst = p.q_out + token * p.out_stride + row * c.d;
                *reinterpret_cast<uint4*>(dst + a) = x[k];
                *reinterpret_cast<uint4*>(dst + b) = y[k];
            } else if (store) {
                const bool is_v = row >= turned;
                const int64_t at = row_at(c, block, (int)(slot & (c.b - 1)), row - (is_v ? turned : p.hq));
                uint8_t* cache = is_v ? c.v_cache : c.k_cache;
                if constexpr (KV == UA_DTYPE_BF16) {
                    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(cache) + at;
                    *reinterpret_cast<uint4*>(dst + a) = x[k];
                    *reinterpret_cast<uint4*>(dst + b) = y[k];
                } else {
                    const float scale = is_v ? c.v_scale : c.k_scale, inv = is_v ? v_inv : k_inv;
                    *reinterpret_cast<uint2*>(cache + at + a) = to_e4m3<POW2>(x[k], scale, inv);
                    *reinterpret_cast<uint2*>(cache + at + b) = to_e4m3<POW2>(y[k], scale, inv);
                }
            }
        }
        base += kRows * step;
        if (base - row0 >= rows) break;       // the same for the whole CTA
        load(base);
    }
}

// 4-bit caches: 16 dims share a scale, so a thread owns 16 neighbouring dims, and where
// halves are paired reads the other half as well.
template <bool POW2, bool PAIRS>
__global__ void __launch_bounds__(kThreads)
rope_store_fp4_kernel(const RopeParams p, const __grid_constant__ RopeTable table, float k_inv, float v_inv) {
    __shared__ float2 cs[kMaxFreq];
    const CacheParams& c = p.c;
    const int64_t token = blockIdx.x;
    griddep_wait();
    const int n = table.n, groups = c.d >> 4, group_log2 = 31 - __clz(groups);
    const int grp = threadIdx.x & (groups - 1), step = kThreads >> group_log2, rows = p.hq + 2 * c.hk;
    const int64_t slot = p.slots[token];
    token_turns(table, p.positions[token], cs, 8);
    __syncthreads();
    const int64_t block = slot >> (31 - __clz(c.b));
    const bool store = slot >= 0 && block < c.num_blocks;
    if (slot >= 0 && !store && threadIdx.x == 0) atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
    const RowPlace place{p, token};
    for (int row0 = 0; row0 < rows; row0 += step) {
        const int row = row0 + (threadIdx.x >> group_log2);
        const bool live = row < rows, is_v = row >= p.hq + c.hk;
        Group r{};
        if (live) {
            const __nv_bfloat16* src = place(row);
            // (q_out may be q: no read-only loads.)
            uint4 own[2], other[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = grp * 16 + 8 * k;
                own[k] = *reinterpret_cast<const uint4*>(src + j);
                if (!PAIRS && !is_v && j < 2 * n) other[k] = *reinterpret_cast<const uint4*>(src + (j < n ? j + n : j - n));
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = grp * 16 + 8 * k;
                uint32_t u[4] = {own[k].x, own[k].y, own[k].z, own[k].w};
                if (!is_v && j < 2 * n) {
                    const uint32_t v[4] = {other[k].x, other[k].y, other[k].z, other[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u0 = bf16_lo(u[i]), u1 = bf16_hi(u[i]);
                        if constexpr (PAIRS) {
                            const float2 t = cs[turn_at(j / 2 + i, 8, n)];
                            u[i] = pack_bf16x2(u0 * t.x - u1 * t.y, u0 * t.y + u1 * t.x);
                        } else {
                            // The same operations as in the pair's two places above.
                            const int m = (j < n ? j : j - n) + 2 * i;
                            const float2 t0 = cs[turn_at(m, 8, n)], t1 = cs[turn_at(m + 1, 8, n)];
                            const float v0 = bf16_lo(v[i]), v1 = bf16_hi(v[i]);
                            u[i] = j < n ? pack_bf16x2(u0 * t0.x - v0 * t0.y, u1 * t1.x - v1 * t1.y)
                                         : pack_bf16x2(v0 * t0.y + u0 * t0.x, v1 * t1.y + u1 * t1.x);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) r.w[4 * k + i] = u[i];
            }
        }
        __syncwarp();            // a row is read by one warp before it is written
        if (!live) continue;
        if (row < p.hq)
            store_group(p.q_out + token * p.out_stride + row * c.d + grp * 16, r);
        else if (store)
            store_values<UA_DTYPE_FP4_E2M1, POW2>(c, is_v ? c.v_cache : c.k_cache, block, (int)(slot & (c.b - 1)),
                                                  row - p.hq - (is_v ? c.hk : 0), grp, r, is_v ? c.v_scale : c.k_scale,
                                                  is_v ? v_inv : k_inv);
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
                    : (pow2 ? rope_store_fp4_kernel<true, PAIRS> : rope_store_fp4_kernel<false, PAIRS>);
    // Half the threads where they hold a token's rows in one sweep: 8185 tokens of 20 rows at
    // d = 128 into an fp8 cache 12.1 us with 64 threads, 14.9 with 128, 22.6 with 256; 65536
    // tokens of 48 rows 231, 229 and 309.
    const int64_t units = (int64_t)(p.hq + 2 * p.c.hk) * (p.c.d / 16);
    const int threads = p.c.kv_dtype != UA_DTYPE_FP4_E2M1 && units <= 64 * kRows ? 64 : kThreads;
    return launch_early(kern, dim3((unsigned)p.total_q), threads, 0, stream, p, t, k_inv, v_inv);
}

}  // namespace

cudaError_t launch_rope_store(const RopeParams& p, const RopeTable& t, cudaStream_t stream) {
    return t.pairs ? launch_layout<true>(p, t, stream) : launch_layout<false>(p, t, stream);
}

}  // namespace ua
