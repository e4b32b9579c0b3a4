// ua_fp4.cu -- attention over a 4-bit (e2m1, one e4m3 scale per 16 dims) paged
// cache: decode, and small chunks in tiles of 8 or 16 packed rows.
//
// The math is the streaming (m, l, o) recurrence of every kernel here, in base
// 2 with the lazy re-anchor.  A decode step reads each cached value once and
// uses it for at most 16 rows, so what it can cost is the path from the 4-bit
// code to a tensor-core operand: at 6.8 TB/s of codes an SM receives about 41
// elements per clock.  The products therefore run as warp-level m16n8k16 MMAs
// whose A operand -- the cached values, keys on M for S^T = K Q^T and dims on M
// for O^T += V^T P^T -- is built in registers: codes come out of shared memory
// once, become f16 there (code x scale has 6 significant bits, exact in f16),
// and go into the MMA, with no second trip through shared or tensor memory
// that a tcgen05 operand would need.
//
// One CTA per (KV segment, row tile, KV head, sequence), four warps.  Each
// warp streams its own 32-key steps (step i belongs to warp i mod 4) through
// its own ring of bulk copies, keeps its own (m, l, o), and the CTA merges the
// four at the end; segments are merged by combine_kernel.
//
// Lane layout (lane = 4 * u + t, u < 8, t < 4; "key index" i < 16 of a 16-key
// MMA tile is key rho(i) of it):
//   K: lane (u, t) holds key indexes u and u + 8 and a quarter of the dims;
//      the dims of an MMA's k index may be permuted as long as Q's are too, so
//      the quarter is whole 8- or 16-byte runs of codes.
//   S^T: lane holds key indexes u, u + 8 and rows 2t, 2t + 1 of each 8 rows.
//   P^T: two 8 x 8 transposes (movmatrix) turn S^T's layout into a B operand.
//   V: lane (u, t) holds key indexes 2t, 2t + 1, 2t + 8, 2t + 9 and dims
//      [u d / 8, (u + 1) d / 8); the nibbles of two keys are interleaved so that
//      one conversion yields (key a, key b) of one dim, the MMA's k pair.
//   O^T: lane holds those d / 8 dims of rows 2t, 2t + 1: rescaling needs no
//      exchange, rows line up with S^T's.
// rho pairs keys so that the K loads touch rows of different parity (two
// 64-byte rows fill the 32 banks).
#include <algorithm>
#include <cstdint>

#include "ua_common.cuh"
#include "ua_fp4.cuh"
#include "ua_fp4.h"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kW = 4;           // warps per CTA
constexpr int kStep = 32;       // keys per ring stage
constexpr int kDepth = 4;       // ring stages per warp
constexpr float kLazy4 = 8.0f;  // re-anchor when a step's max exceeds m by this (log2)

template <int D, int NT>
struct FCfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kKS = D / 16;                    // k steps of S^T, M tiles of O^T
    static constexpr int kCodeRow = D / 2;                // bytes of one key's codes
    static constexpr int kScaleRow = D / 16;
    static constexpr int kOp = kStep * (kCodeRow + kScaleRow);   // K or V of one step
    static constexpr int kStage = 2 * kOp;
    static constexpr int kRing = kDepth * kStage;         // per warp
    static constexpr int kOStride = D + 4;                // fp32 row stride of the merge (bank spread)
    static constexpr int kMerge = kRows * kOStride * 4;   // one warp's o, in its own ring
    static_assert(kMerge <= kRing, "merge area");
    static_assert(kOp % 16 == 0, "bulk copy alignment");
    static constexpr int kOffQ = kW * kRing;              // Q^T in fragment order, f16
    static constexpr int kOffMl = kOffQ + NT * kKS * 32 * 8;   // (m, l) [kW][kRows] x 2
    static constexpr int kOffQs = kOffMl + kW * kRows * 8;     // power-of-two scale of each Q row
    static constexpr int kOffBar = kOffQs + kRows * 4;
    static constexpr int kSmem = kOffBar + (kW * kDepth + 1) * 8 + 128;
    static_assert(kSmem <= 232448, "shared memory budget");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}

// Contiguous copy global -> shared (16-byte aligned, a multiple of 16 bytes),
// completion signalled on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Key of a 16-key tile that MMA key index i < 8 stands for (index i + 8: + 8).
__device__ __forceinline__ int rho(int i) { return (i & 1) ? ((i >> 1) + 4) ^ 1 : i >> 1; }

// K codes of one key that lane t holds: D / 4 dims as N words of 8 dims.
template <int D>
__device__ __forceinline__ void load_k_words(const uint8_t* row, int t, uint32_t (&w)[D / 32]) {
    if constexpr (D == 64) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + t * 8);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int c = 0; c < D / 128; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + c * 64 + t * 16);
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
        }
    }
}

// Their scales as f16x2 splats, one per two words (16 dims).
template <int D>
__device__ __forceinline__ void load_k_scales(const uint8_t* row, int t, uint32_t (&s)[D / 64]) {
    if constexpr (D == 64) {
        s[0] = splat_lo(e4m3x2_to_f16(row[t]));
    } else {
#pragma unroll
        for (int c = 0; c < D / 128; ++c) {
            const uint32_t h = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(row + c * 8 + t * 2));
            s[2 * c] = splat_lo(h);
            s[2 * c + 1] = splat_hi(h);
        }
    }
}

// Position of dim e in the fragment-ordered Q^T of one row: (k step, lane
// quarter t, half index 0..3).
template <int D>
__device__ __forceinline__ void q_place(int e, int& step, int& t, int& half) {
    constexpr int kRun = D == 64 ? 16 : 32;      // contiguous dims of a lane
    const int c = e / (4 * kRun), r = e % (4 * kRun);
    t = r / kRun;
    step = c * (kRun / 4) + (r % kRun) / 4;
    half = r & 3;
}

// GEN: softcap, ALiBi or QQ-bias in the score chain.  EMIT: also store every
// row's scores (log2 units) for the key-weight kernel, and always write
// partials.
template <int D, int NT, bool GEN, bool EMIT>
__global__ void __launch_bounds__(kW * 32, (D == 256 ? 1 : NT == 1 ? 3 : 2))
fp4_kernel(const FwdParams p) {
    using C = FCfg<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int u = lane >> 2, t = lane & 3;
    const int s = blockIdx.z;
    const int hkv = blockIdx.y;
    const int rt = blockIdx.x / p.splits;
    const int seg = blockIdx.x % p.splits;
    const bool split = EMIT || p.splits > 1;
    const int g = p.g;

    int sq, sk;
    int64_t q0;
    const uint32_t st = seq_status(p, s, sq, sk, q0);
    if (st && hkv == 0 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, (int)st);
    if (st & UA_DEVERR_CU_SEQLENS) return;
    const int64_t r0 = (int64_t)rt * C::kRows;          // first packed row of the tile
    const int64_t all_rows = (int64_t)g * sq;
    if (r0 >= all_rows) return;
    if (seg >= (split ? seq_segments(p, st, sk) : 1)) return;
    const int nrows = (int)min((int64_t)C::kRows, all_rows - r0);
    const int ctx = sk - sq;
    const bool causal = (p.flags & UA_FLAG_CAUSAL) != 0;
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;
    // Keys any row of the tile sees.
    const int i_first = (int)(r0 / g), i_last = (int)((r0 + nrows - 1) / g);
    int k_end = causal ? min(sk, i_last + ctx + 1) : sk;
    int k_beg = window ? max(0, i_first + ctx - p.window + 1) : 0;
    const int vis_beg = k_beg, vis_end = k_end;
    if (split) {
        k_beg = max(k_beg, seg * p.chunk);
        k_end = (int)min((int64_t)k_end, (int64_t)seg * p.chunk + p.chunk);
    }
    auto out_row = [&](int r) {
        const int64_t rg = r0 + r;
        return (q0 + rg / g) * p.hq + (int64_t)hkv * g + rg % g;
    };
    if (st || k_beg >= k_end) {
        // Malformed lengths (rows written as zeros) or a segment no row sees.
        for (int e = threadIdx.x; e < nrows * D; e += kW * 32) {
            const int64_t row = out_row(e / D);
            if (split) {
                if (e % D == 0) {
                    p.part_ml[(row * p.splits + seg) * 2 + 0] = -INFINITY;
                    p.part_ml[(row * p.splits + seg) * 2 + 1] = 0.f;
                }
            } else {
                p.out[row * D + e % D] = __float2bfloat16_rn(0.f);
            }
        }
        return;
    }
    const int t_begin = k_beg / kStep;
    const int n_steps = (k_end + kStep - 1) / kStep - t_begin;
    const int my_steps = (n_steps - warp + kW - 1) / kW;     // steps warp, warp + kW, ...

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    const uint32_t bar0 = smem_u32(bars + warp * kDepth);
    const uint32_t never = smem_u32(bars + kW * kDepth);
    uint8_t* ring = smem + warp * C::kRing;
    float* ml = reinterpret_cast<float*>(smem + C::kOffMl);
    float* q_scale = reinterpret_cast<float*>(smem + C::kOffQs);
    if (lane == 0) {
        for (int i = 0; i < kDepth; ++i) mbar_init(bar0 + 8 * i, 1);
        if (warp == 0) mbar_init(never, 1);
        fence_mbar_init();
    }
    __syncwarp();

    // ---- ring: copies of a step are issued by the lanes 4 * unit + 2 * part + op
    // (op: K or V; part: codes or scales; unit: paged block of the step -- two
    // at b = 16, else one).  Block ids are fetched one step ahead.
    const int b = p.b;
    const int units = b == 16 ? 2 : 1;
    const int urows = kStep / units;
    const int nblk = (sk + b - 1) / b;
    const int unit = lane >> 2, part = (lane >> 1) & 1, op = lane & 1;
    const int32_t* bt = p.block_table + (int64_t)s * p.bt_stride;
    const int64_t page_bytes = fp4_page_bytes(b, D);
    auto step_key = [&](int i) { return (t_begin + warp + i * kW) * kStep; };
    auto block_of = [&](int i) -> int32_t {      // -2: no such block in this step
        if (unit >= units || i >= my_steps) return -2;
        const int blk = (step_key(i) + unit * 16) / b;
        return blk < nblk ? __ldg(bt + blk) : -2;
    };
    const uint32_t copy_bytes = (uint32_t)urows * (part ? C::kScaleRow : C::kCodeRow);
    const uint32_t dst_off = (uint32_t)op * C::kOp +
                             (part ? (uint32_t)kStep * C::kCodeRow + unit * 16 * C::kScaleRow
                                   : (uint32_t)unit * 16 * C::kCodeRow);
    auto issue = [&](int i, int32_t id) {
        const int slot = i % kDepth;
        const uint32_t bar = bar0 + 8 * slot;
        uint8_t* dst = ring + slot * C::kStage + dst_off;
        const bool here = id != -2;
        const bool good = here && id >= 0 && (int64_t)id < p.num_blocks;
        const unsigned mask = __ballot_sync(0xffffffffu, good);
        if (here && !good) {
            // A bad block: its keys read as zeros (the slots are later
            // overwritten by copies, hence the proxy fence).
            atomicOr(p.err, (int)UA_DEVERR_BLOCK_ID);
            for (uint32_t e = 0; e < copy_bytes; e += 4) *reinterpret_cast<uint32_t*>(dst + e) = 0;
            fence_proxy_async_smem();
        }
        if (lane == 0)
            mbar_arrive_expect_tx(bar, (uint32_t)__popc(mask & 0x11u) * 2u * urows * (C::kCodeRow + C::kScaleRow));
        __syncwarp();
        if (good) {
            const int row = step_key(i) % b & ~(urows - 1);
            const uint8_t* page = static_cast<const uint8_t*>(op ? p.v_cache : p.k_cache) +
                                  ((int64_t)id * p.hk + hkv) * page_bytes;
            bulk_load(smem_u32(dst),
                      part ? page + (int64_t)b * C::kCodeRow + row * C::kScaleRow : page + row * C::kCodeRow,
                      copy_bytes, bar);
        }
    };
    int32_t id_next = block_of(0);
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        const int32_t id = id_next;
        id_next = block_of(i + 1);
        if (i < my_steps) issue(i, id);
    }

    // ---- Q: f16 in fragment order, each row scaled by a power of two so that
    // its largest magnitude lies in [1, 2) (f16 covers 2^-24 below that; the
    // factor goes into the row's score scale).
    for (int r = threadIdx.x >> 3; r < C::kRows; r += kW * 4) {
        constexpr int kPer = D / 8;
        const int e0 = (threadIdx.x & 7) * kPer;
        uint4 w[kPer / 8];
        uint32_t amax = 0;
#pragma unroll
        for (int c = 0; c < kPer / 8; ++c) {
            w[c] = r < nrows ? __ldg(reinterpret_cast<const uint4*>(p.q + out_row(r) * D + e0) + c)
                             : make_uint4(0, 0, 0, 0);
            const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                amax = max(amax, v[k] & 0x7fffu);
                amax = max(amax, (v[k] >> 16) & 0x7fffu);
            }
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
        // Exponent field of the largest magnitude, kept where 2^-e is normal
        // (zeros, infinities and NaN: unscaled).
        const int ef = (int)(amax >> 7);
        const int e = (amax == 0 || ef == 255) ? 0 : min(max(ef, 1), 253) - 127;
        const float down = __int_as_float((127 - e) << 23);
        if ((threadIdx.x & 7) == 0) q_scale[r] = __int_as_float((127 + e) << 23);
#pragma unroll
        for (int c = 0; c < kPer / 8; ++c) {
            const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                int step, tt, half;
                q_place<D>(e0 + c * 8 + k * 2, step, tt, half);
                const uint32_t a = pack_f16x2(bf16_lo(v[k]) * down, bf16_hi(v[k]) * down);
                const uint32_t bb = pack_f16x2(bf16_lo(v[k + 1]) * down, bf16_hi(v[k + 1]) * down);
                uint2* dst = reinterpret_cast<uint2*>(smem + C::kOffQ) +
                             (((r >> 3) * C::kKS + step) * 32 + (r & 7) * 4 + tt);
                *dst = make_uint2(a, bb);
            }
        }
    }
    __syncthreads();

    // ---- per-lane row constants: rows 8 n + 2t + c
    float m[NT][2], l[NT][2], fac[NT][2], slope[NT][2];
    int rlo[NT][2], rhi[NT][2], ri[NT][2];
    int full_lo = 0, full_hi = 0x7fffffff;       // keys every row of the tile sees
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = 8 * n + 2 * t + c;
            const int i = (int)((r0 + min(r, nrows - 1)) / g);
            m[n][c] = -INFINITY;
            l[n][c] = 0.f;
            ri[n][c] = i;
            rhi[n][c] = causal ? min(i + ctx, sk - 1) : sk - 1;
            rlo[n][c] = window ? max(0, i + ctx - p.window + 1) : 0;
            full_lo = max(full_lo, rlo[n][c]);
            full_hi = min(full_hi, rhi[n][c]);
            const float tau = p.scale * p.k_scale * q_scale[r];
            fac[n][c] = GEN ? tau : tau * kLog2e;
            slope[n][c] = 0.f;
            if (GEN && (p.flags & UA_FLAG_ALIBI) && r < nrows)
                slope[n][c] = __ldg(p.alibi + (int64_t)hkv * g + (r0 + r) % g);
            // Rows that do not exist see what the last row sees: their results
            // are never stored, and tile-wide tests stay simple.
        }
    full_lo = max(full_lo, __shfl_xor_sync(0xffffffffu, full_lo, 1));
    full_lo = max(full_lo, __shfl_xor_sync(0xffffffffu, full_lo, 2));
    full_hi = min(full_hi, __shfl_xor_sync(0xffffffffu, full_hi, 1));
    full_hi = min(full_hi, __shfl_xor_sync(0xffffffffu, full_hi, 2));
    const bool softcap = GEN && (p.flags & UA_FLAG_SOFTCAP) != 0;
    const bool alibi = GEN && (p.flags & UA_FLAG_ALIBI) != 0;
    const bool qq = GEN && (p.flags & UA_FLAG_QQ_BIAS) != 0;

    float o[C::kKS][NT][4];
#pragma unroll
    for (int i = 0; i < C::kKS; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[i][n][c] = 0.f;
    const uint2* qf = reinterpret_cast<const uint2*>(smem + C::kOffQ) + lane;

    bool ok = true;
    int done = 0;       // steps whose copies have been waited for
    if (p.stall) {
        // Testing hook: the first K/V wait waits on a barrier that nothing
        // completes and gives up after stall_ns.
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(never, 0, (uint64_t)p.stall_ns));
    }
    for (int i = 0; ok && i < my_steps; ++i) {
        const int slot = i % kDepth;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + 8 * slot, (i / kDepth) & 1))) {
            ok = false;
            break;
        }
        done = i + 1;
        uint8_t* kst = ring + slot * C::kStage;
        uint8_t* vst = kst + C::kOp;
        const int key0 = step_key(i);
        if (key0 < vis_beg || key0 + kStep > vis_end) {
            // Keys no row of the tile sees (past the end, before the window):
            // their V scales become 0, so that whatever the slots hold cannot
            // reach O (0 * NaN is NaN; codes are always finite).
            const int key = key0 + lane;
            if (key < vis_beg || key >= vis_end) {
                uint8_t* sc = vst + kStep * C::kCodeRow + lane * C::kScaleRow;
#pragma unroll
                for (int e = 0; e < C::kScaleRow; e += 4) *reinterpret_cast<uint32_t*>(sc + e) = 0;
                fence_proxy_async_smem();
            }
            __syncwarp();
        }

        // S^T = K Q^T for two 16-key tiles.
        float sacc[2][NT][4];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) sacc[kt][n][c] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            const int ka = kt * 16 + rho(u), kb = ka + 8;
            uint32_t wa[D / 32], wb[D / 32], sa[D / 64], sb[D / 64];
            load_k_words<D>(kst + ka * C::kCodeRow, t, wa);
            load_k_words<D>(kst + kb * C::kCodeRow, t, wb);
            load_k_scales<D>(kst + kStep * C::kCodeRow + ka * C::kScaleRow, t, sa);
            load_k_scales<D>(kst + kStep * C::kCodeRow + kb * C::kScaleRow, t, sb);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t ha[4], hb[4];
                e2m1x8_to_f16(wa[w], ha);
                e2m1x8_to_f16(wb[w], hb);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    ha[k] = mul_f16x2(ha[k], sa[w / 2]);
                    hb[k] = mul_f16x2(hb[k], sb[w / 2]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint2 qv = qf[(n * C::kKS + 2 * w + k) * 32];
                        mma_f16(sacc[kt][n], ha[2 * k], hb[2 * k], ha[2 * k + 1], hb[2 * k + 1], qv.x, qv.y);
                    }
            }
        }

        // Score chain, masks, running maximum.
        const bool full = key0 >= full_lo && key0 + kStep - 1 <= full_hi;
        float tmax[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) tmax[n][0] = tmax[n][1] = -INFINITY;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) {
                    const int c = c4 & 1;
                    const int key = key0 + kt * 16 + rho(u) + (c4 >> 1) * 8;
                    float x = sacc[kt][n][c4] * fac[n][c];
                    if constexpr (GEN) {
                        if (softcap) x = p.softcap * tanh_from_exp2(x / p.softcap);
                        if (alibi) x += slope[n][c] * (float)(key - ctx);
                        if (qq && key >= ctx && key <= rhi[n][c])
                            x += __ldg(p.qq_bias + (int64_t)ri[n][c] * p.qq_stride + (key - ctx));
                        x *= kLog2e;
                    }
                    if (!full && (key < rlo[n][c] || key > rhi[n][c])) x = -INFINITY;
                    if constexpr (EMIT) {
                        const int r = 8 * n + 2 * t + c;
                        if (r < nrows && key < sk) p.scores[out_row(r) * p.score_stride + key] = x;
                    }
                    sacc[kt][n][c4] = x;
                    tmax[n][c] = fmaxf(tmax[n][c], x);
                }
        bool up = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) up |= tmax[n][c] > m[n][c] + kLazy4;
        if (__any_sync(0xffffffffu, up)) {
            // Re-anchor rows whose step maximum (over the 8 lanes that share
            // the row) exceeds m by more than the threshold.
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = tmax[n][c];
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    if (v > m[n][c] + kLazy4) {
                        const float a = fast_exp2(m[n][c] - v);
                        m[n][c] = v;
                        l[n][c] *= a;
#pragma unroll
                        for (int k = 0; k < C::kKS; ++k) {
                            o[k][n][c] *= a;
                            o[k][n][c + 2] *= a;
                        }
                    }
                }
        }

        // P = 2^(x - m): fp32 into the row sums, f16 into the MMA (11 bits;
        // m trails the maximum by at most 8, so P <= 2^8).
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
                const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
                float e[4];
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) {
                    e[c4] = fast_exp2(sacc[kt][n][c4] - ((c4 & 1) ? m1 : m0));
                    l[n][c4 & 1] += e[c4];
                }
                pb[kt][n][0] = transpose8(pack_f16x2(e[0], e[1]));
                pb[kt][n][1] = transpose8(pack_f16x2(e[2], e[3]));
            }

        // O^T += V^T P^T.
        constexpr int kVW = D / 64;              // words of 8 dims per lane and key
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
            for (int w = 0; w < kVW; ++w) {
                uint32_t h[2][2][4];             // [key pair][dim parity][byte]
#pragma unroll
                for (int pr = 0; pr < 2; ++pr) {
                    const int ka = kt * 16 + pr * 8 + t, kb = kt * 16 + pr * 8 + ((t + 4) ^ 1);
                    const uint32_t a = *reinterpret_cast<const uint32_t*>(vst + ka * C::kCodeRow + u * (D / 16) + w * 4);
                    const uint32_t c = *reinterpret_cast<const uint32_t*>(vst + kb * C::kCodeRow + u * (D / 16) + w * 4);
                    const int gi = (u * (D / 8) + w * 8) / 16;   // scale group of these dims
                    const uint8_t* sc = vst + kStep * C::kCodeRow + gi;
                    const uint32_t sp = e4m3x2_to_f16((uint32_t)sc[ka * C::kScaleRow] |
                                                      ((uint32_t)sc[kb * C::kScaleRow] << 8));
                    e2m1x8_to_f16((a & 0x0f0f0f0fu) | ((c & 0x0f0f0f0fu) << 4), h[pr][0]);
                    e2m1x8_to_f16(((a >> 4) & 0x0f0f0f0fu) | (c & 0xf0f0f0f0u), h[pr][1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        h[pr][0][k] = mul_f16x2(h[pr][0][k], sp);
                        h[pr][1][k] = mul_f16x2(h[pr][1][k], sp);
                    }
                }
                // M tile (w, k): row u = dim 8w + 2k of the lane's run, row u + 8 the next.
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16(o[w * 4 + k][n], h[0][0][k], h[0][1][k], h[1][0][k], h[1][1][k], pb[kt][n][0],
                                pb[kt][n][1]);
            }
        }
        __syncwarp();
        const int32_t id = id_next;
        id_next = block_of(i + kDepth + 1);
        if (i + kDepth < my_steps) issue(i + kDepth, id);
    }
    if (!ok) {
        // Let every copy this warp issued land before the CTA ends.
        if (lane == 0) atomicOr(p.err, (int)UA_DEVERR_TIMEOUT);
        for (int i = done; i < min(my_steps, done + kDepth); ++i)
            mbar_wait_bounded(bar0 + 8 * (i % kDepth), (i / kDepth) & 1);
        __syncwarp();
    }

    // ---- merge the warps: each leaves (m, l, o) in shared memory (o over its
    // own ring, every copy into which has been waited for).
    __syncwarp();
    float* om = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float v = l[n][c];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            const int r = 8 * n + 2 * t + c;
            if (u == 0) {
                ml[(warp * C::kRows + r) * 2] = m[n][c];
                ml[(warp * C::kRows + r) * 2 + 1] = v;
            }
            float* dst = om + r * C::kOStride + u * (D / 8);
#pragma unroll
            for (int k = 0; k < C::kKS; k += 2)
                *reinterpret_cast<float4*>(dst + 2 * k) =
                    make_float4(o[k][n][c], o[k][n][c + 2], o[k + 1][n][c], o[k + 1][n][c + 2]);
        }
    __syncthreads();
    for (int e = threadIdx.x; e < nrows * (D / 4); e += kW * 32) {
        const int r = e / (D / 4), d4 = e % (D / 4);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kW; ++w) M = fmaxf(M, ml[(w * C::kRows + r) * 2]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float a = fast_exp2(ml[(w * C::kRows + r) * 2] - M);
                L = fmaf(a, ml[(w * C::kRows + r) * 2 + 1], L);
                const float4 v = *reinterpret_cast<const float4*>(smem + w * C::kRing + (r * C::kOStride + d4 * 4) * 4);
                acc.x = fmaf(a, v.x, acc.x);
                acc.y = fmaf(a, v.y, acc.y);
                acc.z = fmaf(a, v.z, acc.z);
                acc.w = fmaf(a, v.w, acc.w);
            }
        }
        const int64_t row = out_row(r);
        float f = p.v_scale;
        if (split) {
            const int64_t at = (row * p.splits + seg) * D + d4 * 4;
            part_store(p, at, acc.x * f);
            part_store(p, at + 1, acc.y * f);
            part_store(p, at + 2, acc.z * f);
            part_store(p, at + 3, acc.w * f);
            if (d4 == 0) {
                p.part_ml[(row * p.splits + seg) * 2 + 0] = M;
                p.part_ml[(row * p.splits + seg) * 2 + 1] = L;
            }
            continue;
        }
        if (p.flags & UA_FLAG_SINKS) {
            // The sink joins the denominator (log2 units); +inf takes all of it.
            const float s2 = __ldg(p.sinks + (int64_t)hkv * g + (r0 + r) % g) * kLog2e;
            if (s2 == INFINITY) {
                L = 0.f;
            } else if (s2 > M) {
                const float a = M == -INFINITY ? 0.f : fast_exp2(M - s2);
                f *= a;
                L = L * a + 1.0f;
            } else if (s2 != -INFINITY) {
                L += fast_exp2(s2 - M);
            }
        }
        f = L > 0.f ? f * __frcp_rn(L) : 0.f;
        const uint32_t lo = pack_bf16x2(acc.x * f, acc.y * f), hi = pack_bf16x2(acc.z * f, acc.w * f);
        *reinterpret_cast<uint2*>(p.out + row * D + d4 * 4) = make_uint2(lo, hi);
    }
}

template <int D, int NT, bool GEN, bool EMIT>
cudaError_t launch_t(const Fp4Plan& plan, const FwdParams& p, cudaStream_t stream) {
    using C = FCfg<D, NT>;
    auto kern = fp4_kernel<D, NT, GEN, EMIT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(plan.splits * plan.row_tiles), (unsigned)p.hk, (unsigned)p.num_seqs);
    kern<<<grid, kW * 32, C::kSmem, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Fp4Plan& plan, const FwdParams& p, cudaStream_t stream) {
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI | UA_FLAG_QQ_BIAS)) != 0;
    const bool emit = p.scores != nullptr;
    if (plan.rows == 8) {
        if (emit) return launch_t<D, 1, true, true>(plan, p, stream);
        return gen ? launch_t<D, 1, true, false>(plan, p, stream) : launch_t<D, 1, false, false>(plan, p, stream);
    }
    if (emit) return launch_t<D, 2, true, true>(plan, p, stream);
    return gen ? launch_t<D, 2, true, false>(plan, p, stream) : launch_t<D, 2, false, false>(plan, p, stream);
}

}  // namespace

bool plan_fp4(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4Plan* plan) {
    *plan = Fp4Plan();
    const int64_t rows = (int64_t)p.g * p.max_seqlen_q;
    plan->rows = rows <= 8 ? 8 : 16;
    const int64_t tiles = (rows + plan->rows - 1) / plan->rows;
    // Segments of at least 512 keys (four steps per warp), about three waves
    // of the three CTAs an SM holds.
    const int64_t base = (int64_t)p.hk * p.num_seqs * tiles;
    const int64_t want = (9LL * num_sms + base - 1) / base;
    const int64_t by_len = std::max<int64_t>(1, p.max_seqlen_k / 512);
    int64_t splits = std::min<int64_t>(std::min<int64_t>(want, by_len), 64);
    const size_t per_split = (size_t)p.total_q * p.hq * (p.d + 2) * sizeof(float);
    splits = std::min<int64_t>(splits, per_split ? (int64_t)(workspace_bytes / per_split) : 1);
    splits = std::max<int64_t>(splits, 1);
    const int64_t per = (p.max_seqlen_k + splits - 1) / splits;
    plan->chunk = (int)std::min<int64_t>((per + 127) / 128 * 128, 1 << 30);
    plan->splits = (int)((p.max_seqlen_k + plan->chunk - 1) / plan->chunk);
    if (tiles * plan->splits > 0x7fffffffLL || p.hk > 65535) return false;
    plan->row_tiles = (int)tiles;
    plan->launches = plan->splits > 1 ? 2 : 1;
    return true;
}

cudaError_t launch_fp4(const Fp4Plan& plan, const FwdParams& p, cudaStream_t stream) {
    switch (p.d) {
        case 64: return launch_d<64>(plan, p, stream);
        case 128: return launch_d<128>(plan, p, stream);
        case 256: return launch_d<256>(plan, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ua
