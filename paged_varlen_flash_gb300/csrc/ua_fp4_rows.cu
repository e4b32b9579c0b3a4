// ua_fp4_rows.cu -- attention over a 4-bit cache for calls with many packed rows
// per KV head (prompt chunks, observation windows), on tcgen05.
//
// With a tile of 128 rows every cached value is used 128 times, so the values
// are worth a trip through shared memory: converter threads read codes and
// scales from the pages, write f16 tiles (code x scale is exact in f16) in the
// 128-byte-swizzled layout a TMA copy of a 16-bit cache would have, and the
// products are the prefill kernels': S = Q K^T and O += P V, tcgen05.mma with
// M = 128 rows, P in tensor memory over its own S tile.  Per 128-key tile at
// d = 128 the tensor pipe needs 1,024 cycles, the converters about 370 issue
// slots per SM sub-partition and the softmax about 600, so the three run side
// by side near the MMAs' pace.
//
// One CTA per (KV segment, tile of floor(128 / g) positions, KV head, sequence),
// heaviest tile first.  Roles (12 warps):
//   warps 0-3   softmax and epilogue: thread r owns row r (tensor-memory lane r)
//               and all 128 key columns of an S tile;
//   warps 4-7   converters: Q once (f16, each row scaled by a power of two into
//               [1, 2)), then K and V tiles; the next tile's codes are in
//               registers before the current one's stage is free;
//   warp 8      MMA issuer and tensor-memory owner: S(j + 1) goes out before it
//               waits for P(j), so the tensor pipe works through the softmax;
//   warps 9-11  complete the warpgroup that gives up registers.
// Tensor memory: S(0), S(1) in columns [0, 256), O in [256, 256 + d).
#include <algorithm>
#include <cstdint>

#include "ua_common.cuh"
#include "ua_fp4.cuh"
#include "ua_fp4.h"
#include "ua_prefill_common.cuh"
#include "ua_ptx.cuh"
#include "ua_tc.cuh"

namespace ua {
namespace {

using namespace pf;

constexpr int kBN = 128;           // keys per tile
constexpr int kThreadsR = 384;
constexpr int kWarpMmaR = 8;
// 128 x (224 + 168 + 112) registers are the 384 x 168 of the launch.
constexpr uint32_t kRegsSoftmaxR = 224;
constexpr uint32_t kRegsIssueR = 112;

template <int D>
struct RCfg {
    static constexpr int kStages = D == 256 ? 1 : 2;    // K and V tiles in shared memory
    static constexpr int kPanels = D / 64;
    static constexpr int kPanel = kBN * 128;            // 128 rows x 64 dims, f16
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kTile;
    static constexpr int kOffV = kOffK + kStages * kTile;
    static constexpr int kOffScale = kOffV + kStages * kTile;   // Q's row scales
    static constexpr int kOffBar = kOffScale + kRows * 4;
    // q_full, k_full, v_full, k_empty, v_empty [kStages], s_full[2], p_full[2],
    // o_done[2], drain, never
    static constexpr int kNumBars = 1 + 4 * kStages + 8;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmem = kOffMisc + 16 + 1024;
    static constexpr int kTmemO = 2 * kBN;
    static constexpr int kChunks = D / 32;              // 16-byte runs of codes per key
    static constexpr int kEach = kBN * kChunks / 128;   // of them per converter thread and tile
    static_assert(kSmem <= 232448, "shared memory budget");
};

// One tile's codes of a converter thread: run i is chunk (128 i + t) mod kChunks
// of key (128 i + t) / kChunks.
template <int D>
struct Codes {
    uint4 c[RCfg<D>::kEach];
    uint32_t s[RCfg<D>::kEach];    // two e4m3 scales
};

template <int D, bool GEN, bool EMIT>
__global__ void __launch_bounds__(kThreadsR, 1) fp4_rows_kernel(const FwdParams p) {
    using C = RCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int s = blockIdx.z;
    const int hkv = blockIdx.y;
    const int tiles = (int)(gridDim.x / p.splits);
    const int seg = blockIdx.x % p.splits;
    const int tile = tiles - 1 - blockIdx.x / p.splits;
    const bool split = EMIT || p.splits > 1;
    const int g = p.g;
    const int ppt = kRows / g;                   // positions per tile
    const int first = tile * ppt;

    int sq, sk;
    int64_t q0;
    const uint32_t st = seq_status(p, s, sq, sk, q0);
    if (st && hkv == 0 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, (int)st);
    if (st & UA_DEVERR_CU_SEQLENS) return;
    if (first >= sq) return;
    if (seg >= (split ? seq_segments(p, st, sk) : 1)) return;
    const int last = min(first + ppt, sq) - 1;
    const int ctx = sk - sq;
    const bool causal = (p.flags & UA_FLAG_CAUSAL) != 0;
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;
    // Keys any row of the tile sees, and this segment's.
    const int vis_beg = window ? max(0, first + ctx - p.window + 1) : 0;
    const int vis_end = causal ? min(sk, last + ctx + 1) : sk;
    int k_beg = vis_beg, k_end = vis_end;
    if (split) {
        k_beg = max(k_beg, seg * p.chunk);
        k_end = (int)min((int64_t)k_end, (int64_t)seg * p.chunk + p.chunk);
    }
    if (st || k_beg >= k_end) {
        // Malformed lengths (rows written as zeros) or a segment no row sees.
        for (int e = threadIdx.x; e < kRows * (D / 8); e += kThreadsR) {
            const int r = e / (D / 8), c = e % (D / 8), i = first + r / g;
            if (r >= g * ppt || i > last) continue;
            const int64_t row = (q0 + i) * p.hq + hkv * g + r % g;
            if (split) {
                if (c == 0) {
                    p.part_ml[(row * p.splits + seg) * 2 + 0] = -INFINITY;
                    p.part_ml[(row * p.splits + seg) * 2 + 1] = 0.f;
                }
            } else {
                *reinterpret_cast<uint4*>(p.out + row * D + c * 8) = make_uint4(0, 0, 0, 0);
            }
        }
        return;
    }
    const int t_begin = k_beg / kBN;
    const int n = (k_end + kBN - 1) / kBN - t_begin;

    uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    const uint32_t q_full = smem_u32(bar_mem);
    const uint32_t k_full0 = smem_u32(bar_mem + 1);
    const uint32_t v_full0 = k_full0 + 8 * C::kStages;
    const uint32_t k_empty0 = v_full0 + 8 * C::kStages;
    const uint32_t v_empty0 = k_empty0 + 8 * C::kStages;
    const uint32_t s_full0 = v_empty0 + 8 * C::kStages;
    const uint32_t p_full0 = s_full0 + 16;
    const uint32_t o_done0 = s_full0 + 32;
    const uint32_t drain = s_full0 + 48;
    const uint32_t never = s_full0 + 56;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    float* q_scale = reinterpret_cast<float*>(smem + C::kOffScale);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 128);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(k_full0 + 8 * i, 128);     // the converters
            mbar_init(v_full0 + 8 * i, 128);
            mbar_init(k_empty0 + 8 * i, 1);
            mbar_init(v_empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full0 + 8 * i, 1);
            mbar_init(p_full0 + 8 * i, kRows);
            mbar_init(o_done0 + 8 * i, 1);
        }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMmaR) {
        tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    auto wwait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, p.err));
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssueR));
        if (warp == kWarpMmaR) {
            // ------------------------------ MMA issuer ------------------------------
            constexpr uint32_t idesc_qk = tc::idesc_f16_f32(kRows, kBN, false, false);
            constexpr int kNV = D == 64 ? 64 : 128;      // dims per P.V MMA
            constexpr uint32_t idesc_pv = tc::idesc_f16_f32(kRows, kNV, false, true);
            const uint32_t sQ = smem_u32(smem + C::kOffQ);
            auto issue_qk = [&](int j) -> bool {
                const int stg = j % C::kStages;
                // Testing hook: the first K wait waits on a barrier that nothing
                // completes and gives up after stall_ns.
                if (p.stall && j == 0 &&
                    !__all_sync(0xffffffffu, wait_or_abort(never, 0, abort_flag, p.err, (uint64_t)p.stall_ns)))
                    return false;
                if (!wwait(k_full0 + 8 * stg, (j / C::kStages) & 1)) return false;
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint32_t kst = smem_u32(smem + C::kOffK) + stg * C::kTile;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int off = (k >> 2) * C::kPanel + (k & 3) * 32;
                        tc::mma_bf16(tmem + (j & 1) * kBN, tc::smem_desc_sw128(sQ + off, 16, 1024),
                                     tc::smem_desc_sw128(kst + off, 16, 1024), idesc_qk, k > 0 ? 1u : 0u);
                    }
                    tc::commit(s_full0 + 8 * (j & 1));
                    tc::commit(k_empty0 + 8 * stg);
                }
                __syncwarp();
                return true;
            };
            bool ok = wwait(q_full, 0) && issue_qk(0);
            for (int j = 0; ok && j < n; ++j) {
                // S(j + 1) overwrites P(j - 1), whose P.V this thread issued
                // before: MMAs of one thread run in issue order.
                if (j + 1 < n && !(ok = issue_qk(j + 1))) break;
                const int stg = j % C::kStages;
                if (!(ok = wwait(p_full0 + 8 * (j & 1), (j >> 1) & 1))) break;
                if (!(ok = wwait(v_full0 + 8 * stg, (j / C::kStages) & 1))) break;
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint32_t vst = smem_u32(smem + C::kOffV) + stg * C::kTile;
#pragma unroll
                    for (int k = 0; k < kBN / 16; ++k)
#pragma unroll
                        for (int h = 0; h < D / kNV; ++h)
                            // A = P from tensor memory (16 keys = 8 columns), B = V
                            // MN-major, two 64-dim panels.
                            tc::mma_bf16_ts(tmem + C::kTmemO + h * kNV, tmem + (j & 1) * kBN + k * 8,
                                            tc::smem_desc_sw128(vst + h * 2 * C::kPanel + k * 16 * 128, C::kPanel, 1024),
                                            idesc_pv, (j > 0 || k > 0) ? 1u : 0u);
                    tc::commit(o_done0 + 8 * (j & 1));
                    tc::commit(v_empty0 + 8 * stg);
                }
                __syncwarp();
            }
            if (*abort_flag) {
                // No MMA may still run when tensor memory is freed.
                if (lane == 0) tc::commit(drain);
                __syncwarp();
                mbar_wait_bounded(drain, 0);
            }
        }
    } else if (warp >= 4) {
        // -------------------------------- converters --------------------------------
        const int t = threadIdx.x - 128;
        const int b_log2 = 31 - __clz(p.b);
        const int nblk = (sk + p.b - 1) >> b_log2;
        const int32_t* bt = p.block_table + (int64_t)s * p.bt_stride;
        const int64_t page_bytes = fp4_page_bytes(p.b, D);
        auto key_of = [&](int j, int i) { return (t_begin + j) * kBN + (i * 128 + t) / C::kChunks; };
        const int chunk = t % C::kChunks;       // the same in every run: 128 is a multiple of kChunks
        // Block id of each run's key; -1: no key.
        int32_t id[C::kEach];
        auto fetch_ids = [&](int j) {
#pragma unroll
            for (int i = 0; i < C::kEach; ++i) {
                const int blk = key_of(j, i) >> b_log2;
                id[i] = j < n && blk < nblk ? __ldg(bt + blk) : -1;
                if (j < n && blk < nblk && (id[i] < 0 || (int64_t)id[i] >= p.num_blocks)) {
                    atomicOr(p.err, (int)UA_DEVERR_BLOCK_ID);
                    id[i] = -1;                 // a bad block: its keys read as zeros
                }
            }
        };
        auto load = [&](const void* cache, int j, bool visible_only, Codes<D>& x) {
#pragma unroll
            for (int i = 0; i < C::kEach; ++i) {
                const int key = key_of(j, i), slot = key & (p.b - 1);
                x.c[i] = make_uint4(0, 0, 0, 0);
                x.s[i] = 0;
                // Keys no row of the tile sees are zeros in V: whatever their
                // slots hold must not reach O (0 * NaN is NaN).
                if (id[i] < 0 || (visible_only && (key < vis_beg || key >= vis_end))) continue;
                const uint8_t* page = static_cast<const uint8_t*>(cache) + ((int64_t)id[i] * p.hk + hkv) * page_bytes;
                x.c[i] = __ldg(reinterpret_cast<const uint4*>(page + slot * (D / 2)) + chunk);
                x.s[i] = __ldg(reinterpret_cast<const uint16_t*>(page + p.b * (D / 2) + slot * (D / 16)) + chunk);
            }
        };
        // Dims 32 chunk .. + 31 of the run's key: panel chunk / 2, four 16-byte
        // units, 128-byte swizzled.
        auto convert = [&](const Codes<D>& x, int j, uint8_t* tile_mem) {
#pragma unroll
            for (int i = 0; i < C::kEach; ++i) {
                const int k = key_of(j, i) & (kBN - 1);
                uint8_t* row = tile_mem + (chunk >> 1) * C::kPanel + k * 128;
                const uint32_t sc = e4m3x2_to_f16(x.s[i]), s0 = splat_lo(sc), s1 = splat_hi(sc);
                const uint32_t w[4] = {x.c[i].x, x.c[i].y, x.c[i].z, x.c[i].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t h[4];
                    e2m1x8_to_f16(w[q], h);
                    const uint32_t f = q < 2 ? s0 : s1;
                    *reinterpret_cast<uint4*>(row + ((((chunk & 1) * 4 + q) ^ (k & 7)) << 4)) =
                        make_uint4(mul_f16x2(h[0], f), mul_f16x2(h[1], f), mul_f16x2(h[2], f), mul_f16x2(h[3], f));
                }
            }
        };
        Codes<D> kx, vx;
        fetch_ids(0);
        load(p.k_cache, 0, false, kx);
        load(p.v_cache, 0, true, vx);
        fetch_ids(1);
        // Q: eight threads a row, 16 rows at a time.
        for (int r = t >> 3; r < kRows; r += 16) {
            constexpr int kPer = D / 8;
            const int i = first + r / g, e0 = (t & 7) * kPer;
            const bool real = r < g * ppt && i <= last;
            uint4 x[kPer / 8];
            uint32_t amax = 0;
#pragma unroll
            for (int c = 0; c < kPer / 8; ++c) {
                x[c] = real ? __ldg(reinterpret_cast<const uint4*>(
                                  p.q + ((q0 + i) * p.hq + hkv * g + r % g) * D + e0) + c)
                            : make_uint4(0, 0, 0, 0);
                amax = __vmaxu2(amax, __vmaxu2(__vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu),
                                               __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu)));
            }
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
                const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[k]) : "f"(bf16_hi(v[k]) * down), "f"(bf16_lo(v[k]) * down));
                const int dim = e0 + c * 8;
                *reinterpret_cast<uint4*>(smem + C::kOffQ + (dim >> 6) * C::kPanel + r * 128 +
                                          ((((dim & 63) >> 3) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
        for (int j = 0; j < n; ++j) {
            const int stg = j % C::kStages;
            if (j >= C::kStages && !wwait(k_empty0 + 8 * stg, ((j / C::kStages) + 1) & 1)) break;
            convert(kx, j, smem + C::kOffK + stg * C::kTile);
            fence_proxy_async_smem();
            mbar_arrive(k_full0 + 8 * stg);
            load(p.k_cache, j + 1, false, kx);   // past the last tile every id is -1
            if (j >= C::kStages && !wwait(v_empty0 + 8 * stg, ((j / C::kStages) + 1) & 1)) break;
            convert(vx, j, smem + C::kOffV + stg * C::kTile);
            fence_proxy_async_smem();
            mbar_arrive(v_full0 + 8 * stg);
            load(p.v_cache, j + 1, true, vx);
            fetch_ids(j + 2);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmaxR));
        // ------------------------------ softmax, epilogue ------------------------------
        const int r = threadIdx.x;
        const int pos = first + r / g;
        const bool valid = r < g * ppt && pos <= last;
        const int head = hkv * g + r % g;
        const bool live = __any_sync(0xffffffffu, valid);   // else the warp only keeps the barriers going
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const int hi = causal ? min(pos + ctx, sk - 1) : sk - 1;
        const int lo = window ? max(0, pos + ctx - p.window + 1) : 0;
        const int full_hi = causal ? min(first + ctx, sk - 1) : sk - 1;   // keys every row sees
        const int full_lo = window ? max(0, last + ctx - p.window + 1) : 0;
        const bool softcap = GEN && (p.flags & UA_FLAG_SOFTCAP) != 0;
        const bool alibi = GEN && (p.flags & UA_FLAG_ALIBI) != 0;
        const bool qq = GEN && (p.flags & UA_FLAG_QQ_BIAS) != 0;
        const float slope = alibi && valid ? __ldg(p.alibi + head) : 0.f;
        const int64_t row = (q0 + pos) * p.hq + head;
        float m = -INFINITY, l = 0.f;
        bool ok = wwait(q_full, 0);              // q_scale
        const float tau = p.scale * p.k_scale * q_scale[r];
        const float fac = GEN ? tau : tau * kLog2e;
        for (int j = 0; ok && j < n; ++j) {
            if (!(ok = wwait(s_full0 + 8 * (j & 1), (j >> 1) & 1))) break;
            const int key0 = (t_begin + j) * kBN;
            const uint32_t s_col = trow + (j & 1) * kBN;
            bool reanchor = false;
            float alpha = 1.f;
            if (live) {
                uint32_t sr[kBN / 32][32];
                tc::fence_after_sync();
#pragma unroll
                for (int c = 0; c < kBN / 32; ++c) tc::ld32(s_col + c * 32, sr[c]);
                tc::wait_ld();
#pragma unroll
                for (int c = 0; c < kBN / 32; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float x = __uint_as_float(sr[c][e]) * fac;
                        if constexpr (GEN) {
                            const int key = key0 + c * 32 + e;
                            if (softcap) x = p.softcap * tanh_from_exp2(x / p.softcap);
                            if (alibi) x += slope * (float)(key - ctx);
                            if (qq && valid && key >= ctx && key <= hi)
                                x += __ldg(p.qq_bias + (int64_t)pos * p.qq_stride + (key - ctx));
                            x *= kLog2e;
                        }
                        sr[c][e] = __float_as_uint(x);
                    }
                if (key0 < full_lo || key0 + kBN - 1 > full_hi) {
#pragma unroll
                    for (int c = 0; c < kBN / 32; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int key = key0 + c * 32 + e;
                            if (key < lo || key > hi) sr[c][e] = __float_as_uint(-INFINITY);
                        }
                }
                if (EMIT && valid) {
                    // 128 consecutive floats a thread (the row stride is a
                    // multiple of 128), whole sectors by 32-byte stores.
                    float* dst = p.scores + row * p.score_stride + key0;
#pragma unroll
                    for (int c = 0; c < kBN / 32; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c * 32 + e),
                                         "r"(sr[c][e]), "r"(sr[c][e + 1]), "r"(sr[c][e + 2]), "r"(sr[c][e + 3]),
                                         "r"(sr[c][e + 4]), "r"(sr[c][e + 5]), "r"(sr[c][e + 6]), "r"(sr[c][e + 7])
                                         : "memory");
                }
                float mx[8];
#pragma unroll
                for (int a = 0; a < 8; ++a) mx[a] = -INFINITY;
#pragma unroll
                for (int c = 0; c < kBN / 32; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 16)
#pragma unroll
                        for (int a = 0; a < 8; ++a)
                            mx[a] = fmax3(mx[a], __uint_as_float(sr[c][e + 2 * a]), __uint_as_float(sr[c][e + 2 * a + 1]));
                const float top = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                reanchor = top > m + kLazy;
                if (reanchor) {
                    alpha = fast_exp2(m - top);
                    m = top;
                }
                // P = 2^(x - m): fp32 into the row sum, f16 over the first 64
                // columns of S (every S value of this row has been read).
                const float mu = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < kBN / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float p0 = fast_exp2(__uint_as_float(sr[c][e]) - mu);
                        const float p1 = fast_exp2(__uint_as_float(sr[c][e + 1]) - mu);
                        sum[(e >> 1) & 3] += p0 + p1;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[e / 2]) : "f"(p1), "f"(p0));
                    }
                    tc::st16(s_col + c * 16, pk);
                }
                l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
                tc::wait_st();
            }
            if (live && j > 0 && __any_sync(0xffffffffu, reanchor)) {
                // O holds the P.V of the tiles up to j - 1.  (S(j) being full
                // means that P.V(j - 2) is done, so the parity is unambiguous.)
                if (!(ok = wwait(o_done0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1))) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tc::ld32(trow + C::kTmemO + c * 32, o);
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                    tc::st32(trow + C::kTmemO + c * 32, o);
                }
                tc::wait_st();
            }
            tc::fence_before_sync();
            mbar_arrive(p_full0 + 8 * (j & 1));
        }
        if (ok) ok = wwait(o_done0 + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1);
        if (ok && live) {
            // tcgen05.ld is warp-collective: every lane of a live warp loads.
            tc::fence_after_sync();
            float f = p.v_scale;
            if (split) {
                if (valid) {
                    p.part_ml[(row * p.splits + seg) * 2 + 0] = m;
                    p.part_ml[(row * p.splits + seg) * 2 + 1] = l;
                }
            } else {
                float L = l;
                if (p.flags & UA_FLAG_SINKS) {
                    const float s2 = __ldg(p.sinks + head) * kLog2e;
                    if (s2 == INFINITY) {
                        L = 0.f;
                    } else if (s2 > m) {
                        const float a = m == -INFINITY ? 0.f : fast_exp2(m - s2);
                        f *= a;
                        L = L * a + 1.0f;
                    } else if (s2 != -INFINITY) {
                        L += fast_exp2(s2 - m);
                    }
                }
                f = L > 0.f ? f * __frcp_rn(L) : 0.f;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tc::ld32(trow + C::kTmemO + c * 32, o);
                tc::wait_ld();
                if (!valid) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                if (split) {
                    part_store32(p, (row * p.splits + seg) * D + c * 32, o);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + row * (int64_t)D + c * 32);
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        dst[e / 8] = make_uint4(pack_bf16x2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])),
                                                pack_bf16x2(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                                                pack_bf16x2(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])),
                                                pack_bf16x2(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
                }
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarpMmaR) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool GEN, bool EMIT>
cudaError_t launch_rows_t(const Fp4RowsPlan& plan, const FwdParams& p, cudaStream_t stream) {
    auto kern = fp4_rows_kernel<D, GEN, EMIT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(plan.tiles * plan.splits), (unsigned)p.hk, (unsigned)p.num_seqs);
    kern<<<grid, kThreadsR, RCfg<D>::kSmem, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_rows_d(const Fp4RowsPlan& plan, const FwdParams& p, cudaStream_t stream) {
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI | UA_FLAG_QQ_BIAS)) != 0;
    if (p.scores) return gen ? launch_rows_t<D, true, true>(plan, p, stream) : launch_rows_t<D, false, true>(plan, p, stream);
    return gen ? launch_rows_t<D, true, false>(plan, p, stream) : launch_rows_t<D, false, false>(plan, p, stream);
}

}  // namespace

bool plan_fp4_rows(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4RowsPlan* plan) {
    *plan = Fp4RowsPlan();
    if (p.g > kRows || (int64_t)p.g * p.max_seqlen_q < kFp4RowsMin) return false;
    const int ppt = kRows / p.g;
    const int64_t tiles = (p.max_seqlen_q + ppt - 1) / ppt;
    // Segments of at least four key tiles, as many as give two CTAs per SM.
    const int64_t base = (int64_t)p.hk * p.num_seqs * tiles;
    const int64_t want = (2LL * num_sms + base - 1) / base;
    const int64_t by_len = std::max<int64_t>(1, p.max_seqlen_k / (4 * kBN));
    int64_t splits = std::min<int64_t>(std::min<int64_t>(want, by_len), 64);
    const size_t per_split = fp4_workspace_bytes(p.total_q * p.hq, p.d);
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, (int64_t)(workspace_bytes / per_split)));
    const int64_t per = (p.max_seqlen_k + splits - 1) / splits;
    plan->chunk = (int)std::min<int64_t>((per + kBN - 1) / kBN * kBN, 1 << 30);
    plan->splits = (int)((p.max_seqlen_k + (int64_t)plan->chunk - 1) / plan->chunk);
    if (tiles * plan->splits > 0x7fffffffLL || p.hk > 65535) return false;
    plan->tiles = (int)tiles;
    return true;
}

cudaError_t launch_fp4_rows(const Fp4RowsPlan& plan, const FwdParams& p, cudaStream_t stream) {
    switch (p.d) {
        case 64: return launch_rows_d<64>(plan, p, stream);
        case 128: return launch_rows_d<128>(plan, p, stream);
        case 256: return launch_rows_d<256>(plan, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ua
