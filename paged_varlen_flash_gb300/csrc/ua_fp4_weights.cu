// ua_fp4_weights.cu -- accumulated attention weight of every key of a 4-bit cache,
// for calls with many packed rows per KV head (an observation window, a chunk).
//
// Storing every row's scores costs 8 bytes per (row, key): with 128 rows per KV
// head and d = 128 seven times the cache itself.  S^T = K Q^T is computed a
// second time instead, from the K pages alone, with keys on the MMA's M: a thread
// owns a key and adds the weights 2^(x - lse) of its rows from the tile's columns,
// in row order -- no atomics, one order, nothing stored but the sum.  Whole calls,
// us, scores stored / computed again (32 / 8 heads, d = 128 where not said; the
// first with the attention kernel's earlier segments): 8 sequences of 1000 to 12000
// keys, 8 to 32 query tokens, 133 / 124; 16 of 4096, 32 tokens, 172 / 122; 2 of 6000,
// 200 tokens, 357 / 179; one prompt of 1000 tokens 1095 / 210; one of 30000 keys, 8
// tokens, 61 / 65; 4 of 9000, 2 KV heads, d = 256, 96 / 81 and with a softcap (a
// second tanh per score) 119 / 138.  Every call of the tcgen05 attention kernel
// takes this one, the two slower kinds with it: that kernel stores no scores.
// What bounds it: a CTA starts in 5 us (Q, the rows' denominators, the first
// pages); then 1.3 us per key tile with two CTAs on the SM, half conversion and
// half exponentials.
//
// The key tiles of all (sequence, KV head) pairs, in order, are cut into equal
// shares, one per resident CTA (two per SM up to d = 128), whatever the lengths
// are; a CTA takes its share in pieces of one pair, each over all row tiles that
// see any of its keys.  Roles (10 warps):
//   warps 0-3  thread = key: sums; also the constants of the row tile's rows;
//   warps 4-7  convert the K tiles to f16, 64 dims at a time (a ring of such
//              panels, so that one is converted while the last one is multiplied);
//              warps 0-7 convert Q, once per row tile;
//   warp 8     issues S^T, owns tensor memory (two tiles of up to 128 columns);
//   warp 9     bulk copies of the K pages into a ring of 4-bit tiles.
#include <algorithm>
#include <cstdint>

#include "ua_common.cuh"
#include "ua_fp4.cuh"
#include "ua_fp4.h"
#include "ua_fp4_tiles.cuh"
#include "ua_launch.h"
#include "ua_prefill_common.cuh"
#include "ua_ptx.cuh"
#include "ua_tc.cuh"
#include "ua_weights.h"

namespace ua {
namespace {

using namespace pf;

constexpr int kThreadsW = 320;
constexpr int kWarpMma = 8;
constexpr int kWarpPages = 9;
constexpr int kKeysW = 128;         // keys per tile
constexpr int kMaxRun = 16;         // key tiles per piece at most

template <int D>
struct KCfg {
    static constexpr int kPanels = D / 64;
    static constexpr int kPanel = kKeysW * 128;          // 128 rows x 64 dims, f16
    static constexpr int kSlots = D == 256 ? 6 : 3;      // f16 panels of K
    static constexpr int kRing = 2;                      // 4-bit K tiles
    static constexpr int kRaw = kKeysW * (D / 2 + D / 16);
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kPanels * kPanel;
    static constexpr int kOffRaw = kOffK + kSlots * kPanel;
    static constexpr int kOffSum = kOffRaw + kRing * kRaw;            // [kMaxRun][128] sums
    static constexpr int kOffScale = kOffSum + kMaxRun * kKeysW * 4;  // Q's row scales
    static constexpr int kOffRow = kOffScale + kRows * 4;             // [2][64] factors and -lse of two rows
    static constexpr int kOffSlope = kOffRow + 2 * kRows * 8;         // [2][128]
    static constexpr int kOffSee = kOffSlope + 2 * kRows * 4;         // [2][128] first and last key seen
    static constexpr int kOffBar = kOffSee + 2 * kRows * 8;
    // q_full, q_empty, {k full, k empty} [kSlots], {raw full, raw empty} [kRing],
    // s_full[2], s_empty[2], rows_full[2], drain
    static constexpr int kNumBars = 2 + 2 * kSlots + 2 * kRing + 7;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmem = kOffMisc + 16 + 32 + 1024;
    static constexpr int kCtas = D == 256 ? 1 : 2;
    static_assert(kSmem * kCtas <= 231424, "shared memory budget");
};

// A piece: key tiles [kt0, kt1) of one sequence and KV head.
struct Piece {
    int s, hkv, kt0, kt1;
    int sq, sk;
    int64_t q0;
};

// Where a CTA is in its share of the key tiles.
struct Walk {
    int64_t pos, end;      // tiles, counted over the batch
    int64_t base;          // tiles before sequence s
    int s;
};

__device__ __forceinline__ int64_t tiles_of(const FwdParams& p, int s, int& sq, int& sk, int64_t& q0) {
    const uint32_t st = seq_status(p, s, sq, sk, q0);
    return st || sq <= 0 ? 0 : (sk + kKeysW - 1) / kKeysW;
}

__device__ __forceinline__ bool next_piece(const FwdParams& p, Walk& w, Piece& pc) {
    if (w.pos >= w.end) return false;
    int64_t tiles;
    for (;;) {
        tiles = tiles_of(p, w.s, pc.sq, pc.sk, pc.q0);
        if (w.pos - w.base < tiles * p.hk) break;
        w.base += tiles * p.hk;
        ++w.s;
    }
    pc.s = w.s;
    pc.hkv = (int)((w.pos - w.base) / tiles);
    pc.kt0 = (int)((w.pos - w.base) % tiles);
    pc.kt1 = (int)min(min(tiles, (int64_t)pc.kt0 + kMaxRun), pc.kt0 + (w.end - w.pos));
    w.pos += pc.kt1 - pc.kt0;
    return true;
}

// One warp: the batch's tiles, and the sequence in which the CTA's share begins.
__device__ __forceinline__ Walk first_piece(const FwdParams& p) {
    const int lane = threadIdx.x & 31;
    int sq, sk;
    int64_t q0, total = 0;
    for (int s = lane; s < p.num_seqs; s += 32) total += tiles_of(p, s, sq, sk, q0);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= p.hk;
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    Walk w{min(total, share * blockIdx.x), min(total, share * blockIdx.x + share), 0, 0};
    if (w.pos >= w.end) return w;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
        const int64_t n = s0 + lane < p.num_seqs ? tiles_of(p, s0 + lane, sq, sk, q0) * p.hk : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, w.base + incl > w.pos);
        if (hit) {
            const int at = __ffs(hit) - 1;
            w.s = s0 + at;
            w.base += __shfl_sync(0xffffffffu, incl - n, at);
            break;
        }
        w.base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return w;
}

template <int D, bool GEN>
__global__ void __launch_bounds__(kThreadsW, KCfg<D>::kCtas)
fp4_weights_kernel(const FwdParams p, const float* in_w, float* out_w, int64_t stride, float decay) {
    using C = KCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = p.g;
    const bool causal = (p.flags & UA_FLAG_CAUSAL) != 0;
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;
    const int ppt = kRows / g;                           // positions per row tile
    Piece pc{};

    // Row tile rt: its rows and the key tiles [a, z) of the piece that any of them sees.
    struct Span {
        TileRows rows;
        int a, z;
    };
    auto span_of = [&](int rt) {
        Span w;
        const int ctx = pc.sk - pc.sq;
        w.rows = TileRows{pc.q0, pc.hkv, g, rt * ppt, min(rt * ppt + ppt, pc.sq) - 1};
        const int beg = window ? max(0, w.rows.first + ctx - p.window + 1) : 0;
        const int end = causal ? min(pc.sk, w.rows.last + ctx + 1) : pc.sk;
        w.a = max(pc.kt0, beg / kKeysW);
        w.z = min(pc.kt1, (end + kKeysW - 1) / kKeysW);
        return w;
    };
    auto row_tiles = [&]() { return (pc.sq + ppt - 1) / ppt; };
    auto columns = [&](const TileRows& r) { return ((r.last - r.first + 1) * g + 31) / 32 * 32; };

    uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    const uint32_t q_full = smem_u32(bar_mem), q_empty = q_full + 8;
    const uint32_t k_full0 = q_full + 16, k_empty0 = k_full0 + 8 * C::kSlots;
    const uint32_t raw_full0 = k_empty0 + 8 * C::kSlots, raw_empty0 = raw_full0 + 8 * C::kRing;
    const uint32_t s_full0 = raw_empty0 + 8 * C::kRing, s_empty0 = s_full0 + 16;
    const uint32_t rows_full0 = s_empty0 + 16, drain = rows_full0 + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    float* q_scale = reinterpret_cast<float*>(smem + C::kOffScale);
    float* sums = reinterpret_cast<float*>(smem + C::kOffSum);
    float4* row_const = reinterpret_cast<float4*>(smem + C::kOffRow);
    float* row_slope = reinterpret_cast<float*>(smem + C::kOffSlope);
    int2* row_see = reinterpret_cast<int2*>(smem + C::kOffSee);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 256);
        mbar_init(q_empty, 129);             // the MMAs and the readers of q_scale
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(k_full0 + 8 * i, 128);
            mbar_init(k_empty0 + 8 * i, 1);
        }
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(raw_full0 + 8 * i, 1);
            mbar_init(raw_empty0 + 8 * i, 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full0 + 8 * i, 1);
            mbar_init(s_empty0 + 8 * i, 128);
            mbar_init(rows_full0 + 8 * i, 128);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    Walk* shared_walk = reinterpret_cast<Walk*>(smem + C::kOffMisc + 16);
    if (warp == 0) {
        const Walk w = first_piece(p);
        if (lane == 0) *shared_walk = w;
    }
    if (warp == kWarpMma) {
        tc::tmem_alloc(smem_u32(tmem_slot), 256);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    Walk walk = *shared_walk;
    auto wwait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, p.err));
    };

    bool ok = true;
    int it = 0, qn = 0;                      // (row tile, key tile) pairs and row tiles so far, all pieces
    if (warp == kWarpMma) {
        const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
        const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
        while (ok && next_piece(p, walk, pc)) {
            for (int rt = 0; ok && rt < row_tiles(); ++rt) {
                const Span w = span_of(rt);
                if (w.a >= w.z) continue;
                const uint32_t idesc = tc::idesc_f16_f32(kKeysW, columns(w.rows), false, false);
                if (!(ok = wwait(q_full, qn & 1))) break;
                for (int kt = w.a; kt < w.z; ++kt, ++it) {
                    if (it >= 2 && !(ok = wwait(s_empty0 + 8 * (it & 1), ((it >> 1) + 1) & 1))) break;
                    for (int pn = 0; pn < C::kPanels; ++pn) {
                        const int at = it * C::kPanels + pn, slot = at % C::kSlots;
                        if (!(ok = wwait(k_full0 + 8 * slot, (at / C::kSlots) & 1))) break;
                        tc::fence_after_sync();
                        if (lane == 0) {
                            const uint64_t kp = kd + slot * (C::kPanel >> 4), qp = qd + pn * (C::kPanel >> 4);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_bf16(tmem + (it & 1) * 128, kp + k * 2, qp + k * 2, idesc, pn + k > 0 ? 1u : 0u);
                            tc::commit(k_empty0 + 8 * slot);
                            if (pn + 1 == C::kPanels) {
                                tc::commit(s_full0 + 8 * (it & 1));
                                if (kt + 1 == w.z) tc::commit(q_empty);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                ++qn;
            }
        }
        if (*abort_flag) {
            // No MMA of this thread may still run when tensor memory is freed.
            if (lane == 0) tc::commit(drain);
            __syncwarp();
            mbar_wait_bounded(drain, 0);
        }
    } else if (warp == kWarpPages) {
        // Lane = page of the tile; codes and scales go to the raw tile's two parts.
        const int b_log2 = 31 - __clz(p.b), pages = kKeysW >> b_log2;
        const int64_t page_bytes = fp4_page_bytes(p.b, D);
        const uint32_t code_bytes = (uint32_t)p.b * (D / 2), scale_bytes = (uint32_t)p.b * (D / 16);
        while (ok && next_piece(p, walk, pc)) {
            const int nblk = (pc.sk + p.b - 1) >> b_log2;
            const uint8_t* cache = static_cast<const uint8_t*>(p.k_cache) + pc.hkv * page_bytes;
            const int32_t* bt = p.block_table + (int64_t)pc.s * p.bt_stride;
            auto id_of = [&](int kt) -> int32_t {        // -2: no such page
                const int blk = (kt * kKeysW >> b_log2) + lane;
                return lane < pages && blk < nblk ? __ldg(bt + blk) : -2;
            };
            for (int rt = 0; ok && rt < row_tiles(); ++rt) {
                const Span w = span_of(rt);
                int32_t id_next = w.a < w.z ? id_of(w.a) : -2;
                for (int kt = w.a; kt < w.z; ++kt, ++it) {
                    const int slot = it % C::kRing;
                    const int32_t id = id_next;
                    if (kt + 1 < w.z) id_next = id_of(kt + 1);
                    if (it >= C::kRing && !(ok = wwait(raw_empty0 + 8 * slot, ((it / C::kRing) + 1) & 1))) break;
                    const bool good = id >= 0 && (int64_t)id < p.num_blocks;
                    const unsigned mask = __ballot_sync(0xffffffffu, good);
                    uint8_t* codes = smem + C::kOffRaw + slot * C::kRaw + lane * code_bytes;
                    uint8_t* scales = smem + C::kOffRaw + slot * C::kRaw + kKeysW * (D / 2) + lane * scale_bytes;
                    if (lane < pages && !good) {
                        // Bad blocks (reported by the attention kernel) and pages past
                        // the end are zeros; the slot is later overwritten by copies.
                        for (uint32_t e = 0; e < scale_bytes; e += 4) *reinterpret_cast<uint32_t*>(scales + e) = 0;
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_expect_tx(raw_full0 + 8 * slot, (uint32_t)__popc(mask) * (code_bytes + scale_bytes));
                    __syncwarp();
                    if (good) {
                        const uint8_t* src = cache + (int64_t)id * p.hk * page_bytes;
                        bulk_load(smem_u32(codes), src, code_bytes, raw_full0 + 8 * slot);
                        bulk_load(smem_u32(scales), src + code_bytes, scale_bytes, raw_full0 + 8 * slot);
                    }
                }
            }
        }
        if (*abort_flag)
            // Let every copy this warp issued land before the CTA ends.
            for (int j = max(0, it - C::kRing); j < it; ++j)
                mbar_wait_bounded(raw_full0 + 8 * (j % C::kRing), (j / C::kRing) & 1);
        __syncwarp();
    } else if (warp >= 4) {
        const int t = threadIdx.x & 127;
        const int half = t & 1, k0 = t >> 1;             // 32 dims of a panel; keys k0, k0 + 64
        while (ok && next_piece(p, walk, pc)) {
            for (int rt = 0; ok && rt < row_tiles(); ++rt) {
                const Span w = span_of(rt);
                if (w.a >= w.z) continue;
                if (qn > 0 && !(ok = wwait(q_empty, (qn - 1) & 1))) break;
                stage_q<D, 256, D == 256 ? 2 : 4>(p, w.rows, threadIdx.x, smem + C::kOffQ, q_scale);
                fence_proxy_async_smem();
                mbar_arrive(q_full);
                ++qn;
                for (int kt = w.a; kt < w.z; ++kt, ++it) {
                    const int raw_slot = it % C::kRing;
                    if (!(ok = wwait(raw_full0 + 8 * raw_slot, (it / C::kRing) & 1))) break;
                    const uint8_t* raw = smem + C::kOffRaw + raw_slot * C::kRaw;
#pragma unroll 1
                    for (int pn = 0; pn < C::kPanels; ++pn) {
                        const int at = it * C::kPanels + pn, slot = at % C::kSlots, chunk = 2 * pn + half;
                        uint4 codes[2];
                        uint32_t s8[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int k = k0 + 64 * i;
                            codes[i] = *reinterpret_cast<const uint4*>(raw + k * (D / 2) + chunk * 16);
                            s8[i] = *reinterpret_cast<const uint16_t*>(raw + kKeysW * (D / 2) + k * (D / 16) + chunk * 2);
                        }
                        if (at >= C::kSlots && !(ok = wwait(k_empty0 + 8 * slot, ((at / C::kSlots) + 1) & 1))) break;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            stage_codes(codes[i], s8[i], chunk, k0 + 64 * i, smem + C::kOffK + slot * C::kPanel);
                        fence_proxy_async_smem();
                        mbar_arrive(k_full0 + 8 * slot);
                    }
                    if (!ok) break;
                    mbar_arrive(raw_empty0 + 8 * raw_slot);
                }
            }
        }
    } else {
        const int t = threadIdx.x;
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const bool softcap = GEN && (p.flags & UA_FLAG_SOFTCAP) != 0;
        const bool alibi = GEN && (p.flags & UA_FLAG_ALIBI) != 0;
        const bool qq = GEN && (p.flags & UA_FLAG_QQ_BIAS) != 0;
        const float cap = p.softcap * kLog2e;
        while (ok && next_piece(p, walk, pc)) {
            const int sk = pc.sk, ctx = sk - pc.sq, n = seq_segments(p, 0u, sk);
            for (int i = pc.kt0; i < pc.kt1; ++i) sums[(i - pc.kt0) * kKeysW + t] = 0.f;
            for (int rt = 0; ok && rt < row_tiles(); ++rt) {
                const Span w = span_of(rt);
                if (w.a >= w.z) continue;
                if (qn > 0 && !(ok = wwait(q_empty, (qn - 1) & 1))) break;
                stage_q<D, 256, D == 256 ? 2 : 4>(p, w.rows, t, smem + C::kOffQ, q_scale);
                fence_proxy_async_smem();
                mbar_arrive(q_full);
                // Thread t lays out row t: scores are x = s * factor in log2 units (tanh's
                // argument with a softcap).  Rows that do not exist see nothing.
                float4* rc = row_const + (qn & 1) * (kRows / 2);
                float* slopes = row_slope + (qn & 1) * kRows;
                int2* see = row_see + (qn & 1) * kRows;
                float lse = INFINITY, slope = 0.f;
                int2 keys = make_int2(0x7fffffff, -1);
                if (w.rows.real(t)) {
                    const int pos = w.rows.pos(t), h = w.rows.head(t);
                    lse = row_lse(p, w.rows.row(p, t), h, n);
                    if (alibi) slope = __ldg(p.alibi + h) * kLog2e;
                    keys = make_int2(window ? max(0, pos + ctx - p.window + 1) : 0, causal ? min(pos + ctx, sk - 1) : sk - 1);
                }
                slopes[t] = slope;
                see[t] = keys;
                if (!(ok = wwait(q_full, qn & 1))) break;    // q_scale
                float* c2 = reinterpret_cast<float*>(rc + (t >> 1)) + (t & 1);
                c2[0] = p.scale * p.k_scale * q_scale[t] * (softcap ? 1.f / p.softcap : kLog2e);
                c2[2] = -lse;
                mbar_arrive(q_empty);
                mbar_arrive(rows_full0 + 8 * (qn & 1));
                if (!(ok = wwait(rows_full0 + 8 * (qn & 1), (qn >> 1) & 1))) break;
                ++qn;
                const int cols = columns(w.rows);
                const int full_lo = window ? max(0, w.rows.last + ctx - p.window + 1) : 0;
                const int full_hi = causal ? min(w.rows.first + ctx, sk - 1) : sk - 1;
                for (int kt = w.a; kt < w.z; ++kt, ++it) {
                    if (!(ok = wwait(s_full0 + 8 * (it & 1), (it >> 1) & 1))) break;
                    tc::fence_after_sync();
                    const int key = kt * kKeysW + t;
                    const bool edge = kt * kKeysW < full_lo || kt * kKeysW + kKeysW - 1 > full_hi;
                    float2 sum = make_float2(0.f, 0.f);      // even and odd rows
#pragma unroll 1
                    for (int c = 0; c < cols; c += 32) {
                        uint32_t x[32];
                        tc::ld32(trow + (it & 1) * 128 + c, x);
                        tc::wait_ld();
                        if constexpr (GEN) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float4 r = rc[(c + e) >> 1];
                                float v = __uint_as_float(x[e]) * (e & 1 ? r.y : r.x);
                                if (softcap) v = cap * tanh_from_exp2(v);
                                if (alibi) v += slopes[c + e] * (float)(key - ctx);
                                if (qq && key >= ctx && key <= see[c + e].y)
                                    v += __ldg(p.qq_bias + (int64_t)w.rows.pos(c + e) * p.qq_stride + (key - ctx)) * kLog2e;
                                x[e] = __float_as_uint(fast_exp2(v + (e & 1 ? r.w : r.z)));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float4 r = rc[(c + e) >> 1];
                                const float2 v = exp2_pair_f32(ffma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                                                     make_float2(r.x, r.y), make_float2(r.z, r.w)));
                                x[e] = __float_as_uint(v.x);
                                x[e + 1] = __float_as_uint(v.y);
                            }
                        }
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const int2 k = see[c + e];
                                if (key < k.x || key > k.y) x[e] = 0;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            sum = fadd2(sum, make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
                    }
                    sums[(kt - pc.kt0) * kKeysW + t] += sum.x + sum.y;
                    tc::fence_before_sync();
                    mbar_arrive(s_empty0 + 8 * (it & 1));
                }
            }
            if (!ok) break;
            const int64_t at = ((int64_t)pc.s * p.hk + pc.hkv) * stride;
            for (int kt = pc.kt0; kt < pc.kt1; ++kt) {
                const int key = kt * kKeysW + t;
                if (key >= sk) break;
                float v = sums[(kt - pc.kt0) * kKeysW + t];
                if (in_w && decay != 0.f && key < ctx) v = fmaf(decay, in_w[at + key], v);
                out_w[at + key] = v;
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 256);
    }
    griddep_wait();                          // runs beside the combine, and ends after it
}

template <int D>
cudaError_t launch_key_weights(const FwdParams& p, int num_sms, const float* in_w, float* out_w, int64_t stride,
                               float decay, cudaStream_t stream) {
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI | UA_FLAG_QQ_BIAS)) != 0;
    auto kern = gen ? fp4_weights_kernel<D, true> : fp4_weights_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    const double tiles = (double)((p.max_seqlen_k + kKeysW - 1) / kKeysW) * p.hk * p.num_seqs;
    const int ctas = (int)std::max(1., std::min(tiles, (double)num_sms * KCfg<D>::kCtas));
    return launch_early(kern, dim3((unsigned)ctas), kThreadsW, KCfg<D>::kSmem, stream, p, in_w, out_w, stride, decay);
}

}  // namespace

cudaError_t launch_fp4_weights(const FwdParams& p, int num_sms, const float* in_w, float* out_w, int64_t stride,
                               float decay, cudaStream_t stream) {
    switch (p.d) {
        case 64: return launch_key_weights<64>(p, num_sms, in_w, out_w, stride, decay, stream);
        case 128: return launch_key_weights<128>(p, num_sms, in_w, out_w, stride, decay, stream);
        case 256: return launch_key_weights<256>(p, num_sms, in_w, out_w, stride, decay, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ua
