// ua_fp4_rows.cu -- attention over a 4-bit cache for calls with many packed rows
// per KV head (prompt chunks, observation windows), on tcgen05.
//
// With a tile of 128 rows every cached value is used 128 times, so the values
// are worth a trip through shared memory: converter threads read codes and
// scales from the pages, write f16 tiles (code x scale is exact in f16) in the
// 128-byte-swizzled layout a TMA copy of a 16-bit cache would have, and the
// products are the prefill kernels': S = Q K^T and O += P V, tcgen05.mma with
// M = 128 rows, P in tensor memory over its own S tile.
//
// One CTA per (KV segment, tile of floor(128 / g) positions, KV head, sequence),
// heaviest tile first.  Roles (15 warps):
//   warps 0-3   softmax and epilogue: thread r owns row r (tensor-memory lane r);
//               two passes over the tile's columns, 64 at a time (maximum, then
//               P), so the code stays small: four roles share each scheduler's
//               instruction cache, and a fully unrolled row cost 2-3 times as
//               many cycles per instruction;
//   warps 4-7   convert the K tiles, warps 8-11 the V tiles, both together Q
//               before (f16, each row scaled by a power of two into [1, 2));
//   warp 12     QK^T issuer and tensor-memory owner; S(j) waits for P.V(j - 2),
//               whose P its columns hold;
//   warp 13     bulk copies of the pages into a ring of 4-bit tiles;
//   warp 14     P.V issuer.  (One thread issuing both needed 2,500 cycles per
//               tile for MMAs of 1,024.)
// Key tiles are 128 keys, at d = 256 64 (shared memory).
//
// Measured: 1.55 us per tile of 128 x 128 at d = 128 (MMAs alone 0.52), the chain
// convert -> QK^T -> softmax -> P.V; 16 sequences of 4096 keys and 8 KV heads, 64
// rows each, 49 us; 8 of 1000 to 12000 keys in four segments 67 us, of which a
// third is a tail of CTAs with longer sequences than the others'.  Codes held in registers by the
// converters instead of the staged ring: 106 to 128 us for the latter.
// Tensor memory: S(0), S(1) in columns [0, 256), O in [256, 256 + d).
#include <algorithm>
#include <cstdint>

#include "ua_common.cuh"
#include "ua_fp4.cuh"
#include "ua_fp4.h"
#include "ua_fp4_tiles.cuh"
#include "ua_prefill_common.cuh"
#include "ua_ptx.cuh"
#include "ua_tc.cuh"

namespace ua {
namespace {

using namespace pf;

constexpr int kThreadsR = 480;
constexpr int kWarpQk = 12;        // also owns tensor memory
constexpr int kWarpCopy = 13;
constexpr int kCols = 64;          // columns of S a softmax thread holds at a time

template <int D>
struct RCfg {
    static constexpr int kBN = D == 256 ? 64 : 128;     // keys per tile
    static constexpr int kStages = D == 256 ? 1 : 2;    // f16 K and V tiles
    static constexpr int kRing = D == 64 ? 4 : 3;       // 4-bit K and V tiles
    static constexpr int kPanels = D / 64;
    static constexpr int kQPanel = kRows * 128;         // 128 rows x 64 dims, f16
    static constexpr int kPanel = kBN * 128;            // kBN keys x 64 dims, f16
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kRaw = kBN * (D / 2 + D / 16); // codes, then scales
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kPanels * kQPanel;
    static constexpr int kOffV = kOffK + kStages * kTile;
    static constexpr int kOffRawK = kOffV + kStages * kTile;
    static constexpr int kOffRawV = kOffRawK + kRing * kRaw;
    static constexpr int kOffScale = kOffRawV + kRing * kRaw;   // Q's row scales
    static constexpr int kOffBar = kOffScale + kRows * 4;
    // q_full, {k, v} x {full, empty} [kStages], {k, v} x {raw full, raw empty}
    // [kRing], s_full[2], p_full[2], o_done[2], drain[2], never
    static constexpr int kNumBars = 1 + 4 * kStages + 4 * kRing + 9;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmem = kOffMisc + 16 + 1024;
    static constexpr int kTmemO = 256;
    static constexpr int kChunks = D / 32;              // 16-byte runs of codes per key
    static constexpr int kEach = kBN * kChunks / 128;   // of them per converter thread and tile
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(kRaw % 16 == 0, "bulk copy alignment");
};

// The dims (one bit per 16) that are NaN in V at keys [lo, hi) of sequence s.
__device__ __noinline__ uint32_t nan_groups(const FwdParams& p, int s, int hkv, int lo, int hi) {
    const int scale_row = p.d / 16, b_log2 = 31 - __clz(p.b);
    const int64_t page_bytes = fp4_page_bytes(p.b, p.d);
    uint32_t found = 0;
    for (int key = lo; key < hi; ++key) {
        const int32_t id = __ldg(p.block_table + (int64_t)s * p.bt_stride + (key >> b_log2));
        if (id < 0 || (int64_t)id >= p.num_blocks) continue;       // reads as zeros
        const uint8_t* sc = static_cast<const uint8_t*>(p.v_cache) + ((int64_t)id * p.hk + hkv) * page_bytes +
                            p.b * (p.d / 2) + (key & (p.b - 1)) * scale_row;
        for (int e = 0; e < scale_row; ++e)
            if ((sc[e] & 0x7f) == 0x7f) found |= 1u << e;
    }
    return found;
}

template <int D, bool GEN>
__global__ void __launch_bounds__(kThreadsR, 1) fp4_rows_kernel(const FwdParams p) {
    using C = RCfg<D>;
    constexpr int kBN = C::kBN;
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
    const bool split = p.scores || p.splits > 1;   // key weights read the rows' (m, l)
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
    // Keys every row of the tile sees.
    const int full_lo = window ? max(0, last + ctx - p.window + 1) : 0;
    const int full_hi = causal ? min(first + ctx, sk - 1) : sk - 1;

    uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    const uint32_t q_full = smem_u32(bar_mem);
    constexpr int kS = 8 * C::kStages, kR = 8 * C::kRing;
    const uint32_t k_full0 = smem_u32(bar_mem + 1), v_full0 = k_full0 + kS;
    const uint32_t k_empty0 = v_full0 + kS, v_empty0 = k_empty0 + kS;
    const uint32_t rk_full0 = v_empty0 + kS, rv_full0 = rk_full0 + kR;
    const uint32_t rk_empty0 = rv_full0 + kR, rv_empty0 = rk_empty0 + kR;
    const uint32_t s_full0 = rv_empty0 + kR;
    const uint32_t p_full0 = s_full0 + 16;
    const uint32_t o_done0 = s_full0 + 32;
    const uint32_t drain = s_full0 + 48;
    const uint32_t never = s_full0 + 64;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile int* nan_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
    float* q_scale = reinterpret_cast<float*>(smem + C::kOffScale);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 256);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(k_full0 + 8 * i, 128);     // the converters
            mbar_init(v_full0 + 8 * i, 128);
            mbar_init(k_empty0 + 8 * i, 1);
            mbar_init(v_empty0 + 8 * i, 1);
        }
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(rk_full0 + 8 * i, 1);
            mbar_init(rv_full0 + 8 * i, 1);
            mbar_init(rk_empty0 + 8 * i, 128);
            mbar_init(rv_empty0 + 8 * i, 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full0 + 8 * i, 1);
            mbar_init(p_full0 + 8 * i, kRows);
            mbar_init(o_done0 + 8 * i, 1);
        }
        mbar_init(drain, 1);
        mbar_init(drain + 8, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        *nan_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpQk) {
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

    if (warp >= 12) {
        if (warp != kWarpCopy) {
            // ------------------------- MMA issuers (one thread each) -------------------------
            // Shared-memory descriptors are bases plus compile-time offsets (the
            // address field counts 16 bytes).
            bool ok = true;
            if (warp == kWarpQk) {
                constexpr uint32_t idesc = tc::idesc_f16_f32(kRows, kBN, false, false);
                const uint64_t qd = tc::smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
                const uint64_t kd = tc::smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
                ok = wwait(q_full, 0);
                for (int j = 0; ok && j < n; ++j) {
                    const int stg = j % C::kStages;
                    // Testing hook: the first K wait waits on a barrier that
                    // nothing completes and gives up after stall_ns.
                    if (p.stall && j == 0 &&
                        !(ok = __all_sync(0xffffffffu, wait_or_abort(never, 0, abort_flag, p.err, (uint64_t)p.stall_ns))))
                        break;
                    if (j >= 2 && !(ok = wwait(o_done0 + 8 * (j & 1), ((j - 2) >> 1) & 1))) break;
                    if (!(ok = wwait(k_full0 + 8 * stg, (j / C::kStages) & 1))) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const uint64_t kst = kd + stg * (C::kTile >> 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc::mma_bf16(tmem + (j & 1) * 128, qd + (k >> 2) * (C::kQPanel >> 4) + (k & 3) * 2,
                                         kst + (k >> 2) * (C::kPanel >> 4) + (k & 3) * 2, idesc, k > 0 ? 1u : 0u);
                        tc::commit(s_full0 + 8 * (j & 1));
                        tc::commit(k_empty0 + 8 * stg);
                    }
                    __syncwarp();
                }
            } else {
                constexpr int kNV = D == 64 ? 64 : 128;      // dims per P.V MMA
                constexpr uint32_t idesc = tc::idesc_f16_f32(kRows, kNV, false, true);
                const uint64_t vd = tc::smem_desc_sw128(smem_u32(smem + C::kOffV), C::kPanel, 1024);
                for (int j = 0; ok && j < n; ++j) {
                    const int stg = j % C::kStages;
                    if (!(ok = wwait(v_full0 + 8 * stg, (j / C::kStages) & 1))) break;
                    if (!(ok = wwait(p_full0 + 8 * (j & 1), (j >> 1) & 1))) break;
                    tc::fence_after_sync();
                    if (lane == 0) {
                        const uint64_t vst = vd + stg * (C::kTile >> 4);
#pragma unroll
                        for (int k = 0; k < kBN / 16; ++k)
#pragma unroll
                            for (int h = 0; h < D / kNV; ++h)
                                // A = P from tensor memory (16 keys = 8 columns), B = V
                                // MN-major, two 64-dim panels.
                                tc::mma_bf16_ts(tmem + C::kTmemO + h * kNV, tmem + (j & 1) * 128 + k * 8,
                                                vst + h * 2 * (C::kPanel >> 4) + k * 128, idesc,
                                                (j > 0 || k > 0) ? 1u : 0u);
                        tc::commit(o_done0 + 8 * (j & 1));
                        tc::commit(v_empty0 + 8 * stg);
                    }
                    __syncwarp();
                }
            }
            if (*abort_flag) {
                // No MMA of this thread may still run when tensor memory is freed.
                const uint32_t dr = drain + (warp == kWarpQk ? 0 : 8);
                if (lane == 0) tc::commit(dr);
                __syncwarp();
                mbar_wait_bounded(dr, 0);
            }
        } else {
            // ------------------------------ bulk copies ------------------------------
            // Pages are contiguous (codes, then scales); a tile is whole pages
            // (or, of a 64-key page at d = 256, one).  Lane = (page, operand);
            // codes and scales go to the tile's two parts.  Block ids are
            // fetched one tile ahead.
            const int b_log2 = 31 - __clz(p.b), page = lane >> 1, op = lane & 1;
            const int pages = kBN >> b_log2, nblk = (sk + p.b - 1) >> b_log2;
            const int64_t page_bytes = fp4_page_bytes(p.b, D);
            const uint8_t* cache = static_cast<const uint8_t*>(op ? p.v_cache : p.k_cache) + hkv * page_bytes;
            const int32_t* bt = p.block_table + (int64_t)s * p.bt_stride;
            const uint32_t code_bytes = (uint32_t)p.b * (D / 2), scale_bytes = (uint32_t)p.b * (D / 16);
            const uint32_t full0 = op ? rv_full0 : rk_full0, empty0 = op ? rv_empty0 : rk_empty0;
            uint8_t* ring = smem + (op ? C::kOffRawV : C::kOffRawK);
            auto id_of = [&](int j) -> int32_t {       // -2: no such page
                const int blk = ((t_begin + j) * kBN >> b_log2) + page;
                return j < n && page < pages && blk < nblk ? __ldg(bt + blk) : -2;
            };
            int32_t id_next = id_of(0);
            int issued = 0;
            for (int j = 0; j < n; ++j) {
                const int slot = j % C::kRing;
                const int32_t id = id_next;
                id_next = id_of(j + 1);
                if (j >= C::kRing && !wwait(empty0 + 8 * slot, ((j / C::kRing) + 1) & 1)) break;
                const bool good = id >= 0 && (int64_t)id < p.num_blocks;
                const unsigned mask = __ballot_sync(0xffffffffu, good);
                uint8_t* codes = ring + slot * C::kRaw + page * code_bytes;
                uint8_t* scales = ring + slot * C::kRaw + kBN * (D / 2) + page * scale_bytes;
                if (page < pages && !good) {
                    // A bad block's keys, and those past the last block, are
                    // zeros (scale 0; codes are always finite).  The slot is
                    // later overwritten by copies, hence the proxy fence.
                    if (id != -2) atomicOr(p.err, (int)UA_DEVERR_BLOCK_ID);
                    for (uint32_t e = 0; e < scale_bytes; e += 4) *reinterpret_cast<uint32_t*>(scales + e) = 0;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane < 2)
                    mbar_arrive_expect_tx(full0 + 8 * slot, (uint32_t)__popc(mask & (op ? 0xaaaaaaaau : 0x55555555u)) *
                                                                (code_bytes + scale_bytes));
                __syncwarp();
                if (good) {
                    const uint8_t* src = cache + (int64_t)id * p.hk * page_bytes;
                    bulk_load(smem_u32(codes), src, code_bytes, full0 + 8 * slot);
                    bulk_load(smem_u32(scales), src + code_bytes, scale_bytes, full0 + 8 * slot);
                }
                issued = j + 1;
            }
            if (*abort_flag)
                // Let every copy this warp issued land before the CTA ends.
                for (int j = max(0, issued - C::kRing); j < issued; ++j)
                    mbar_wait_bounded(full0 + 8 * (j % C::kRing), (j / C::kRing) & 1);
            __syncwarp();
        }
    } else if (warp >= 4) {
        // -------------------------------- converters --------------------------------
        const bool is_v = warp >= 8;
        const int t = threadIdx.x & 127;
        stage_q<D, 256, D == 256 ? 2 : 4>(p, TileRows{q0, hkv, g, first, last}, threadIdx.x - 128, smem + C::kOffQ, q_scale);
        fence_proxy_async_smem();
        mbar_arrive(q_full);
        const uint32_t full0 = is_v ? v_full0 : k_full0, empty0 = is_v ? v_empty0 : k_empty0;
        const uint32_t raw_full0 = is_v ? rv_full0 : rk_full0, raw_empty0 = is_v ? rv_empty0 : rk_empty0;
        uint8_t* tiles_mem = smem + (is_v ? C::kOffV : C::kOffK);
        const uint8_t* raw_mem = smem + (is_v ? C::kOffRawV : C::kOffRawK);
        // Run i of a thread: 16-byte chunk t mod kChunks of key 128 i / kChunks + t / kChunks.
        const int chunk = t % C::kChunks, k0 = t / C::kChunks;
        for (int j = 0; j < n; ++j) {
            const int stg = j % C::kStages, slot = j % C::kRing;
            if (!wwait(raw_full0 + 8 * slot, (j / C::kRing) & 1)) break;
            if (j >= C::kStages && !wwait(empty0 + 8 * stg, ((j / C::kStages) + 1) & 1)) break;
            const uint8_t* raw = raw_mem + slot * C::kRaw;
            uint8_t* tile_mem = tiles_mem + stg * C::kTile + (chunk >> 1) * C::kPanel;
            // Keys no row of the tile sees are zeros in V: whatever their slots
            // hold must not reach O (0 * NaN is NaN).  So are NaN scales of keys
            // that only some rows see; the epilogue gives those rows the NaN.
            const int key0 = (t_begin + j) * kBN;
            const bool edge = is_v && (key0 < full_lo || key0 + kBN - 1 > full_hi);
#pragma unroll 2
            for (int i = 0; i < C::kEach; ++i) {
                const int k = k0 + i * (128 / C::kChunks);
                const uint4 c = *reinterpret_cast<const uint4*>(raw + k * (D / 2) + chunk * 16);
                uint32_t s8 = *reinterpret_cast<const uint16_t*>(raw + kBN * (D / 2) + k * (D / 16) + chunk * 2);
                if (edge && (key0 + k < full_lo || key0 + k > full_hi)) {
                    if (key0 + k < vis_beg || key0 + k >= vis_end) {
                        s8 = 0;
                    } else if ((s8 & 0x7f) == 0x7f || (s8 & 0x7f00) == 0x7f00) {
                        if ((s8 & 0x7f) == 0x7f) s8 &= 0xff00;
                        if ((s8 & 0x7f00) == 0x7f00) s8 &= 0xff;
                        *nan_flag = 1;
                    }
                }
                stage_codes(c, s8, chunk, k, tile_mem);
            }
            fence_proxy_async_smem();
            mbar_arrive(full0 + 8 * stg);
            mbar_arrive(raw_empty0 + 8 * slot);
        }
    } else {
        // ------------------------------ softmax, epilogue ------------------------------
        const int r = threadIdx.x;
        const int pos = first + r / g;
        const bool valid = r < g * ppt && pos <= last;
        const int head = hkv * g + r % g;
        const bool live = __any_sync(0xffffffffu, valid);   // else the warp only keeps the barriers going
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const int hi = causal ? min(pos + ctx, sk - 1) : sk - 1;
        const int lo = window ? max(0, pos + ctx - p.window + 1) : 0;
        const bool softcap = GEN && (p.flags & UA_FLAG_SOFTCAP) != 0;
        const bool alibi = GEN && (p.flags & UA_FLAG_ALIBI) != 0;
        const bool qq = GEN && (p.flags & UA_FLAG_QQ_BIAS) != 0;
        const float slope = alibi && valid ? __ldg(p.alibi + head) * kLog2e : 0.f;
        const int64_t row = (q0 + pos) * p.hq + head;
        float m = -INFINITY, l = 0.f;
        bool ok = wwait(q_full, 0);              // q_scale
        const float tau = p.scale * p.k_scale * q_scale[r];
        // The score chain is in log2 units from the products on.  A factor of zero
        // (tau below fp32: tiny k_scale and query) would make NaN of masked scores;
        // at the smallest normal number every score still is 0 to 2^-100.
        const float cap = p.softcap * kLog2e, fac = fmaxf(tau * (softcap ? 1.f / p.softcap : kLog2e), 0x1p-126f);
        for (int j = 0; ok && j < n; ++j) {
            if (!(ok = wwait(s_full0 + 8 * (j & 1), (j >> 1) & 1))) break;
            const int key0 = (t_begin + j) * kBN;
            const uint32_t s_col = trow + (j & 1) * 128;
            const bool edge = key0 < full_lo || key0 + kBN - 1 > full_hi;
            bool reanchor = false;
            float alpha = 1.f;
            if (live) {
                tc::fence_after_sync();
                // First pass: the maximum.  Plain scores stay as the MMA left
                // them (their factor is positive); a general score chain is
                // finished here and written back for the second pass.
                float top = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < kBN; c += kCols) {
                    uint32_t x[kCols / 32][32];
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h) tc::ld32(s_col + c + h * 32, x[h]);
                    tc::wait_ld();
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h) {
                        const int key = key0 + c + h * 32;
                        if constexpr (GEN) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float v = __uint_as_float(x[h][e]) * fac;
                                if (softcap) v = cap * tanh_from_exp2(v);
                                if (alibi) v += slope * (float)(key + e - ctx);
                                if (qq && valid && key + e >= ctx && key + e <= hi)
                                    v += __ldg(p.qq_bias + (int64_t)pos * p.qq_stride + (key + e - ctx)) * kLog2e;
                                x[h][e] = __float_as_uint(v);
                            }
                        }
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (key + e < lo || key + e > hi) x[h][e] = __float_as_uint(-INFINITY);
                        }
                        if (GEN || edge) tc::st32(s_col + c + h * 32, x[h]);
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int a = 0; a < 4; ++a)
                                mx[a] = fmax3(mx[a], __uint_as_float(x[h][e + 2 * a]), __uint_as_float(x[h][e + 2 * a + 1]));
                        top = fmax3(top, fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    }
                }
                if (GEN || edge) tc::wait_st();
                if constexpr (!GEN) top *= fac;
                reanchor = top > m + kLazy;
                if (reanchor) {
                    alpha = fast_exp2(m - top);
                    m = top;
                }
                // Second pass: P = 2^(x - m), fp32 into the row sum, f16 (below
                // 2^-14 off by up to 2^-25, of a sum that is at least 1) over
                // columns of S that have been read (16 of P for 32 of S).
                const float mu = m == -INFINITY ? 0.f : m;
                const float2 f2 = make_float2(GEN ? 1.f : fac, GEN ? 1.f : fac), nm2 = make_float2(-mu, -mu);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int c = 0; c < kBN; c += kCols) {
                    uint32_t x[kCols / 32][32];
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h) tc::ld32(s_col + c + h * 32, x[h]);
                    tc::wait_ld();
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 pr = exp2_pair_f32(
                                ffma2(make_float2(__uint_as_float(x[h][e]), __uint_as_float(x[h][e + 1])), f2, nm2));
                            sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], pr);
                            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[e / 2]) : "f"(pr.y), "f"(pr.x));
                        }
                        tc::st16(s_col + c / 2 + h * 16, pk);
                    }
                }
                const float2 both = fadd2(sum[0], sum[1]);
                l = l * alpha + (both.x + both.y);
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
        if (ok) ok = wwait(v_full0 + 8 * ((n - 1) % C::kStages), ((n - 1) / C::kStages) & 1);   // nan_flag
        if (ok && live) {
            // Dims that are NaN at keys this row sees and others of the tile do not.
            uint32_t nans = 0;
            if (valid && *nan_flag) {
                const int beg = max(lo, t_begin * kBN), end = min(hi + 1, (t_begin + n) * kBN);
                nans = nan_groups(p, s, hkv, beg, min(end, full_lo)) | nan_groups(p, s, hkv, max(beg, full_hi + 1), end);
            }
            // tcgen05.ld is warp-collective: every lane of a live warp loads.
            tc::fence_after_sync();
            float f = p.v_scale;
            if (split) {
                if (valid) {
                    p.part_ml[(row * p.splits + seg) * 2 + 0] = stored_max(m, l);
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
                for (int e = 0; e < 32; ++e)
                    o[e] = nans >> (2 * c + e / 16) & 1 ? 0x7fffffffu : __float_as_uint(__uint_as_float(o[e]) * f);
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
    if (warp == kWarpQk) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t launch_rows_d(const Fp4RowsPlan& plan, const FwdParams& p, cudaStream_t stream) {
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI | UA_FLAG_QQ_BIAS)) != 0;
    auto kern = gen ? fp4_rows_kernel<D, true> : fp4_rows_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(plan.tiles * plan.splits), (unsigned)p.hk, (unsigned)p.num_seqs);
    kern<<<grid, kThreadsR, RCfg<D>::kSmem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool plan_fp4_rows(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4RowsPlan* plan) {
    *plan = Fp4RowsPlan();
    if (p.g > kRows || p.max_seqlen_k > 1 << 30 || (int64_t)p.g * p.max_seqlen_q < kFp4RowsMin) return false;
    const int ppt = kRows / p.g;
    const int64_t tiles = (p.max_seqlen_q + ppt - 1) / ppt;
    // Segments.  A CTA (one per SM) costs its key tiles plus about ten tiles' time
    // to start and finish, a segment about one more in the join.  The host knows
    // the longest sequence only, so the number taken is the one whose time is
    // least over two batches: all that long (whole waves of CTAs), and lengths
    // spread evenly below it (half the CTAs of every further segment leave at
    // once; beyond one wave the work is shared out, with a tail).  Measured, key
    // weights included, 8 KV heads, 128 rows (us at 2 / 3 / 4 / 6 / 8 segments): 8
    // sequences of 12000 keys 148 / 179 / 161 / 171 / 179, of 1000 to 12000 120 /
    // 105 / 118 / 113 / 118; 4 of 12000 120 / 105 / 95 / 116 / 108, of 1000 to 12000
    // 108 / 93 / 83 / 97 / 91.  (All at d = 128: at d = 256, where a tile is 64 keys,
    // the count is as if two tiles were one.  A window is not looked at: segments
    // that hold none of its keys leave at once, the others share it.)
    const int64_t base = (int64_t)p.hk * p.num_seqs * tiles;
    const int64_t key_tiles = (p.max_seqlen_k + 127) / 128;
    int64_t splits = 1;
    double best = 0.;
    for (int64_t s = 1; s <= std::min<int64_t>(64, std::max<int64_t>(1, key_tiles / 4)); ++s) {
        const double each = 10. + (double)((key_tiles + s - 1) / s), live = (double)base * (s + 1) / 2.;
        const double work = (double)base * ((double)key_tiles + 10. * (s + 1)) / (2. * num_sms);
        const double cost = (double)((base * s + num_sms - 1) / num_sms) * each +
                            (live <= num_sms ? each : std::max(each, work + 0.6 * each)) + (double)s;
        if (s == 1 || cost < best) {
            best = cost;
            splits = s;
        }
    }
    const size_t per_split = fp4_workspace_bytes(p.total_q * p.hq, p.d);
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, (int64_t)(workspace_bytes / per_split)));
    const int64_t per = (p.max_seqlen_k + splits - 1) / splits;
    plan->chunk = (int)std::min<int64_t>((per + 127) / 128 * 128, 1 << 30);
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
