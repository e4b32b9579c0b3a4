// ua_fp4_rows.cu -- attention over a 4-bit cache for calls with many packed rows
// per KV head (prompt chunks, observation windows), and of draft trees over 4-bit and
// fp8 caches, on tcgen05.
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
// Draft trees (TREE) differ in what a row sees: chunk keys by its row of the mask, the
// window and ALiBi by the nodes' positions; every tile that reaches past the context is
// looked at key by key.  64 requests of 16 to 32 nodes, 512 to 8192 keys, 32 / 8 heads,
// d = 128: 288 us (causal chunks the same); one of 8 nodes, 999 keys, 8 / 2 heads, d = 64: 14.
//
// An fp8 cache (F8, trees at d = 128) comes through the tensor maps of its pages, rows of
// 128 bytes swizzled; its codes are exact in f16 too, and NaN stands in single values. The
// same 64 requests 274 us; expanding the cache to bf16 pages first would move 1.8 GB more.
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
#include "ua_tree_mask.cuh"

namespace ua {
namespace {

using namespace pf;

constexpr int kThreadsR = 480;
constexpr int kWarpQk = 12;        // also owns tensor memory
constexpr int kWarpCopy = 13;
constexpr int kCols = 64;          // columns of S a softmax thread holds at a time

// F8: an e4m3 cache, whose tiles are twice the bytes.
template <int D, bool F8>
struct RCfg {
    static constexpr int kBN = D == 256 ? 64 : 128;     // keys per tile
    static constexpr int kStages = D == 256 ? 1 : 2;    // f16 K and V tiles
    static constexpr int kRing = F8 ? 2 : D == 64 ? 4 : 3;    // K and V tiles as they are cached
    static constexpr int kPanels = D / 64;
    static constexpr int kQPanel = kRows * 128;         // 128 rows x 64 dims, f16
    static constexpr int kPanel = kBN * 128;            // kBN keys x 64 dims, f16
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kRaw = F8 ? kBN * D : kBN * (D / 2 + D / 16);    // (4 bits: codes, then scales)
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
    static constexpr int kChunks = D / (F8 ? 16 : 32);  // 16-byte runs of codes per key
    static constexpr int kEach = kBN * kChunks / 128;   // of them per converter thread and tile
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(kRaw % 16 == 0, "bulk copy alignment");
    static_assert(!F8 || (D == 128 && kOffRawK % 1024 == 0), "swizzled rows of 128 bytes");
};

// A row's mask and what seen_keys wants beside it; mask = null: a row that sees all keys asked for.
struct TreeRow {
    const uint32_t* mask;
    int64_t q0;
    int ctx, sq, sk, lo;
    __device__ __forceinline__ bool sees(const FwdParams& p, int key) const {
        return !mask || (seen_keys(p, mask, q0, key, ctx, sq, sk, lo) & 1u) != 0;
    }
};

// The dims (one bit per 16) that are NaN in V at those of the keys [lo, hi) of sequence s
// that the row sees.
__device__ __noinline__ uint32_t nan_groups(const FwdParams& p, int s, int hkv, int lo, int hi, TreeRow row) {
    const int scale_row = p.d / 16, b_log2 = 31 - __clz(p.b);
    const int64_t page_bytes = fp4_page_bytes(p.b, p.d);
    uint32_t found = 0;
    for (int key = lo; key < hi; ++key) {
        if (!row.sees(p, key)) continue;
        const int32_t id = __ldg(p.block_table + (int64_t)s * p.bt_stride + (key >> b_log2));
        if (id < 0 || (int64_t)id >= p.num_blocks) continue;       // reads as zeros
        const uint8_t* sc = static_cast<const uint8_t*>(p.v_cache) + ((int64_t)id * p.hk + hkv) * page_bytes +
                            p.b * (p.d / 2) + (key & (p.b - 1)) * scale_row;
        for (int e = 0; e < scale_row; ++e)
            if ((sc[e] & 0x7f) == 0x7f) found |= 1u << e;
    }
    return found;
}

// The dims 32 c .. 32 c + 31 that are NaN in an e4m3 cache's V at those keys.
__device__ __noinline__ uint32_t nan_dims(const FwdParams& p, int s, int hkv, int lo, int hi, int c, TreeRow row) {
    const int b_log2 = 31 - __clz(p.b);
    uint32_t found = 0;
    for (int key = lo; key < hi; ++key) {
        if (!row.sees(p, key)) continue;
        const int32_t id = __ldg(p.block_table + (int64_t)s * p.bt_stride + (key >> b_log2));
        if (id < 0 || (int64_t)id >= p.num_blocks) continue;       // reads as zeros
        const uint8_t* v = static_cast<const uint8_t*>(p.v_cache) +
                           (((int64_t)id * p.b + (key & (p.b - 1))) * p.hk + hkv) * p.d + 32 * c;
        for (int e = 0; e < 32; ++e)
            if ((v[e] & 0x7f) == 0x7f) found |= 1u << e;
    }
    return found;
}

template <int D, bool GEN, bool TREE, bool F8>
__device__ __forceinline__ void rows_body(const FwdParams& p, const CUtensorMap* tm_k, const CUtensorMap* tm_v) {
    using C = RCfg<D, F8>;
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
    const int vis_beg = window ? max(0, (TREE ? 0 : first) + ctx - p.window + 1) : 0;
    const int vis_end = causal && !TREE ? min(sk, last + ctx + 1) : sk;
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
    const int full_lo = window ? max(0, (TREE ? sq - 1 : last) + ctx - p.window + 1) : 0;
    const int full_hi = TREE ? ctx - 1 : causal ? min(first + ctx, sk - 1) : sk - 1;

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
                if (j >= n || page >= pages || blk >= nblk) return -2;
                const int32_t id = __ldg(bt + blk);
                return F8 && id == -2 ? -1 : id;
            };
            int32_t id_next = id_of(0);
            int issued = 0;
            for (int j = 0; j < n; ++j) {
                const int slot = j % C::kRing;
                const int32_t id = id_next;
                id_next = id_of(j + 1);
                if (j >= C::kRing && !wwait(empty0 + 8 * slot, ((j / C::kRing) + 1) & 1)) break;
                if constexpr (F8) {
                    // Boxes of a block's slots, 128 bytes each; a bad block's are filled with zeros.
                    const bool there = id != -2;
                    const unsigned boxes = __ballot_sync(0xffffffffu, there);
                    if (there && (id < 0 || (int64_t)id >= p.num_blocks)) atomicOr(p.err, (int)UA_DEVERR_BLOCK_ID);
                    if (lane < 2)
                        mbar_arrive_expect_tx(full0 + 8 * slot,
                                              (uint32_t)__popc(boxes & (op ? 0xaaaaaaaau : 0x55555555u)) * p.b * 128);
                    __syncwarp();
                    if (there)
                        tma_load_4d(smem_u32(ring + slot * C::kRaw + page * p.b * 128), op ? tm_v : tm_k, 0, hkv, 0, id,
                                    full0 + 8 * slot);
                    issued = j + 1;
                    continue;
                }
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
            if constexpr (F8) {
#pragma unroll 2
                for (int i = 0; i < C::kEach; ++i) {
                    const int k = k0 + i * (128 / C::kChunks), key = key0 + k;
                    const uint4 c = *reinterpret_cast<const uint4*>(raw + k * 128 + ((chunk ^ (k & 7)) << 4));
                    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[2 * e] = e4m3x2_to_f16(w[e] & 0xffffu);
                        h[2 * e + 1] = e4m3x2_to_f16(w[e] >> 16);
                    }
                    if (edge && (key < full_lo || key > full_hi)) {
                        if (key < vis_beg || key >= vis_end) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] = 0;
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t x = h[e];
                                if ((x & 0x7c00u) == 0x7c00u) h[e] &= 0xffff0000u;
                                if ((x & 0x7c000000u) == 0x7c000000u) h[e] &= 0xffffu;
                                if (h[e] != x) *nan_flag = 1;
                            }
                        }
                    }
                    uint8_t* row = tiles_mem + stg * C::kTile + (chunk >> 2) * C::kPanel + k * 128;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<uint4*>(row + ((((chunk & 3) * 2 + e) ^ (k & 7)) << 4)) =
                            make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
                }
            }
#pragma unroll 2
            for (int i = 0; i < (F8 ? 0 : C::kEach); ++i) {
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
        int lo = window ? max(0, pos + ctx - p.window + 1) : 0;
        const uint32_t* mask = TREE ? p.tree_mask + (q0 + min(pos, last)) * p.mask_stride : nullptr;
        if (TREE && (p.flags & (UA_FLAG_WINDOW | UA_FLAG_ALIBI)) && valid) {
            const int at = p.positions[q0 + pos];
            if (at < ctx || at >= sk) atomicOr(p.err, (int)UA_DEVERR_TREE);
            if (window) lo = max(0, node_position(p, q0, pos, ctx, sk) - p.window + 1);
        }
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
                        uint32_t see = 0xffffffffu;
                        if (TREE && edge) see = seen_keys(p, mask, q0, key, ctx, sq, sk, lo);
                        if constexpr (GEN) {
                            int at = key + lane;              // position of the lane's key
                            if (TREE && alibi && at >= ctx && at < sk) at = node_position(p, q0, at - ctx, ctx, sk);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float v = __uint_as_float(x[h][e]) * fac;
                                if (softcap) v = cap * tanh_from_exp2(v);
                                if (alibi) v += slope * (float)((TREE ? __shfl_sync(0xffffffffu, at, e) : key + e) - ctx);
                                if (qq && valid && key + e >= ctx && key + e <= hi)
                                    v += __ldg(p.qq_bias + (int64_t)pos * p.qq_stride + (key + e - ctx)) * kLog2e;
                                x[h][e] = __float_as_uint(v);
                            }
                        }
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (TREE ? !(see >> e & 1u) : key + e < lo || key + e > hi)
                                    x[h][e] = __float_as_uint(-INFINITY);
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
            const bool look = valid && *nan_flag;
            const int beg = max(TREE ? vis_beg : lo, t_begin * kBN), end = min(TREE ? sk : hi + 1, (t_begin + n) * kBN);
            const TreeRow sees{mask, q0, ctx, sq, sk, lo};
            if (!F8 && look) {
                nans = nan_groups(p, s, hkv, beg, min(end, full_lo), sees) |
                       nan_groups(p, s, hkv, max(beg, max(full_lo, full_hi + 1)), end, sees);
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
                if (F8 && look)
                    nans = nan_dims(p, s, hkv, beg, min(end, full_lo), c, sees) |
                           nan_dims(p, s, hkv, max(beg, max(full_lo, full_hi + 1)), end, c, sees);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = nans >> (F8 ? e : 2 * c + e / 16) & 1 ? 0x7fffffffu : __float_as_uint(__uint_as_float(o[e]) * f);
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

template <int D, bool GEN, bool TREE>
__global__ void __launch_bounds__(kThreadsR, 1) fp4_rows_kernel(const FwdParams p) {
    rows_body<D, GEN, TREE, false>(p, nullptr, nullptr);
}

template <bool GEN>
__global__ void __launch_bounds__(kThreadsR, 1)
fp8_tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
    rows_body<128, GEN, true, true>(p, &tm_k, &tm_v);
}

template <int D>
cudaError_t launch_rows_d(const Fp4RowsPlan& plan, const FwdParams& p, cudaStream_t stream) {
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI | UA_FLAG_QQ_BIAS)) != 0;
    auto kern = p.tree_mask ? (gen ? fp4_rows_kernel<D, true, true> : fp4_rows_kernel<D, false, true>)
                            : (gen ? fp4_rows_kernel<D, true, false> : fp4_rows_kernel<D, false, false>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RCfg<D, false>::kSmem);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(plan.tiles * plan.splits), (unsigned)p.hk, (unsigned)p.num_seqs);
    kern<<<grid, kThreadsR, RCfg<D, false>::kSmem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool plan_fp4_rows(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4RowsPlan* plan) {
    *plan = Fp4RowsPlan();
    if (p.g > kRows || p.max_seqlen_k > 1 << 30 || (!p.tree_mask && (int64_t)p.g * p.max_seqlen_q < kFp4RowsMin))
        return false;
    const int ppt = kRows / p.g;
    // (One tile at least: it reports sequences of more rows than a call allows, also one of none.)
    const int64_t tiles = std::max(1, (p.max_seqlen_q + ppt - 1) / ppt);
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

cudaError_t launch_fp8_tree(const Fp4RowsPlan& plan, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const FwdParams& p,
                            cudaStream_t stream) {
    if (p.d != 128) return cudaErrorInvalidValue;
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI)) != 0;
    auto kern = gen ? fp8_tree_kernel<true> : fp8_tree_kernel<false>;
    constexpr int smem = RCfg<128, true>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(plan.tiles * plan.splits), (unsigned)p.hk, (unsigned)p.num_seqs);
    kern<<<grid, kThreadsR, smem, stream>>>(tm_k, tm_v, p);
    return cudaGetLastError();
}

}  // namespace ua
