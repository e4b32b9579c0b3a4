// ua_tree.cu -- attention for trees of drafted tokens over a bf16 paged cache, on tcgen05.
//
// A chunk's token sees every key of its context and, of the chunk's own keys, those
// whose bit its row of the mask has (its ancestors and itself).  With g query heads per
// KV head and S_q nodes a KV head has g S_q rows, a few up to some hundreds: every
// cached value is used that often, which is less than the tensor cores could do per
// byte of HBM (about 277 rows), so a batch of trees is bound by reading K and V once.
//
// One CTA per (row tile of floor(128 / g) nodes, KV segment, KV head, sequence), the
// row tiles of a segment next to each other (they read the same K and V, from L2 after
// the first).  S = Q K^T and O += P V are tcgen05.mma with M = 128 rows; P goes over
// its own S in tensor memory.  At d = 64 and 128 a CTA keeps one S tile (256 columns of
// tensor memory with O) and few K/V stages, so that two CTAs share an SM: while one
// waits for its copies or for its softmax, the other one's copies are in flight.  At
// d = 256 Q and the tiles (64 keys) fill an SM's shared memory, and one CTA overlaps
// its own softmax and MMAs over two S tiles.
//
// Roles (7 warps):
//   warps 0-3  softmax and epilogue: thread r owns row r (tensor-memory lane r); two
//              passes over the tile's columns (maximum, then P), 64 at a time;
//   warp 4     copies (TMA): Q, then the K and V tiles, one lane per paged block;
//   warp 5     MMA issuer and owner of tensor memory;
//   warp 6     looks through V tiles with keys that some row does not see.
//
// Masked keys: their scores are replaced, whatever K holds.  Their V rows reach the
// product with P = 0, and 0 times an infinity or NaN is NaN; so warp 6 clears values
// that are not finite in such tiles, and the epilogue adds them again to the rows that
// see their key (a flag, no cost while all values are finite).
#include <algorithm>
#include <cstdint>

#include "ua_common.cuh"
#include "ua_prefill_common.cuh"
#include "ua_ptx.cuh"
#include "ua_tc.cuh"
#include "ua_tmap.h"
#include "ua_tree.h"

namespace ua {
namespace {

using namespace pf;

constexpr int kThreadsT = 224;
constexpr int kWarpCopy = 4;
constexpr int kWarpMmaT = 5;
constexpr int kWarpFix = 6;
constexpr int kCols = 64;          // columns of S a softmax thread holds at a time

template <int D>
struct TCfg {
    static constexpr int kBN = D == 256 ? 64 : 128;     // keys per tile
    static constexpr int kStages = D == 128 ? 1 : 2;    // K and V tiles each
    static constexpr int kBufs = D == 256 ? 2 : 1;      // S tiles
    static constexpr int kCtas = D == 256 ? 1 : 2;      // per SM
    static constexpr int kPanels = D / 64;
    static constexpr int kQPanel = kRows * 128;         // 128 rows x 64 dims
    static constexpr int kPanel = kBN * 128;            // kBN keys x 64 dims
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kPanels * kQPanel;
    static constexpr int kOffV = kOffK + kStages * kTile;
    static constexpr int kOffBar = kOffV + kStages * kTile;
    // q_full, {k_full, k_empty, v_full, v_ready, v_empty}[kStages], s_full[2],
    // p_full[2], o_done[2], drain, never
    static constexpr int kNumBars = 1 + 5 * kStages + 8;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmem = kOffMisc + 16 + 1024;
    static constexpr int kTmemO = kBufs * kBN;
    static constexpr uint32_t kCols2 = D == 256 ? 512 : 256;    // tensor-memory columns
    static_assert(kTmemO + D <= (int)kCols2, "tensor memory budget");
    static_assert(kCtas * (kSmem + 1024) <= 233472, "shared memory budget");
};

// The position of the chunk's key c, within the range that a tree can have.
__device__ __forceinline__ int node_position(const FwdParams& p, int64_t q0, int c, int ctx, int sk) {
    return min(max(__ldg(p.positions + q0 + c), ctx), sk - 1);
}

// Which of the 32 keys from kb on a row sees (bit e: key kb + e).  lo: the first
// position inside the row's window.
__device__ __forceinline__ uint32_t seen_keys(const FwdParams& p, const uint32_t* row, int64_t q0, int kb, int ctx, int sq,
                                              int sk, int lo) {
    const int c0 = kb - ctx;
    if (c0 >= sq) return 0u;
    uint32_t bits = 0xffffffffu;
    if (c0 > -32) {
        const int w = c0 >> 5;             // -1: the words in front of the chunk are all ones
        const uint32_t a = w < 0 ? 0xffffffffu : __ldg(row + w);
        const uint32_t b = w + 1 < p.mask_stride ? __ldg(row + w + 1) : 0u;
        bits = __funnelshift_r(a, b, c0 & 31);
        if (sq - c0 < 32) bits &= (1u << (sq - c0)) - 1u;
    }
    const int low = min(lo, ctx) - kb;     // context keys in front of the window
    if (low > 0) bits &= low >= 32 ? 0u : 0xffffffffu << low;
    if (lo > ctx)                          // a window shorter than the branch
        for (int e = max(0, -c0); e < 32; ++e)
            if ((bits >> e & 1u) && node_position(p, q0, c0 + e, ctx, sk) < lo) bits &= ~(1u << e);
    return bits;
}

// Values that are not finite among a row's visible V of keys [beg, end): the sum of
// them (0 if there are none) for 32 dims from c on is added to o.
__device__ __noinline__ void add_unbounded(const FwdParams& p, int s, int hkv, int64_t q0, const uint32_t* row, int beg, int end,
                                           int ctx, int sq, int sk, int lo, int c, uint32_t (&o)[32]) {
    const int b_log2 = 31 - __clz(p.b);
    for (int key = beg; key < end; ++key) {
        if (!(seen_keys(p, row, q0, key, ctx, sq, sk, lo) & 1u)) continue;
        const int32_t id = __ldg(p.block_table + (int64_t)s * p.bt_stride + (key >> b_log2));
        if (id < 0 || (int64_t)id >= p.num_blocks) continue;        // read as zeros
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v_cache) +
                                 (((int64_t)id * p.b + (key & (p.b - 1))) * p.hk + hkv) * p.d + c;
        for (int e = 0; e < 32; ++e) {
            const float x = __bfloat162float(v[e]);
            if (!(fabsf(x) <= 3.4e38f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
        }
    }
}

template <int D, bool GEN>
__global__ void __launch_bounds__(kThreadsT, TCfg<D>::kCtas)
tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const FwdParams p, int tiles) {
    using C = TCfg<D>;
    constexpr int kBN = C::kBN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int s = blockIdx.z;
    const int hkv = blockIdx.y;
    const int tile = blockIdx.x % tiles;
    const int seg = blockIdx.x / tiles;
    const bool split = p.splits > 1;
    const int g = p.g;
    const int ppt = kRows / g;                   // nodes per tile
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
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;
    // Positions of the chunk lie in [ctx, sk): keys in front of ctx - W + 1 are seen by
    // no row, those from sk - W on by every row, up to the chunk.
    const int vis_beg = window ? max(0, ctx - p.window + 1) : 0;
    int k_beg = vis_beg, k_end = sk;
    if (split) {
        k_beg = max(k_beg, seg * p.chunk);
        k_end = (int)min((int64_t)k_end, (int64_t)seg * p.chunk + p.chunk);
    }
    if (st || k_beg >= k_end) {
        // Malformed lengths (rows written as zeros) or a segment no row sees.
        for (int e = threadIdx.x; e < kRows * (D / 8); e += kThreadsT) {
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
    const int full_lo = window ? max(0, sk - p.window) : 0;     // [full_lo, ctx): seen by every row

    uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    constexpr int kS = 8 * C::kStages;
    const uint32_t q_full = smem_u32(bar_mem);
    const uint32_t k_full0 = q_full + 8, k_empty0 = k_full0 + kS;
    const uint32_t v_full0 = k_empty0 + kS, v_ready0 = v_full0 + kS, v_empty0 = v_ready0 + kS;
    const uint32_t s_full0 = v_empty0 + kS, p_full0 = s_full0 + 16, o_done0 = s_full0 + 32;
    const uint32_t drain = s_full0 + 48, never = s_full0 + 56;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    volatile int* odd_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(k_full0 + 8 * i, 1);
            mbar_init(k_empty0 + 8 * i, 1);
            mbar_init(v_full0 + 8 * i, 1);
            mbar_init(v_ready0 + 8 * i, 1);
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
        *odd_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMmaT) {
        tc::tmem_alloc(smem_u32(tmem_slot), C::kCols2);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sQ = smem_u32(smem + C::kOffQ);
    const uint32_t sK = smem_u32(smem + C::kOffK);
    const uint32_t sV = smem_u32(smem + C::kOffV);
    auto wwait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, p.err));
    };
    // Tiles with a key that some row does not see.
    auto edge_tile = [&](int key0) { return key0 < full_lo || key0 + kBN > ctx; };

    if (warp == kWarpCopy) {
        // --------------------------------- copies ---------------------------------
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            mbar_arrive_expect_tx(q_full, (uint32_t)(g * ppt) * 128u * C::kPanels);
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn)
                tma_load_3d(sQ + pn * C::kQPanel, &tm_q, pn * 64, hkv * g, (int)q0 + first, q_full);
        }
        __syncwarp();
        const int b = p.b;
        const int nblk_seq = (sk + b - 1) / b;
        const int32_t* bt = p.block_table + (int64_t)s * p.bt_stride;
        auto tile_id = [&](int j) -> int32_t {
            const int blk0 = (t_begin + j) * kBN / b;
            return lane < min(kBN / b, nblk_seq - blk0) ? __ldg(bt + blk0 + lane) : 0;
        };
        int32_t id_next = tile_id(0);
        int k_out = 0, v_out = 0;      // tiles whose copies were issued
        for (int j = 0; j < n; ++j) {
            const int stg = j % C::kStages;
            const int blk0 = (t_begin + j) * kBN / b;
            const int nb = min(kBN / b, nblk_seq - blk0);
            const uint32_t bytes = (uint32_t)nb * b * 128 * C::kPanels;
            const int32_t id = id_next;
            if (j + 1 < n) id_next = tile_id(j + 1);
            if (lane < nb && (id < 0 || (int64_t)id >= p.num_blocks)) atomicOr(p.err, (int)UA_DEVERR_BLOCK_ID);
            if (j >= C::kStages && !wwait(k_empty0 + 8 * stg, ((j / C::kStages) + 1) & 1)) break;
            if (lane == 0) mbar_arrive_expect_tx(k_full0 + 8 * stg, bytes);
            __syncwarp();
            if (lane < nb) {
#pragma unroll
                for (int pn = 0; pn < C::kPanels; ++pn)
                    tma_load_4d(sK + stg * C::kTile + pn * C::kPanel + lane * b * 128, &tm_k, pn * 64, hkv, 0, id,
                                k_full0 + 8 * stg);
            }
            k_out = j + 1;
            if (j >= C::kStages && !wwait(v_empty0 + 8 * stg, ((j / C::kStages) + 1) & 1)) break;
            if (lane == 0) mbar_arrive_expect_tx(v_full0 + 8 * stg, bytes);
            __syncwarp();
            if (lane < nb) {
#pragma unroll
                for (int pn = 0; pn < C::kPanels; ++pn)
                    tma_load_4d(sV + stg * C::kTile + pn * C::kPanel + lane * b * 128, &tm_v, pn * 64, hkv, 0, id,
                                v_full0 + 8 * stg);
            }
            v_out = j + 1;
        }
        if (*abort_flag && lane == 0) {
            // Let every copy this warp issued land before the CTA ends.
            mbar_wait_bounded(q_full, 0);
            for (int j = max(0, k_out - C::kStages); j < k_out; ++j)
                mbar_wait_bounded(k_full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
            for (int j = max(0, v_out - C::kStages); j < v_out; ++j)
                mbar_wait_bounded(v_full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == kWarpMmaT) {
        // ------------------------- MMA issuer (one thread) -------------------------
        // MMAs of one thread run in issue order, so the Q K^T that goes over columns
        // holding P cannot overtake the P V that reads them.
        constexpr int kNV = D == 64 ? 64 : 128;       // dims per P V MMA
        constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kRows, kBN, false, false);
        constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kRows, kNV, false, true);
        const uint64_t qd = tc::smem_desc_sw128(sQ, 16, 1024);
        const uint64_t kd = tc::smem_desc_sw128(sK, 16, 1024);
        const uint64_t vd = tc::smem_desc_sw128(sV, C::kPanel, 1024);
        auto issue_qk = [&](int j) -> bool {
            const int stg = j % C::kStages, buf = j % C::kBufs;
            // Testing hook: the first K wait waits on a barrier that nothing
            // completes and gives up after stall_ns.
            if (p.stall && j == 0 &&
                !__all_sync(0xffffffffu, wait_or_abort(never, 0, abort_flag, p.err, (uint64_t)p.stall_ns)))
                return false;
            if (!wwait(k_full0 + 8 * stg, (j / C::kStages) & 1)) return false;
            tc::fence_after_sync();
            if (lane == 0) {
                const uint64_t kst = kd + (uint64_t)(stg * (C::kTile >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_bf16(tmem + buf * kBN, qd + (k >> 2) * (C::kQPanel >> 4) + (k & 3) * 2,
                                 kst + (k >> 2) * (C::kPanel >> 4) + (k & 3) * 2, idesc_qk, k > 0 ? 1u : 0u);
                tc::commit(s_full0 + 8 * buf);
                tc::commit(k_empty0 + 8 * stg);
            }
            __syncwarp();
            return true;
        };
        bool ok = wwait(q_full, 0) && issue_qk(0);
        for (int j = 0; ok && j < n; ++j) {
            const int stg = j % C::kStages, buf = j % C::kBufs;
            // With two S tiles the next one is filled while the softmax has this one.
            if (C::kBufs == 2 && j + 1 < n && !(ok = issue_qk(j + 1))) break;
            if (!(ok = wwait(v_ready0 + 8 * stg, (j / C::kStages) & 1))) break;
            if (!(ok = wwait(p_full0 + 8 * buf, (j / C::kBufs) & 1))) break;
            tc::fence_after_sync();
            if (lane == 0) {
                const uint64_t vst = vd + (uint64_t)(stg * (C::kTile >> 4));
#pragma unroll
                for (int k = 0; k < kBN / 16; ++k)
#pragma unroll
                    for (int h = 0; h < D / kNV; ++h)
                        // A = P from tensor memory (16 keys = 8 columns), B = V
                        // MN-major, two 64-dim panels.
                        tc::mma_bf16_ts(tmem + C::kTmemO + h * kNV, tmem + buf * kBN + k * 8,
                                        vst + h * 2 * (C::kPanel >> 4) + k * 128, idesc_pv, (j > 0 || k > 0) ? 1u : 0u);
                tc::commit(o_done0 + 8 * buf);
                tc::commit(v_empty0 + 8 * stg);
            }
            __syncwarp();
            if (C::kBufs == 1 && j + 1 < n) ok = issue_qk(j + 1);
        }
        if (*abort_flag) {
            // No MMA of this thread may still run when tensor memory is freed.
            if (lane == 0) tc::commit(drain);
            __syncwarp();
            mbar_wait_bounded(drain, 0);
        }
    } else if (warp == kWarpFix) {
        // ------------------- V values that some rows must not see -------------------
        for (int j = 0; j < n; ++j) {
            const int stg = j % C::kStages, key0 = (t_begin + j) * kBN;
            if (!wwait(v_full0 + 8 * stg, (j / C::kStages) & 1)) break;
            if (edge_tile(key0)) {
                uint8_t* v = smem + C::kOffV + stg * C::kTile;
                bool odd = false;
                auto clear = [&](int k_lo, int k_hi) {         // keys of the tile
                    const int words = (k_hi - k_lo) * 8;       // 16 bytes each, per panel
                    for (int pn = 0; pn < C::kPanels; ++pn)
                        for (int e = lane; e < words; e += 32) {
                            uint4* at = reinterpret_cast<uint4*>(v + pn * C::kPanel + k_lo * 128) + e;
                            uint4 x = *at;
                            uint32_t* w = &x.x;
                            bool hit = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((w[i] & 0x7f80u) == 0x7f80u) {
                                    w[i] &= 0xffff0000u;
                                    hit = true;
                                }
                                if ((w[i] & 0x7f800000u) == 0x7f800000u) {
                                    w[i] &= 0xffffu;
                                    hit = true;
                                }
                            }
                            if (hit) *at = x;
                            odd |= hit;
                        }
                };
                const int part = min(max(full_lo - key0, 0), kBN);
                clear(0, part);
                clear(max(part, min(max(ctx - key0, 0), kBN)), kBN);
                if (odd) *odd_flag = 1;
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(v_ready0 + 8 * stg);
            __syncwarp();
        }
    } else {
        // ------------------------------ softmax, epilogue ------------------------------
        const int r = threadIdx.x;
        const int i = first + r / g;
        const bool valid = r < g * ppt && i <= last;
        const int head = hkv * g + r % g;
        const bool live = __any_sync(0xffffffffu, valid);   // else the warp only keeps the barriers going
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const bool softcap = GEN && (p.flags & UA_FLAG_SOFTCAP) != 0;
        const bool alibi = GEN && (p.flags & UA_FLAG_ALIBI) != 0;
        const float slope = alibi && valid ? __ldg(p.alibi + head) * kLog2e : 0.f;
        const uint32_t* mask = p.tree_mask + (q0 + min(i, last)) * p.mask_stride;
        int lo = 0;
        if (window && valid) {
            const int at = __ldg(p.positions + q0 + i);
            if (at < ctx || at >= sk) atomicOr(p.err, (int)UA_DEVERR_TREE);
            lo = max(0, node_position(p, q0, i, ctx, sk) - p.window + 1);
        }
        const int64_t row = (q0 + i) * p.hq + head;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        // The score chain is in log2 units from the products on (a factor of zero
        // would make NaN of masked scores).
        const float cap = p.softcap * kLog2e, fac = fmaxf(p.scale * (softcap ? 1.f / p.softcap : kLog2e), 0x1p-126f);
        for (int j = 0; j < n; ++j) {
            const int buf = j % C::kBufs;
            if (!(ok = wwait(s_full0 + 8 * buf, (j / C::kBufs) & 1))) break;
            const int key0 = (t_begin + j) * kBN;
            const uint32_t s_col = trow + buf * kBN;
            const bool edge = edge_tile(key0);
            bool reanchor = false;
            float alpha = 1.f;
            if (live) {
                tc::fence_after_sync();
                // First pass: the maximum.  Plain scores stay as the MMA left them; a
                // general score chain or a mask is applied here and written back.
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
                            const bool nodes = alibi && key + 32 > ctx;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float v = __uint_as_float(x[h][e]) * fac;
                                if (softcap) v = cap * tanh_from_exp2(v);
                                if (alibi) {
                                    int at = key + e;
                                    if (nodes && at >= ctx && at < sk) at = node_position(p, q0, at - ctx, ctx, sk);
                                    v += slope * (float)(at - ctx);
                                }
                                x[h][e] = __float_as_uint(v);
                            }
                        }
                        if (edge) {
                            const uint32_t see = seen_keys(p, mask, q0, key, ctx, sq, sk, lo);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see >> e & 1u)) x[h][e] = __float_as_uint(-INFINITY);
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
                // Second pass: P = 2^(x - m), fp32 into the row sum, bf16 (V's type, as
                // the MMA wants; 2^-8 off each) over columns of S that have been read.
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
                            pk[e / 2] = pack_bf16x2(pr.x, pr.y);
                        }
                        tc::st16(s_col + c / 2 + h * 16, pk);
                    }
                }
                const float2 both = fadd2(sum[0], sum[1]);
                l = l * alpha + (both.x + both.y);
                tc::wait_st();
            }
            if (live && j > 0 && __any_sync(0xffffffffu, reanchor)) {
                // O holds the P V of the tiles up to j - 1.  With one S tile that product
                // was issued in front of this tile's Q K^T, which is complete.
                if (C::kBufs == 2 && !(ok = wwait(o_done0 + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1))) break;
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
            mbar_arrive(p_full0 + 8 * buf);
        }
        if (ok) ok = wwait(o_done0 + 8 * ((n - 1) % C::kBufs), ((n - 1) / C::kBufs) & 1);
        if (ok && live) {
            // tcgen05.ld is warp-collective: every lane of a live warp loads.
            tc::fence_after_sync();
            const bool odd = *odd_flag != 0;
            float f = 1.f;
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
                        f = m == -INFINITY ? 0.f : fast_exp2(m - s2);
                        L = L * f + 1.0f;
                    } else if (s2 != -INFINITY) {
                        L += fast_exp2(s2 - m);
                    }
                }
                f = L > 0.f || L != L ? f * __frcp_rn(L) : 0.f;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tc::ld32(trow + C::kTmemO + c * 32, o);
                tc::wait_ld();
                if (!valid) continue;
                if (odd) {
                    const int beg = t_begin * kBN, end = min((t_begin + n) * kBN, sk);
                    add_unbounded(p, s, hkv, q0, mask, beg, min(end, full_lo), ctx, sq, sk, lo, c * 32, o);
                    add_unbounded(p, s, hkv, q0, mask, max(beg, max(full_lo, ctx)), end, ctx, sq, sk, lo, c * 32, o);
                }
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
    if (warp == kWarpMmaT) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::kCols2);
    }
}

template <int D>
cudaError_t launch_tree_d(const TreePlan& plan, const CUtensorMap& tq, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                          const FwdParams& p, cudaStream_t stream) {
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI)) != 0;
    auto kern = gen ? tree_kernel<D, true> : tree_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(plan.tiles * plan.splits), (unsigned)p.hk, (unsigned)p.num_seqs);
    kern<<<grid, kThreadsT, TCfg<D>::kSmem, stream>>>(tq, tm_k, tm_v, p, plan.tiles);
    return cudaGetLastError();
}

}  // namespace

bool plan_tree(const FwdParams& p, int num_sms, size_t workspace_bytes, TreePlan* plan) {
    *plan = TreePlan();
    if (p.g > kRows || p.max_seqlen_k > 1 << 30 || p.hk > 65535) return false;
    const int ppt = kRows / p.g, bn = p.d == 256 ? 64 : 128, per_sm = p.d == 256 ? 1 : 2;
    const int64_t tiles = (p.max_seqlen_q + ppt - 1) / ppt;
    const int64_t base = tiles * p.hk * p.num_seqs;
    const int64_t slots = (int64_t)per_sm * num_sms;
    // Segments: about four waves of CTAs, each of eight key tiles at least; down to one
    // tile each while SMs are idle.
    int64_t splits = std::min<int64_t>((4 * slots + base - 1) / base, std::max<int64_t>(1, p.max_seqlen_k / (8 * bn)));
    splits = std::max<int64_t>(splits, std::min<int64_t>(slots / base, (p.max_seqlen_k + bn - 1) / bn));
    const size_t per_split = (size_t)p.total_q * p.hq * (p.d + 2) * sizeof(float);
    splits = std::max<int64_t>(1, std::min<int64_t>({splits, 64, (int64_t)(workspace_bytes / per_split)}));
    const int64_t per = (p.max_seqlen_k + splits - 1) / splits;
    plan->chunk = (int)std::min<int64_t>((per + bn - 1) / bn * bn, 1 << 30);
    plan->splits = (int)((p.max_seqlen_k + (int64_t)plan->chunk - 1) / plan->chunk);
    if (tiles * plan->splits > 0x7fffffffLL) return false;
    plan->tiles = (int)tiles;
    return true;
}

cudaError_t launch_tree(const TreePlan& plan, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const FwdParams& p,
                        cudaStream_t stream) {
    // Q map: [total_q, H_q, d]; box = 64 dims x g heads x floor(128 / g) nodes.
    CUtensorMap tq;
    cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.hq, (cuuint64_t)p.total_q};
    cuuint64_t strides[2] = {2ull * p.d, 2ull * p.d * p.hq};
    cuuint32_t box[3] = {64, (cuuint32_t)p.g, (cuuint32_t)(kRows / p.g)};
    if (!encode_bf16_sw128(&tq, p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
    switch (p.d) {
        case 64: return launch_tree_d<64>(plan, tq, tm_k, tm_v, p, stream);
        case 128: return launch_tree_d<128>(plan, tq, tm_k, tm_v, p, stream);
        case 256: return launch_tree_d<256>(plan, tq, tm_k, tm_v, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ua
