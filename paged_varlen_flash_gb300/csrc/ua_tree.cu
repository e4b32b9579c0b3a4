// ua_tree.cu -- attention for trees of drafted tokens over a bf16 paged cache, on tcgen05.
//
// A chunk's token sees every key of its context and, of the chunk's own keys, those
// whose bit its row of the mask has (its ancestors and itself).  With g query heads per
// KV head and S_q nodes a KV head has g S_q rows, a few up to some hundreds: every
// cached value is used that often, which is less than the tensor cores could do per
// byte of HBM (about 277 rows), so a batch of trees is bound by reading K and V once.
//
// Work.  An item is (row tile of floor(128 / g) nodes, sequence, KV head); it has as many
// steps as key tiles that its rows see.  All items' steps behind each other (row tile
// first, so that the row tiles of a batch read the same keys at about the same time) are
// cut into equal shares, one for every CTA that fits the machine.  A CTA walks through
// its share item by item; an item that lies in one share is written at once, one that is
// cut leaves a partial (m, l, o) in every share that it touches, joined by
// tree_merge_kernel in the order of the shares.  So no SM waits for a longer
// sequence of another one, and a batch has at most two partials per CTA.
//
// S = Q K^T and O += P V are tcgen05.mma with M = 128 rows over tiles of 64 keys; P goes
// over its own S in tensor memory.  Two S tiles, so that Q K^T of the next tile runs under
// the softmax of this one.  At d = 64 and 128 two CTAs share an SM (256 columns of tensor
// memory each, 80 and 96 KB of shared memory): while one waits for its copies, the other
// one's are in flight.  At d = 256 one CTA has the SM: Q lies in tensor memory (as the A
// operand from there a Q K^T of N = 64 takes 32 cycles per 16 dims, from shared memory 49:
// the rows of Q alone are 4 KB at 128 bytes a cycle), which leaves shared memory for
// three K and V tiles.  Barriers, tensor memory and the K/V rings live on from item to
// item: the next item's copies and first Q K^T run under the epilogue of the one before.
//
// Roles (8 warps, 9 at d = 256):
//   warps 0-3  softmax and epilogue: thread r owns row r (tensor-memory lane r); two
//              passes over the tile's columns (maximum, then P), with masks and score
//              terms in a short loop of their own;
//   warp 4     walks through the share and copies (TMA) Q and the K tiles, one lane per
//              paged block;
//   warp 5     looks through V tiles with keys that some row does not see;
//   warp 6     copies the V tiles;
//   warp 7     MMA issuer and owner of tensor memory (beside warp 3, which has the last
//              rows and the least to do); at d = 256 warp 8 issues the P V MMAs.
//
// Measured: 64 requests of 16 to 32 nodes, 512 to 8192 keys, 32 / 8 heads, d = 128: 205 us,
// 196 of them this kernel (1.2 GB of K and V, 6.1 TB/s, 0.90 of a plain copy); bound by HBM,
// then by the ramp at both ends.  4 requests of 64 nodes and 30,000 to 65,535 keys, 16 / 2
// heads, d = 256: 154 us with the same inputs again and again, 166 with others every time
// (1,280 and 1,180 TFLOP/s); about 1,630 cycles a tile of MMAs of 1,024, bound
// by the chain softmax -> P V -> Q K^T and L2 (four row tiles read every key, from HBM once).
// 48 trees of up to 64 nodes, softcap, window 1024, d = 64: 30 us, and one of 8 nodes over
// 999 keys 12 us: starting, one tile's latency, the epilogue and the merge.
//
// Masked keys: their scores are replaced, whatever K holds.  Their V rows reach the
// product with P = 0, and 0 times an infinity or NaN is NaN; so warp 5 clears values
// that are not finite in such tiles, and the epilogue adds them again to the rows that
// see their key (a flag, no cost while all values are finite).
#include <algorithm>
#include <cstdint>

#include "ua_common.cuh"
#include "ua_launch.h"
#include "ua_prefill_common.cuh"
#include "ua_ptx.cuh"
#include "ua_tc.cuh"
#include "ua_tmap.h"
#include "ua_tree.h"
#include "ua_tree_mask.cuh"

namespace ua {
namespace {

using namespace pf;

constexpr int kWarpCopy = 4;
constexpr int kWarpFix = 5;
constexpr int kWarpCopyV = 6;
constexpr int kWarpMmaT = 7;
constexpr int kWarpPv = 8;         // d = 256
constexpr int kCols = 64;          // columns of S a softmax thread holds at a time

// Score chains: the scale alone, a softcap, ALiBi with or without a softcap.
enum { kPlain = 0, kCap = 1, kAlibi = 2 };

// A piece of an item, written by the copy warp into a two-slot ring.
struct TreeUnit {
    int32_t live;          // 0: the share is done
    int32_t zero;          // malformed lengths: rows written as zeros
    int32_t s, hkv;
    int32_t q0, sq, sk;
    int32_t first, last;   // nodes of the tile
    int32_t t_begin, n;    // key tiles
    int32_t slot;          // of the partial, -1: the whole item
    int32_t odd;           // values that are not finite were cleared in V
    int32_t pad[3];
};
static_assert(sizeof(TreeUnit) == 64, "unit descriptor");

template <int D>
struct TCfg {
    static constexpr int kBN = 64;                      // keys per tile
    static constexpr int kStages = D == 64 ? 4 : D == 128 ? 2 : 3;    // K and V tiles each
    static constexpr int kBufs = 2;                     // S tiles
    static constexpr int kCtas = D == 256 ? 1 : 2;      // per SM
    static constexpr bool kTwo = D == 256;              // an MMA issuer each for Q K^T and P V
    static constexpr int kThreads = kTwo ? 288 : 256;
    static constexpr int kUnitReaders = 131 + kTwo;     // V copy, MMA and fix warps (a lane each), softmax threads
    static constexpr int kPanels = D / 64;
    static constexpr int kQPanel = kRows * 128;         // 128 rows x 64 dims
    static constexpr int kPanel = kBN * 128;            // kBN keys x 64 dims
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kTwo ? 0 : kPanels * kQPanel;        // d = 256: Q in tensor memory
    static constexpr int kOffV = kOffK + kStages * kTile;
    static constexpr int kOffBar = kOffV + kStages * kTile;
    // q_full, q_empty, {k_full, k_empty, v_full, v_ready, v_empty}[kStages], s_full[2],
    // p_full[2], o_done[2], o_free, u_full[2], u_empty[2], drain[2], never
    static constexpr int kNumBars = 2 + 5 * kStages + 14;
    static constexpr int kOffUnit = (kOffBar + kNumBars * 8 + 63) / 64 * 64;
    static constexpr int kOffMisc = kOffUnit + 2 * (int)sizeof(TreeUnit);
    static constexpr int kSmem = kOffMisc + 128 + 1024;   // (misc: addresses, 9 sums, the start)
    static constexpr int kTmemO = kBufs * kBN;
    static constexpr int kTmemQ = kTmemO + D;           // d = 256: two dims per column
    static constexpr uint32_t kCols2 = D == 256 ? 512 : 256;    // tensor-memory columns
    static_assert(kTmemO + D + (kTwo ? D / 2 : 0) <= (int)kCols2, "tensor memory budget");
    static_assert(kCtas * (kSmem + 1024) <= 233472, "shared memory budget");
};

// 32 bytes at once: a whole sector of a row, where every thread writes a row of its own.
__device__ __forceinline__ void store32b(void* dst, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// (Not to be moved in front of the wait for the kernel in front, which may write what it reads.)
__device__ __forceinline__ void load32b(uint32_t* v, const void* src) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(src)
                 : "memory");
}

// Values that are not finite among a row's visible V of keys [beg, end): the sum of
// them (0 if there are none) for 32 dims from c on is added to o.
__device__ __noinline__ void add_unbounded(const FwdParams& p, int s, int hkv, int64_t q0, const uint32_t* row, int beg, int end,
                                           int ctx, int sq, int sk, int lo, int c, uint32_t (&o)[32]) {
    const int b_log2 = 31 - __clz(p.b);
    for (int key = beg; key < end; ++key) {
        if (!(seen_keys(p, row, q0, key, ctx, sq, sk, lo) & 1u)) continue;
        const int32_t id = p.block_table[(int64_t)s * p.bt_stride + (key >> b_log2)];
        if (id < 0 || (int64_t)id >= p.num_blocks) continue;        // read as zeros
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v_cache) +
                                 (((int64_t)id * p.b + (key & (p.b - 1))) * p.hk + hkv) * p.d + c;
        for (int e = 0; e < 32; ++e) {
            const float x = __bfloat162float(v[e]);
            if (!(fabsf(x) <= 3.4e38f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
        }
    }
}

// 64-bit division where the operands need it.
__device__ __forceinline__ int64_t div_of(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Key tiles of the items of sequence s in row tile r: 0 where it has no such tile, 1 for
// malformed lengths (rows of zeros).
template <int BN>
__device__ __forceinline__ int item_steps(const FwdParams& p, int s, int r, uint32_t& st) {
    int sq, sk;
    int64_t q0;
    st = seq_status<true>(p, s, sq, sk, q0);
    if ((st & UA_DEVERR_CU_SEQLENS) || r * (kRows / p.g) >= sq) return 0;
    if (st) return 1;
    const int beg = (p.flags & UA_FLAG_WINDOW) ? max(0, sk - sq - p.window + 1) : 0;
    return (sk + BN - 1) / BN - beg / BN;
}

// A piece's K or V tiles through their ring, by a whole warp: lane i copies paged block i
// of each tile; block ids are fetched one tile ahead.  kt counts the ring's tiles.  (K and
// V have a warp each: behind V tiles, whose stage waits for the softmax, K tiles came a
// tile's time later.)
template <int D, bool V>
__device__ __forceinline__ bool copy_tiles(const FwdParams& p, const CUtensorMap& tm, uint32_t ring, uint32_t full0,
                                           uint32_t empty0, int& kt, int s, int hkv, int sk, int t_begin, int n,
                                           volatile int* abort_flag) {
    using C = TCfg<D>;
    constexpr int kBN = C::kBN;
    const int lane = threadIdx.x & 31;
    const int b = p.b, b_log2 = 31 - __clz(b), per_tile = kBN >> b_log2, nblk = (sk + b - 1) >> b_log2;
    const int32_t* bt = p.block_table + (int64_t)s * p.bt_stride;
    auto tile_id = [&](int j) -> int32_t {
        const int blk = ((t_begin + j) << (6 - b_log2)) + lane;
        return lane < per_tile && blk < nblk ? bt[blk] : -1;
    };
    static_assert(kBN == 64, "tile of whole blocks");
    int32_t id_next = tile_id(0);
    for (int j = 0; j < n; ++j, ++kt) {
        const int stg = kt % C::kStages;
        const int nb = min(per_tile, nblk - ((t_begin + j) << (6 - b_log2)));
        const int32_t id = id_next;
        if (j + 1 < n) id_next = tile_id(j + 1);
        if (!V && lane < nb && (id < 0 || (int64_t)id >= p.num_blocks)) atomicOr(p.err, (int)UA_DEVERR_BLOCK_ID);
        if (kt >= C::kStages &&
            !__all_sync(0xffffffffu, wait_or_abort(empty0 + 8 * stg, ((kt / C::kStages) + 1) & 1, abort_flag, p.err)))
            return false;
        if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * stg, (uint32_t)nb * b * 128 * C::kPanels);
        __syncwarp();
        if (lane < nb) {
#pragma unroll
            for (int pn = 0; pn < C::kPanels; ++pn)
                tma_load_4d(ring + stg * C::kTile + pn * C::kPanel + lane * b * 128, &tm, pn * 64, hkv, 0, id,
                            full0 + 8 * stg);
        }
    }
    return true;
}

template <int D, int MODE>
__global__ void __launch_bounds__(TCfg<D>::kThreads, TCfg<D>::kCtas)
tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const FwdParams p, const TreeShares w) {
    using C = TCfg<D>;
    constexpr int kBN = C::kBN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = p.g;
    const int ppt = kRows / g;                   // nodes per tile
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;

    uint64_t* bar_mem = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    constexpr int kS = 8 * C::kStages;
    const uint32_t q_full = smem_u32(bar_mem), q_empty = q_full + 8;
    const uint32_t k_full0 = q_full + 16, k_empty0 = k_full0 + kS;
    const uint32_t v_full0 = k_empty0 + kS, v_ready0 = v_full0 + kS, v_empty0 = v_ready0 + kS;
    const uint32_t s_full0 = v_empty0 + kS, p_full0 = s_full0 + 16, o_done0 = s_full0 + 32;
    const uint32_t o_free = s_full0 + 48, u_full0 = s_full0 + 56, u_empty0 = s_full0 + 72;
    const uint32_t drain0 = s_full0 + 88, never = s_full0 + 104;
    TreeUnit* units = reinterpret_cast<TreeUnit*>(smem + C::kOffUnit);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
    int64_t* warp_sums = reinterpret_cast<int64_t*>(smem + C::kOffMisc + 16);   // [9]
    int32_t* start = reinterpret_cast<int32_t*>(smem + C::kOffMisc + 96);       // entry, KV head, step

    if (threadIdx.x == 0) {
        mbar_init(q_full, C::kTwo ? kRows : 1);
        mbar_init(q_empty, 1);
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
            mbar_init(u_full0 + 8 * i, 1);
            mbar_init(u_empty0 + 8 * i, C::kUnitReaders);
        }
        mbar_init(o_free, kRows);
        mbar_init(drain0, 1);
        mbar_init(drain0 + 8, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMmaT) {
        tc::tmem_alloc(smem_u32(tmem_slot), C::kCols2);
        tc::tmem_relinquish();
    }
    griddep_wait();
    // This CTA's share: entries (row tile, sequence) in order, each thread a run of them.
    const uint32_t seqs = (uint32_t)p.num_seqs, entries = (uint32_t)w.tiles * seqs;      // (below 2^31)
    const uint32_t per = (entries + C::kThreads - 1) / C::kThreads;
    const uint32_t e_lo = min(entries, threadIdx.x * per), e_hi = min(entries, e_lo + per);
    int64_t mine = 0;
    int own_steps = 0;                           // of the run's first entry
    for (uint32_t e = e_lo; e < e_hi; ++e) {
        const int r = (int)(e / seqs), s = (int)(e - (uint32_t)r * seqs);
        uint32_t st;
        const int steps = item_steps<kBN>(p, s, r, st);
        if (e == e_lo) own_steps = steps;
        mine += steps ? steps + w.turn : 0;
        if (st && r == 0 && blockIdx.x == 0) atomicOr(p.err, (int)st);
    }
    mine *= p.hk;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sums[warp] = upto;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < C::kThreads / 32; ++i) {
        if (i < warp) upto += warp_sums[i];
        total += warp_sums[i];
    }
    // A share has w.least steps at least; share i begins at floor(total i / shares).
    const int64_t shares = min((int64_t)gridDim.x, div_of(total + w.least - 1, w.least));
    const bool idle = blockIdx.x >= shares;
    const int64_t each = idle ? 0 : div_of(total, shares);
    const uint32_t rest = idle ? 0 : (uint32_t)(total - each * shares);      // below 2^10, like the shares
    auto share_begin = [&](uint32_t i) -> int64_t { return each * i + rest * i / (uint32_t)shares; };
    const int64_t x0 = idle ? 0 : share_begin(blockIdx.x), x1 = idle ? 0 : share_begin(blockIdx.x + 1);
    if (!idle && x0 >= upto - mine && x0 < upto) {
        int64_t at = upto - mine;
        for (uint32_t e = e_lo; e < e_hi; ++e) {
            const int r = (int)(e / seqs), s = (int)(e - (uint32_t)r * seqs);
            uint32_t st;
            const int steps = e == e_lo ? own_steps : item_steps<kBN>(p, s, r, st), item = steps ? steps + w.turn : 0;
            const int64_t all = (int64_t)item * p.hk;
            if (x0 < at + all) {
                const int h = (int)div_of(x0 - at, item);
                start[0] = (int32_t)e;
                start[1] = h;
                start[2] = (int32_t)(x0 - at - (int64_t)h * item);
                start[3] = steps;
                break;
            }
            at += all;
        }
    }
    __syncthreads();
    const uint32_t sQ = smem_u32(smem + C::kOffQ);
    const uint32_t sK = smem_u32(smem + C::kOffK);
    const uint32_t sV = smem_u32(smem + C::kOffV);
    auto wwait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, p.err));
    };

    if (warp == kWarpCopy) {
        // ------------------------ the share's pieces, and copies ------------------------
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        int64_t x = x0;
        uint32_t e = idle ? 0 : (uint32_t)start[0];
        int hkv = idle ? 0 : start[1], step = idle ? 0 : start[2];
        int u = 0, qn = 0, kt = 0;     // units, Q loads, K tiles
        TreeJoin join{0, 0, 0, 0, 0};
        bool ok = true;
        for (;;) {
            const int slot = u & 1;
            if (u >= 2 && !(ok = wwait(u_empty0 + 8 * slot, ((u >> 1) + 1) & 1))) break;
            if (x >= x1) {
                if (lane == 0) {
                    units[slot].live = 0;
                    mbar_arrive(u_full0 + 8 * slot);
                }
                break;
            }
            // The next entry with steps (the first is known): 32 of them are looked at together.
            int steps = x == x0 ? start[3] : 0;
            while (steps == 0 && e < entries) {
                const uint32_t le = e + lane;
                uint32_t st_l = 0;
                const int r_l = (int)(le / seqs), s_l = (int)(le - (uint32_t)r_l * seqs);
                const int n_l = le < entries ? item_steps<kBN>(p, s_l, r_l, st_l) : 0;
                const unsigned some = __ballot_sync(0xffffffffu, n_l > 0);
                const int at = some ? __ffs(some) - 1 : 32;
                if (some) steps = __shfl_sync(0xffffffffu, n_l, at);
                e += at;
            }
            if (steps == 0) {                        // not reached: x < x1 <= total
                ok = false;
                *abort_flag = 1;
                break;
            }
            const int r = (int)(e / seqs), s = (int)(e - (uint32_t)r * seqs);
            int sq, sk;
            int64_t q0;
            const uint32_t st = seq_status<true>(p, s, sq, sk, q0);
            const int ctx = sk - sq, first = r * ppt;
            // The item's last w.turn steps stand for what an item costs besides its tiles.
            const int n_all = (int)min((int64_t)(steps + w.turn - step), x1 - x), n = min(n_all, steps - step);
            const int t_begin = (st || !window ? 0 : max(0, ctx - p.window + 1) / kBN) + step;
            const bool whole = n == steps;
            if (n > 0 && lane == 0) {
                TreeUnit& un = units[slot];
                un.live = 1;
                un.zero = st != 0;
                un.s = s;
                un.hkv = hkv;
                un.q0 = (int32_t)q0;
                un.sq = sq;
                un.sk = sk;
                un.first = first;
                un.last = min(first + ppt, sq) - 1;
                un.t_begin = t_begin;
                un.n = n;
                un.slot = whole ? -1 : 2 * (int)blockIdx.x + (x > x0 ? 1 : 0);
                un.odd = 0;
                mbar_arrive(u_full0 + 8 * slot);
            }
            if (n > 0 && !whole && step == 0) {
                // The item begins here: its shares up to the one that holds its last tile.
                const int64_t end = x + steps;
                join.pieces = (int)(div_of(end * shares - 1, total) - blockIdx.x) + 1;
                join.slot = 2 * (int)blockIdx.x + (x > x0 ? 1 : 0);
                join.row0 = q0 + first;
                join.nodes = min(first + ppt, sq) - first;
                join.hkv = hkv;
            }
            x += n_all;
            step += n_all;
            const int h_now = hkv;
            if (step == steps + w.turn) {
                step = 0;
                if (++hkv == p.hk) {
                    hkv = 0;
                    ++e;
                }
            }
            if (n <= 0) continue;
            ++u;
            if (st) continue;
            if (!C::kTwo) {
                if (qn >= 1 && !(ok = wwait(q_empty, (qn - 1) & 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (uint32_t)(g * ppt) * 128u * C::kPanels);
#pragma unroll
                    for (int pn = 0; pn < C::kPanels; ++pn)
                        tma_load_3d(sQ + pn * C::kQPanel, &tm_q, pn * 64, h_now * g, (int)q0 + first, q_full);
                }
                ++qn;
                __syncwarp();
            }
            ok = copy_tiles<D, false>(p, tm_k, sK, k_full0, k_empty0, kt, s, h_now, sk, t_begin, n, abort_flag);
            if (!ok) break;
        }
        if (lane == 0) w.joins[blockIdx.x] = join;
        if (*abort_flag && lane == 0) {
            // Let every copy this warp issued land before the CTA ends.
            if (qn > 0) mbar_wait_bounded(q_full, (qn - 1) & 1);
            for (int j = max(0, kt - C::kStages); j < kt; ++j)
                mbar_wait_bounded(k_full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == kWarpCopyV) {
        // -------------------------------- copies of V --------------------------------
        int kt = 0;
        bool ok = true;
        for (int u = 0;; ++u) {
            const int slot = u & 1;
            if (!(ok = wwait(u_full0 + 8 * slot, (u >> 1) & 1))) break;
            const TreeUnit& un = units[slot];
            const int live = un.live, zero = un.zero, s = un.s, hkv = un.hkv, sk = un.sk, t_begin = un.t_begin, n = un.n;
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty0 + 8 * slot);
            if (!live) break;
            if (zero) continue;
            if (!(ok = copy_tiles<D, true>(p, tm_v, sV, v_full0, v_empty0, kt, s, hkv, sk, t_begin, n, abort_flag))) break;
        }
        if (*abort_flag && lane == 0)
            for (int j = max(0, kt - C::kStages); j < kt; ++j)
                mbar_wait_bounded(v_full0 + 8 * (j % C::kStages), (j / C::kStages) & 1);
        __syncwarp();
    } else if (warp == kWarpMmaT || warp == kWarpPv) {
        // ----------------------- MMA issuers (one thread each) -----------------------
        // With one issuer MMAs run in its order, so the Q K^T that goes over columns holding
        // P cannot overtake the P V that reads them.  At d = 256, where the MMAs bound the
        // kernel, two issuers wait beside each other, and a Q K^T for the P V two tiles ago
        // (4 long requests 210 -> 191 us).
        constexpr int kNV = D == 64 ? 64 : 128;       // dims per P V MMA
        constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kRows, kBN, false, false);
        constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kRows, kNV, false, true);
        // Descriptors' lower words move with the address (in 16 bytes), the upper ones stay.
        const uint64_t qd = tc::smem_desc_sw128(sQ, 16, 1024);
        const uint64_t kd = tc::smem_desc_sw128(sK, 16, 1024);
        const uint64_t vd = tc::smem_desc_sw128(sV, C::kPanel, 1024);
        const uint32_t q_lo = (uint32_t)qd, qk_hi = (uint32_t)(qd >> 32);
        const uint32_t k_lo = (uint32_t)kd, v_lo = (uint32_t)vd, v_hi = (uint32_t)(vd >> 32);
        const bool does_qk = warp == kWarpMmaT, does_pv = !C::kTwo || warp == kWarpPv;
        int gt = 0, qn = 0;                           // key tiles and units with work before this unit
        bool ok = true;
        for (int u = 0;; ++u) {
            const int slot = u & 1;
            if (!(ok = wwait(u_full0 + 8 * slot, (u >> 1) & 1))) break;
            const int live = units[slot].live, zero = units[slot].zero, n = units[slot].n;
            __syncwarp();
            if (lane == 0) mbar_arrive(u_empty0 + 8 * slot);
            if (!live) break;
            if (zero) continue;
            auto issue_qk = [&](int j) -> bool {
                const int kt = gt + j, stg = kt % C::kStages, buf = kt % C::kBufs;
                // Testing hook: the first K wait waits on a barrier that nothing
                // completes and gives up after stall_ns.
                if (p.stall && kt == 0 &&
                    !__all_sync(0xffffffffu, wait_or_abort(never, 0, abort_flag, p.err, (uint64_t)p.stall_ns)))
                    return false;
                if (C::kTwo && kt >= 2 && !wwait(o_done0 + 8 * buf, ((kt - 2) >> 1) & 1)) return false;
                if (!wwait(k_full0 + 8 * stg, (kt / C::kStages) & 1)) return false;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint32_t kst = k_lo + stg * (C::kTile >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t k_at = kst + (k >> 2) * (C::kPanel >> 4) + (k & 3) * 2;
                        if constexpr (C::kTwo)
                            tc::mma_bf16_ts_lo(tmem + buf * kBN, tmem + C::kTmemQ + k * 8, k_at, qk_hi, idesc_qk, k > 0 ? 1u : 0u);
                        else
                            tc::mma_bf16_lo(tmem + buf * kBN, q_lo + (k >> 2) * (C::kQPanel >> 4) + (k & 3) * 2, qk_hi, k_at,
                                            qk_hi, idesc_qk, k > 0 ? 1u : 0u);
                    }
                    tc::commit(s_full0 + 8 * buf);
                    tc::commit(k_empty0 + 8 * stg);
                    if (!C::kTwo && j + 1 == n) tc::commit(q_empty);      // the last read of Q
                }
                __syncwarp();
                return true;
            };
            auto issue_pv = [&](int j) -> bool {
                const int kt = gt + j, stg = kt % C::kStages, buf = kt % C::kBufs;
                if (!wwait(v_ready0 + 8 * stg, (kt / C::kStages) & 1)) return false;
                if (!wwait(p_full0 + 8 * buf, (kt / C::kBufs) & 1)) return false;
                // The first P V overwrites O: the epilogue in front must have read it.
                if (j == 0 && qn > 0 && !wwait(o_free, (qn - 1) & 1)) return false;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint32_t vst = v_lo + stg * (C::kTile >> 4);
#pragma unroll
                    for (int k = 0; k < kBN / 16; ++k)
#pragma unroll
                        for (int h = 0; h < D / kNV; ++h)
                            // A = P from tensor memory (16 keys = 8 columns), B = V
                            // MN-major, two 64-dim panels.
                            tc::mma_bf16_ts_lo(tmem + C::kTmemO + h * kNV, tmem + buf * kBN + k * 8,
                                               vst + h * 2 * (C::kPanel >> 4) + k * 128, v_hi, idesc_pv,
                                               (j > 0 || k > 0) ? 1u : 0u);
                    tc::commit(o_done0 + 8 * buf);
                    tc::commit(v_empty0 + 8 * stg);
                }
                __syncwarp();
                return true;
            };
            if (does_qk) ok = wwait(q_full, qn & 1) && issue_qk(0);      // (fenced behind its second wait)
            for (int j = 0; ok && j < n; ++j) {
                // The next S tile is filled while the softmax has this one.
                if (does_qk && j + 1 < n) ok = issue_qk(j + 1);
                if (does_pv && ok) ok = issue_pv(j);
            }
            if (!ok) break;
            gt += n;
            ++qn;
        }
        if (*abort_flag) {
            // No MMA of this thread may still run when tensor memory is freed.
            const uint32_t drain = drain0 + (does_qk ? 0 : 8);
            if (tc::elect_one()) tc::commit(drain);
            __syncwarp();
            mbar_wait_bounded(drain, 0);
        }
    } else if (warp == kWarpFix) {
        // ------------------- V values that some rows must not see -------------------
        int gt = 0;
        bool ok = true;
        for (int u = 0; ok; ++u) {
            const int slot = u & 1;
            if (!(ok = wwait(u_full0 + 8 * slot, (u >> 1) & 1))) break;
            const TreeUnit& un = units[slot];
            const int live = un.live, zero = un.zero, n = un.n, t_begin = un.t_begin, sk = un.sk, ctx = sk - un.sq;
            const int full_lo = window ? max(0, sk - p.window) : 0, vis_beg = window ? max(0, ctx - p.window + 1) : 0;
            for (int j = 0; live && !zero && j < n; ++j, ++gt) {
                const int stg = gt % C::kStages, key0 = (t_begin + j) * kBN;
                if (!(ok = wwait(v_full0 + 8 * stg, (gt / C::kStages) & 1))) break;
                if (key0 < full_lo || key0 + kBN > ctx) {
                    uint4* v = reinterpret_cast<uint4*>(smem + C::kOffV + stg * C::kTile);
                    constexpr int kPanel16 = C::kPanel / 16;
                    // Keys of the tile that some row does not see: [0, part) and [from, upto);
                    // slots behind the end are nobody's and become zeros.
                    const int part = min(max(full_lo - key0, 0), kBN), upto = min(sk - key0, kBN);
                    const int from = max(part, min(max(ctx - key0, 0), kBN));
                    for (int pn = 0; pn < C::kPanels; ++pn)
                        for (int e = upto * 8 + lane; e < kBN * 8; e += 32) v[pn * kPanel16 + e] = make_uint4(0, 0, 0, 0);
                    // The largest magnitude as 16-bit integers: 0x7f80 and more is not finite.
                    uint32_t top = 0;
                    auto look = [&](int k_lo, int k_hi) {
                        for (int pn = 0; pn < C::kPanels; ++pn)
#pragma unroll 4
                            for (int e = k_lo * 8 + lane; e < k_hi * 8; e += 32) {
                                const uint4 x = v[pn * kPanel16 + e];
                                top = __vmaxu2(top, x.x & 0x7fff7fffu);
                                top = __vmaxu2(top, x.y & 0x7fff7fffu);
                                top = __vmaxu2(top, x.z & 0x7fff7fffu);
                                top = __vmaxu2(top, x.w & 0x7fff7fffu);
                            }
                    };
                    look(0, part);
                    look(from, upto);
                    if (__any_sync(0xffffffffu, max(top & 0xffffu, top >> 16) >= 0x7f80u)) {
#pragma unroll 1
                        for (int i = lane; i < C::kPanels * kBN * 32; i += 32) {     // words of two values
                            const int k = i / 32 % kBN;
                            if (k >= part && (k < from || k >= upto)) continue;
                            uint32_t* at = reinterpret_cast<uint32_t*>(v) + i;
                            const uint32_t x = *at;
                            uint32_t y = x;
                            if ((x & 0x7f80u) == 0x7f80u) y &= 0xffff0000u;
                            if ((x & 0x7f800000u) == 0x7f800000u) y &= 0xffffu;
                            if (y == x) continue;
                            *at = y;
                            if (key0 + k >= vis_beg) units[slot].odd = 1;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(v_ready0 + 8 * stg);
                __syncwarp();
            }
            // (The slot is given back by the softmax threads behind the epilogue.)
            if (lane == 0) mbar_arrive(u_empty0 + 8 * slot);
            if (!live) break;
        }
    } else if (warp < 4) {
        // ------------------------------ softmax, epilogue ------------------------------
        const int r = threadIdx.x;
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const bool softcap = MODE == kCap || (MODE == kAlibi && (p.flags & UA_FLAG_SOFTCAP) != 0);
        // The score chain is in log2 units from the products on (a factor of zero
        // would make NaN of masked scores).
        const float cap = p.softcap * kLog2e, fac = fmaxf(p.scale * (softcap ? 1.f / p.softcap : kLog2e), 0x1p-126f);
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0, wide_q = (reinterpret_cast<uintptr_t>(p.q) & 31u) == 0;
        int gt = 0;
        bool ok = true;
        for (int u = 0;; ++u) {
            const int slot_u = u & 1;
            if (!(ok = wwait(u_full0 + 8 * slot_u, (u >> 1) & 1))) break;
            const TreeUnit& un = units[slot_u];
            const int live_u = un.live, zero = un.zero, n = un.n, t_begin = un.t_begin;
            const int sq = un.sq, sk = un.sk, ctx = sk - sq, last = un.last, hkv = un.hkv, seq = un.s;
            const int part = un.slot;
            const int64_t q0 = un.q0;
            if (!live_u) break;
            const int i = un.first + r / g;
            const bool valid = r < g * ppt && i <= last;
            const int head = hkv * g + r % g;
            const int64_t row = (q0 + i) * p.hq + head;
            if (zero) {
                if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + row * D);
#pragma unroll 1
                    for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
                }
                mbar_arrive(u_empty0 + 8 * slot_u);
                continue;
            }
            const bool live = __any_sync(0xffffffffu, valid);   // else the warp only keeps the barriers going
            const int full_lo = window ? max(0, sk - p.window) : 0;
            const float slope = MODE == kAlibi && valid ? p.alibi[head] * kLog2e : 0.f;
            const uint32_t* mask = p.tree_mask + (q0 + min(i, last)) * p.mask_stride;
            int lo = 0;
            if ((window || MODE == kAlibi) && valid) {
                const int at = p.positions[q0 + i];
                if (at < ctx || at >= sk) atomicOr(p.err, (int)UA_DEVERR_TREE);
                if (window) lo = max(0, node_position(p, q0, i, ctx, sk) - p.window + 1);
            }
            if constexpr (C::kTwo) {
                // The row of Q into tensor memory.  (The last Q K^T of the unit before is
                // complete: its scores have been read.)
                if (live) {
                    // (Rows that are not there take the last one's values.)
                    const uint4* src = reinterpret_cast<const uint4*>(p.q + (valid ? row : (q0 + last) * p.hq + hkv * g) * D);
#pragma unroll 1
                    for (int c = 0; c < D / 2; c += 64) {
                        // 256 bytes in flight: the loads wait together.
                        uint32_t y[64];
#pragma unroll
                        for (int e = 0; e < 64; e += 8) {
                            if (wide_q) {
                                load32b(y + e, src + (c + e) / 4);
                            } else {
                                const uint4 u = src[(c + e) / 4], v = src[(c + e) / 4 + 1];
                                y[e] = u.x; y[e + 1] = u.y; y[e + 2] = u.z; y[e + 3] = u.w;
                                y[e + 4] = v.x; y[e + 5] = v.y; y[e + 6] = v.z; y[e + 7] = v.w;
                            }
                        }
                        tc::st32(trow + C::kTmemQ + c, *reinterpret_cast<uint32_t(*)[32]>(y));
                        tc::st32(trow + C::kTmemQ + c + 32, *reinterpret_cast<uint32_t(*)[32]>(y + 32));
                    }
                    tc::wait_st();
                }
                tc::fence_before_sync();
                mbar_arrive(q_full);
            }
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                const int kt = gt + j, buf = kt % C::kBufs;
                if (!(ok = wwait(s_full0 + 8 * buf, (kt / C::kBufs) & 1))) break;
                const int key0 = (t_begin + j) * kBN;
                const uint32_t s_col = trow + buf * kBN;
                const bool edge = key0 < full_lo || key0 + kBN > ctx;
                bool reanchor = false;
                float alpha = 1.f;
                if (live) {
                    tc::fence_after_sync();
                    // First pass: the maximum.  Plain scores stay as the MMA left them;
                    // score terms and masks are applied here and written back.
                    float top = -INFINITY;
                    if (MODE != kPlain || edge) {
#pragma unroll 1
                        for (int c = 0; c < kBN; c += 32) {
                            uint32_t x[32];
                            tc::ld32(s_col + c, x);
                            const int key = key0 + c;
                            const uint32_t see = edge ? seen_keys(p, mask, q0, key, ctx, sq, sk, lo) : 0xffffffffu;
                            int at = key + lane;                // position of the lane's key
                            if (MODE == kAlibi && at >= ctx && at < sk) at = node_position(p, q0, at - ctx, ctx, sk);
                            tc::wait_ld();
                            if (softcap) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    x[e] = __float_as_uint(cap * tanh_from_exp2(__uint_as_float(x[e]) * fac));
                            } else if (MODE != kPlain) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * fac);
                            }
                            if constexpr (MODE == kAlibi) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    x[e] = __float_as_uint(__uint_as_float(x[e]) +
                                                           slope * (float)(__shfl_sync(0xffffffffu, at, e) - ctx));
                            }
                            if (edge) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(see >> e & 1u)) x[e] = __float_as_uint(-INFINITY);
                            }
                            tc::st32(s_col + c, x);
                            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
#pragma unroll
                                for (int a = 0; a < 2; ++a)
                                    mx[a] = fmax3(mx[a], __uint_as_float(x[e + 2 * a]), __uint_as_float(x[e + 2 * a + 1]));
                            top = fmax3(top, mx[0], mx[1]);
                        }
                        tc::wait_st();
                    } else {
#pragma unroll 1
                        for (int c = 0; c < kBN; c += kCols) {
                            uint32_t x[kCols / 32][32];
#pragma unroll
                            for (int h = 0; h < kCols / 32; ++h) tc::ld32(s_col + c + h * 32, x[h]);
                            tc::wait_ld();
                            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int h = 0; h < kCols / 32; ++h)
#pragma unroll
                                for (int e = 0; e < 32; e += 8)
#pragma unroll
                                    for (int a = 0; a < 4; ++a)
                                        mx[a] = fmax3(mx[a], __uint_as_float(x[h][e + 2 * a]),
                                                      __uint_as_float(x[h][e + 2 * a + 1]));
                            top = fmax3(top, fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        }
                    }
                    if constexpr (MODE == kPlain) top *= fac;
                    reanchor = top > m + kLazy;
                    if (reanchor) {
                        alpha = fast_exp2(m - top);
                        m = top;
                    }
                    // Second pass: P = 2^(x - m), fp32 into the row sum, bf16 (V's type, as
                    // the MMA wants; 2^-8 off each) over columns of S that have been read.
                    const float mu = m == -INFINITY ? 0.f : m;
                    const float f = MODE == kPlain ? fac : 1.f;
                    const float2 f2 = make_float2(f, f), nm2 = make_float2(-mu, -mu);
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
                    // O holds the P V of the tiles up to j - 1, once the last of them is complete.
                    if (!(ok = wwait(o_done0 + 8 * ((kt - 1) & 1), ((kt - 1) >> 1) & 1))) break;
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
            if (!ok) break;
            gt += n;
            if (!(ok = wwait(o_done0 + 8 * ((gt - 1) % C::kBufs), ((gt - 1) / C::kBufs) & 1))) break;
            if (live) {
                // tcgen05.ld is warp-collective: every lane of a live warp loads.
                tc::fence_after_sync();
                const bool odd = *reinterpret_cast<const volatile int32_t*>(&un.odd) != 0;
                const int64_t prow = (int64_t)part * w.slot_rows + r;
                float f = 1.f;
                if (part >= 0) {
                    if (valid) {
                        p.part_ml[prow * 2 + 0] = stored_max(m, l);
                        p.part_ml[prow * 2 + 1] = l;
                    }
                } else {
                    float L = l;
                    if (p.flags & UA_FLAG_SINKS) {
                        const float s2 = p.sinks[head] * kLog2e;
                        if (s2 == INFINITY) {
                            L = 0.f;
                        } else if (s2 > m) {
                            f = m == -INFINITY ? 0.f : fast_exp2(m - s2);
                            L = L * f + 1.0f;
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
                    if (odd) {
                        const int beg = t_begin * kBN, end = min((t_begin + n) * kBN, sk);
                        add_unbounded(p, seq, hkv, q0, mask, beg, min(end, full_lo), ctx, sq, sk, lo, c * 32, o);
                        add_unbounded(p, seq, hkv, q0, mask, max(beg, max(full_lo, ctx)), end, ctx, sq, sk, lo, c * 32, o);
                    }
                    if (part >= 0) {
                        // Column by column: a warp's 32 rows are neighbours there (row by row
                        // these stores took 15,600 cycles at d = 256, this way
                        // 8,200).
                        const int64_t at = ((int64_t)part * D + c * 32) * w.slot_rows + r;
                        if (p.part_bf16) {
                            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.part_o) + at;
#pragma unroll
                            for (int e = 0; e < 32; ++e, dst += w.slot_rows) *dst = __float2bfloat16_rn(__uint_as_float(o[e]));
                        } else {
                            float* dst = p.part_o + at;
#pragma unroll
                            for (int e = 0; e < 32; ++e, dst += w.slot_rows) *dst = __uint_as_float(o[e]);
                        }
                    } else {
                        uint32_t h[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            h[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
                        __nv_bfloat16* dst = p.out + row * (int64_t)D + c * 32;
                        if (wide) {
                            store32b(dst, h);
                            store32b(dst + 16, h + 8);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(h[e], h[e + 1], h[e + 2], h[e + 3]);
                        }
                    }
                }
            }
            // O has been read: the next unit's first P V may overwrite it.
            tc::fence_before_sync();
            mbar_arrive(o_free);
            mbar_arrive(u_empty0 + 8 * slot_u);
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarpMmaT) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::kCols2);
    }
}

constexpr int kMergeCols = 8;

// Joins the pieces of the item that begins in share blockIdx.x and is cut by its end, in
// their order.  A thread has eight dims of a row, its warp 32 neighbouring rows, as the
// partials lie; four pieces' loads wait together.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const FwdParams p, const TreeShares w) {
    constexpr int N = kMergeCols, kAhead = 4;
    const int task = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int col = task % (D / N) * N, r = task / (D / N) * 32 + (threadIdx.x & 31);
    griddep_wait();                          // the partials are complete
    const TreeJoin join = w.joins[blockIdx.x];
    if (join.pieces == 0 || r >= join.nodes * p.g) return;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    float o[N], top = -INFINITY, l = 0.f;
#pragma unroll
    for (int t = 0; t < N; ++t) o[t] = 0.f;
#pragma unroll 1
    for (int m0 = 0; m0 < join.pieces; m0 += kAhead) {
        float x[kAhead][N];
        float2 st[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            st[q] = make_float2(-INFINITY, 0.f);
            if (m0 + q >= join.pieces) continue;
            // Piece m > 0 is the first of share blockIdx.x + m.
            const int64_t slot = m0 + q ? 2 * ((int)blockIdx.x + m0 + q) : join.slot;
            st[q] = ml[slot * w.slot_rows + r];
            const int64_t at = (slot * D + col) * w.slot_rows + r;
#pragma unroll
            for (int t = 0; t < N; ++t) x[q][t] = part_load(p, at + (int64_t)t * w.slot_rows);
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            if (st[q].x == -INFINITY) continue;      // a piece without keys: its o means nothing
            const float t = fmaxf(top, st[q].x), a = fast_exp2(top - t), b = fast_exp2(st[q].x - t);
            top = t;
            l = l * a + st[q].y * b;
#pragma unroll
            for (int k = 0; k < N; ++k) o[k] = o[k] * a + x[q][k] * b;
        }
    }
    const int i = r / p.g, h = join.hkv * p.g + r - i * p.g;
    float f = 1.f;
    if (p.flags & UA_FLAG_SINKS) {
        const float s2 = p.sinks[h] * kLog2e;
        if (s2 == INFINITY) {
            l = 0.f;
        } else if (s2 > top) {
            f = top == -INFINITY ? 0.f : fast_exp2(top - s2);
            l = l * f + 1.0f;
        } else if (s2 != -INFINITY) {
            l += fast_exp2(s2 - top);
        }
    }
    f = l > 0.f ? f * __frcp_rn(l) : 0.f;
    *reinterpret_cast<uint4*>(p.out + ((join.row0 + i) * p.hq + h) * D + col) =
        make_uint4(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f), pack_bf16x2(o[4] * f, o[5] * f),
                   pack_bf16x2(o[6] * f, o[7] * f));
}

template <int D>
cudaError_t launch_tree_d(const TreePlan& plan, const CUtensorMap& tq, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                          const FwdParams& p, cudaStream_t stream) {
    auto kern = (p.flags & UA_FLAG_ALIBI)     ? tree_kernel<D, kAlibi>
                : (p.flags & UA_FLAG_SOFTCAP) ? tree_kernel<D, kCap>
                                              : tree_kernel<D, kPlain>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TCfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_early(kern, dim3((unsigned)plan.ctas), TCfg<D>::kThreads, TCfg<D>::kSmem, stream, tq, tm_k, tm_v, p, plan.shares);
    if (e != cudaSuccess || plan.ctas == 1) return e;
    const unsigned tasks = (unsigned)((plan.shares.slot_rows + 31) / 32 * (D / kMergeCols));
    return launch_early(tree_merge_kernel<D>, dim3((unsigned)plan.ctas, (tasks + 7) / 8), 256, 0, stream, p, plan.shares);
}

int ctas_per_sm(int d) { return d == 256 ? 1 : 2; }

// Bytes of the partials of `ctas` shares whose tiles have `rows` rows, and of the joins.
size_t shares_bytes(int64_t ctas, int64_t rows, int d) {
    return (size_t)ctas * (2 * rows * (d + 2) * sizeof(float) + sizeof(TreeJoin)) + 16;
}

}  // namespace

size_t tree_workspace_bytes(const ua_problem_desc& d, int num_sms) {
    const int64_t g = d.num_q_heads / d.num_kv_heads;
    if (g > kRows) return 0;
    const int64_t rows = std::min<int64_t>(kRows / g, d.max_total_q) * g;
    return shares_bytes((int64_t)ctas_per_sm(d.head_size) * num_sms, rows, d.head_size);
}

bool plan_tree(FwdParams* fp, int num_sms, void* workspace, size_t workspace_bytes, TreePlan* plan) {
    const FwdParams& p = *fp;
    *plan = TreePlan();
    if (p.g > kRows || p.max_seqlen_k > 1 << 30) return false;
    const int ppt = kRows / p.g, bn = TCfg<64>::kBN;
    // (One tile at least: it reports sequences of more rows than a call allows, also one of none.)
    const int64_t tiles = std::max(1, (p.max_seqlen_q + ppt - 1) / ppt);
    // Nodes of a tile: no sequence has more than all tokens, whatever bound the call names.
    const int64_t rows = std::max<int64_t>(1, std::min<int64_t>({ppt, p.max_seqlen_q, p.total_q})) * p.g;
    if (tiles * p.num_seqs > 0x7fffffffLL) return false;
    // No more CTAs than steps (as far as the host knows) and than the workspace has room for.
    const int64_t steps = tiles * p.num_seqs * p.hk * ((p.max_seqlen_k + bn - 1) / bn);
    int64_t ctas = std::min<int64_t>((int64_t)ctas_per_sm(p.d) * num_sms, steps);
    ctas = std::max<int64_t>(1, ctas);
    while (ctas > 1 && shares_bytes(ctas, rows, p.d) > workspace_bytes) ctas = ctas * 7 / 8;
    plan->ctas = (int)ctas;
    plan->shares.tiles = (int)tiles;
    // Not too small shares: one request of 8000 keys, 2 KV heads, d = 64: 33.5, 23.2, 17.5 and
    // 16.5 us with 1, 2, 4 and 6 steps at least; 8 KV heads at d = 128 31.1, 31.0, 22.0 and 22.9.
    plan->shares.least = 5;
    // An item's turn (Q, the first tile's way through the pipeline, the epilogue) in key tiles:
    // 64 requests of 16 to 32 nodes at d = 128 225, 218, 213 and 212 us with 0, 2, 4 and 7 of
    // them, 48 small trees at d = 64 30 us with 3 and 33 with 8; at d = 256 159 and 157 us.
    plan->shares.turn = p.d == 256 ? 8 : 4;
    plan->shares.slot_rows = (int)rows;
    // Partials in front, then (m, l), then the joins.
    fp->part_o = static_cast<float*>(workspace);
    fp->part_ml = fp->part_o + (size_t)ctas * 2 * rows * p.d;
    plan->shares.joins = reinterpret_cast<TreeJoin*>((reinterpret_cast<uintptr_t>(fp->part_ml + (size_t)ctas * 4 * rows) + 15) &
                                                     ~uintptr_t(15));
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
