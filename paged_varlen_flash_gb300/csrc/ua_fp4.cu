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
// Work split.  A job is a (sequence, KV head, row tile); its keys count in
// steps of 32.  All steps of all jobs, in order, are cut into equal shares, one
// per resident warp, so that every SM streams the same number of bytes
// whatever the lengths are.  Warps share nothing but the search for their
// place: each streams its steps through its own ring of bulk copies, keeps its
// own (m, l, o) and has the next piece's copies in flight before it stores the
// last one's result, so no warp ever waits for another.  A job that a share
// boundary cuts has several pieces; each leaves (m, l, o) in the workspace and
// merge_kernel joins them in piece order.
//
// Measured: calls on the 64-request decode batch (270 k keys, 32 / 8 heads, d =
// 128, 346 MB) take 83 us with the merge, 4.2 TB/s; with two and four times the
// requests 15 us and 5.1 TB/s.  The same calls with the products and the softmax
// left out take 63 us, or 10 us and 6.5 TB/s (4 requests of 30,000 to 65,535 keys
// at d = 256: 42 and 31; one request of 1,000 keys: 12.5 and 10.4).  What the
// instructions add is latency as much as issue: 360 per warp and 16 keys (K about
// 107, V 134) fill 58 % of the issue slots of the 12 warps that 162 registers
// leave an SM, and a warp's two stages of copies cover little more than one step
// of them.  Four CTAs per SM
// were slower (115 us against 104 then), and so was claiming the last quarter of
// the steps dynamically (124 against 86: a change of piece waits 4 us).
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
#include <type_traits>

#include "ua_common.cuh"
#include "ua_fp4.cuh"
#include "ua_fp4.h"
#include "ua_launch.h"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kW = 4;           // warps per CTA
constexpr int kStep = 32;       // keys per ring stage
constexpr int kDepth = 2;       // ring stages per warp
constexpr int kSub = 4;         // sequences per thread and round of the work split
constexpr int kRound = kW * 32 * kSub;
constexpr int kTeamRows = 1024; // up to here merge_kernel gives a row whole CTAs
constexpr float kLazy4 = 8.0f;  // re-anchor when a step's max exceeds m by this (log2)

template <int D, int NT>
struct FCfg {
    static constexpr int kRows = 8 * NT;
    static constexpr int kKS = D / 16;                    // k steps of S^T, M tiles of O^T
    static constexpr int kCodeRow = D / 2;                // bytes of one key's codes
    static constexpr int kScaleRow = D / 16;
    static constexpr int kOp = kStep * (kCodeRow + kScaleRow);   // K or V of one step
    static constexpr int kStage = 2 * kOp;
    static constexpr int kQBytes = NT * kKS * 32 * 8;     // Q^T in fragment order, f16
    static constexpr int kWarp = kDepth * kStage + kQBytes + kRows * 4;   // ring, Q, Q's row scales
    static constexpr int kOffBar = kW * kWarp;
    static constexpr int kOffScan = kOffBar + (kW * kDepth + 1) * 8 + 8;
    static constexpr int kSmem = kOffScan + kRound * 4 + kSub * kW * 4;
    static_assert(kOp % 16 == 0 && kWarp % 16 == 0, "bulk copy alignment");
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

// V codes of one key that lane u holds: D / 8 dims as words of 8 dims.
template <int D>
__device__ __forceinline__ void load_v_words(const uint8_t* row, int u, uint32_t (&w)[D / 64]) {
    if constexpr (D == 64) {
        w[0] = *reinterpret_cast<const uint32_t*>(row + u * 4);
    } else if constexpr (D == 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + u * 8);
        w[0] = v.x; w[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(row + u * 16);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
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

// A wait gave up: report it, and let the warp's copies still in flight (the
// `n` steps from `first` on) land before the CTA ends.
__device__ __noinline__ void give_up(const FwdParams& p, uint32_t bar0, int first, int n) {
    if ((threadIdx.x & 31) == 0) atomicOr(p.err, (int)UA_DEVERR_TIMEOUT);
    for (int i = first; i < first + n; ++i) mbar_wait_bounded(bar0 + 8 * (i % kDepth), (i / kDepth) & 1);
    __syncwarp();
}

// Resident CTAs per SM that the registers allow (168 registers at three).
template <int D, int NT>
constexpr int kCtas = D == 256 ? (NT == 1 ? 2 : 1) : NT == 1 ? 3 : 2;

// One sequence's part of the work.
struct SeqWork {
    int64_t q0;       // first packed row
    int sq, sk;
    int beg;          // first step any of its rows sees
    int steps;        // steps of each of its jobs
    int tiles;        // row tiles per KV head
    uint32_t st;
};

template <int ROWS>
__device__ __forceinline__ uint32_t seq_work(const FwdParams& p, int s, SeqWork& w) {
    w.st = seq_status(p, s, w.sq, w.sk, w.q0);
    w.beg = w.steps = w.tiles = 0;
    if (w.st || w.sq <= 0) return 0;
    if (p.flags & UA_FLAG_WINDOW) w.beg = max(0, w.sk - w.sq - p.window + 1) / kStep;
    w.steps = (w.sk + kStep - 1) / kStep - w.beg;
    w.tiles = (p.g * w.sq + ROWS - 1) / ROWS;
    return (uint32_t)w.steps * w.tiles * p.hk;    // the planner keeps the batch's sum below 2^31
}

// Inclusive sums over the sequences of one round (thread i holds sequences
// i, i + 128, ... of it) into `prefix`; returns the round's total.
__device__ __forceinline__ uint32_t round_scan(const uint32_t (&n)[kSub], uint32_t* prefix, uint32_t* sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t incl[kSub];
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
        incl[k] = n[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl[k], o);
            if (lane >= o) incl[k] += v;
        }
        if (lane == 31) sums[k * kW + warp] = incl[k];
    }
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int k = 0; k < kSub; ++k)
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (w == warp) prefix[k * kW * 32 + threadIdx.x] = before + incl[k];
            before += sums[k * kW + w];
        }
    __syncthreads();
    return before;
}

// What a row's merged (m, l) make of its o: sum o * v_scale / l with the sink
// joined to the denominator (log2 units; a +inf sink takes all of it).
__device__ __forceinline__ float row_factor(const FwdParams& p, int head, float m, float l) {
    float f = p.v_scale;
    if (p.flags & UA_FLAG_SINKS) {
        const float s2 = __ldg(p.sinks + head) * kLog2e;
        if (s2 == INFINITY) {
            l = 0.f;
        } else if (s2 > m) {
            const float a = m == -INFINITY ? 0.f : fast_exp2(m - s2);
            f *= a;
            l = l * a + 1.0f;
        } else if (s2 != -INFINITY) {
            l += fast_exp2(s2 - m);
        }
    }
    return l > 0.f ? f * __frcp_rn(l) : 0.f;
}

// GEN: softcap, ALiBi or QQ-bias in the score chain.  EMIT: also store every
// row's scores (log2 units) and its final (m, l) for the key-weight kernel.
template <int D, int NT, bool GEN, bool EMIT>
__global__ void __launch_bounds__(kW * 32, (kCtas<D, NT>))
fp4_kernel(const FwdParams p) {
    using C = FCfg<D, NT>;
    // Used without rounding its address up: every consumer needs 16 bytes at
    // most, and the compiler keeps shared-memory (not generic) accesses.
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int u = lane >> 2, t = lane & 3;
    const int g = p.g;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    const uint32_t bar0 = smem_u32(bars + warp * kDepth);
    const uint32_t never = smem_u32(bars + kW * kDepth);
    uint8_t* ring = smem + warp * C::kWarp;
    uint8_t* q_frag = ring + kDepth * C::kStage;
    float* q_scale = reinterpret_cast<float*>(q_frag + C::kQBytes);
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + C::kOffScan);
    uint32_t* sums = prefix + kRound;
    if (lane == 0) {
        for (int i = 0; i < kDepth; ++i) mbar_init(bar0 + 8 * i, 1);
        if (warp == 0) mbar_init(never, 1);
        fence_mbar_init();
    }
    griddep_launch();

    // ---- work split: the batch's steps, then each warp's first sequence.  One
    // round covers 512 sequences; a second pass over the metadata is needed
    // only beyond that.
    uint32_t n[kSub], total = 0;
    auto load_round = [&](int s0, bool report) {
#pragma unroll
        for (int k = 0; k < kSub; ++k) {
            const int s = s0 + k * kW * 32 + (int)threadIdx.x;
            SeqWork w;
            w.st = 0;
            n[k] = s < p.num_seqs ? seq_work<C::kRows>(p, s, w) : 0u;
            if (report && s < p.num_seqs && w.st && s % (int)gridDim.x == (int)blockIdx.x) {
                atomicOr(p.err, (int)w.st);
                // Malformed lengths: the rows are written as zeros.
                if (!(w.st & UA_DEVERR_CU_SEQLENS))
                    for (int64_t e = 0; e < (int64_t)w.sq * p.hq * (D / 8); ++e)
                        reinterpret_cast<uint4*>(p.out + w.q0 * p.hq * D)[e] = make_uint4(0, 0, 0, 0);
            }
        }
    };
    uint32_t round_total = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kRound) {
        load_round(s0, true);
        round_total = round_scan(n, prefix, sums);
        total += round_total;
    }
    // p.chunk bounds the share from below: no job has more than p.splits pieces.
    const uint32_t warps = gridDim.x * kW;
    const uint32_t share = max((uint32_t)p.chunk, (total + warps - 1) / warps);
    const uint32_t my = blockIdx.x * kW + warp;
    uint32_t pos = (uint32_t)min((uint64_t)total, (uint64_t)my * share);
    const uint32_t pos_end = min(total, pos + share);
    int s = -1;
    uint32_t seq_base = 0;                // steps before sequence s
    for (int s0 = 0, base = 0; s0 < p.num_seqs; s0 += kRound) {
        if (p.num_seqs > kRound) {
            __syncthreads();
            load_round(s0, false);
            round_total = round_scan(n, prefix, sums);
        }
        if (s < 0 && pos < pos_end && pos - base < round_total) {
            // First sequence of the round whose inclusive sum exceeds pos.
            for (int i = 0; i < kRound; i += 32) {
                const unsigned hit = __ballot_sync(0xffffffffu, prefix[i + lane] > pos - base);
                if (hit) {
                    const int at = i + __ffs(hit) - 1;
                    s = s0 + at;
                    seq_base = base + (at ? prefix[at - 1] : 0u);
                    break;
                }
            }
        }
        base += round_total;
    }
    if (pos >= pos_end) return;
    SeqWork sw;
    seq_work<C::kRows>(p, s, sw);

    // ---- ring: a step's copies are issued by lanes 0-3, lane = 2 * run + op (op:
    // K or V).  A page is one contiguous run, codes then scales, so at b = 16 the
    // step is two whole pages per operand (run = page), at b = 32 one, and at
    // b = 64 half a page in two runs (run 0: codes, run 1: scales); a page's
    // image in the stage has codes first, then scales, in every case.
    const int b = p.b, b_log2 = 31 - __clz(b);   // b is 16, 32 or 64
    const int run = lane >> 1, op = lane & 1;
    const int runs = b == 32 ? 1 : 2;
    const int64_t page_bytes = fp4_page_bytes(b, D);
    constexpr int kTile = 16 * (C::kCodeRow + C::kScaleRow);      // image of 16 keys at b = 16
    const uint32_t copy_bytes = b == 16 ? kTile : b == 32 ? C::kOp : kStep * (run ? C::kScaleRow : C::kCodeRow);
    const uint32_t dst_off = (uint32_t)op * C::kOp + run * (b == 16 ? kTile : kStep * C::kCodeRow);
    // Offsets of the stage image: codes of 16-key tile kt at kt * code_kt, scales
    // at scale_0 + kt * scale_kt.
    const int code_kt = b == 16 ? kTile : 16 * C::kCodeRow;
    const int scale_0 = b == 16 ? 16 * C::kCodeRow : kStep * C::kCodeRow;
    const int scale_kt = b == 16 ? kTile : 16 * C::kScaleRow;
    const bool causal = (p.flags & UA_FLAG_CAUSAL) != 0;
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;
    const bool softcap = GEN && (p.flags & UA_FLAG_SOFTCAP) != 0;
    const bool alibi = GEN && (p.flags & UA_FLAG_ALIBI) != 0;
    const bool qq = GEN && (p.flags & UA_FLAG_QQ_BIAS) != 0;
    // The score chain is in log2 units from the products on.
    const float cap = p.softcap * kLog2e, cap_inv = softcap ? 1.f / p.softcap : kLog2e;

    // ---- the piece that is being copied and, from its first step on, computed
    int it = 0;                  // steps this warp has issued in earlier pieces
    int hkv, piece, pieces, sk, ctx, nrows, r0, i_first, h_first, vis_beg, vis_end, step0, steps, nblk;
    int64_t q0;
    const int32_t* bt;
    const uint8_t* cache;
    int32_t id_next;
    auto step_key = [&](int i) { return (step0 + i) * kStep; };
    auto block_of = [&](int i) -> int32_t {      // -2: no such block in this step
        if (run >= runs || i >= steps) return -2;
        const int blk = (step_key(i) + (b == 16 ? run * 16 : 0)) >> b_log2;
        return blk < nblk ? __ldg(bt + blk) : -2;
    };
    // Start the copies of step i; its block ids have been fetched one step ahead.
    auto issue = [&](int i) {
        const int32_t id = id_next;
        id_next = block_of(i + 1);
        if (i >= steps) return;
        const int slot = (it + i) % kDepth;
        const uint32_t bar = bar0 + 8 * slot;
        uint8_t* dst = ring + slot * C::kStage + dst_off;
        const bool good = id >= 0 && (int64_t)id < p.num_blocks;
        const unsigned mask = __ballot_sync(0xffffffffu, good);
        if (id != -2 && !good) {
            // A bad block: its keys read as zeros (the slots are later
            // overwritten by copies, hence the proxy fence).
            atomicOr(p.err, (int)UA_DEVERR_BLOCK_ID);
            for (uint32_t e = 0; e < copy_bytes; e += 4) *reinterpret_cast<uint32_t*>(dst + e) = 0;
            fence_proxy_async_smem();
        }
        // At b = 16 either page may be missing; else the whole step is there or not.
        if (lane == 0)
            mbar_arrive_expect_tx(bar, b == 16 ? (uint32_t)__popc(mask) * kTile : mask ? (uint32_t)C::kStage : 0u);
        __syncwarp();
        if (good) {
            // The second half of a 64-key page starts one copy further.
            const uint32_t half = b == 64 && (step_key(i) & 32) ? copy_bytes : 0;
            bulk_load(smem_u32(dst), cache + (int64_t)id * p.hk * page_bytes + half, copy_bytes, bar);
        }
    };
    // Tile row r: position i_first + (h_first + r) / g, head (h_first + r) mod g.
    auto pos_of = [&](int r) { return i_first + (int)((unsigned)(h_first + r) / (unsigned)g); };
    auto head_of = [&](int r) { return hkv * g + (int)((unsigned)(h_first + r) % (unsigned)g); };
    auto out_row = [&](int r) { return (q0 + pos_of(r)) * p.hq + head_of(r); };
    // Take the next piece, steps [pos, ...) of one job: start its copies, lay out
    // its Q (the last piece's steps are done with theirs).
    auto take = [&]() {
        while (pos - seq_base >= (uint32_t)sw.steps * sw.tiles * p.hk) {
            seq_base += (uint32_t)sw.steps * sw.tiles * p.hk;
            seq_work<C::kRows>(p, ++s, sw);
        }
        const uint32_t job = (pos - seq_base) / (uint32_t)sw.steps;
        const uint32_t job_base = seq_base + job * (uint32_t)sw.steps;
        const uint32_t end = min(pos_end, job_base + (uint32_t)sw.steps);
        hkv = (int)(job / (uint32_t)sw.tiles);
        r0 = (int)(job % (uint32_t)sw.tiles) * C::kRows;        // first packed row of the tile
        const uint32_t first = job_base / share;
        pieces = (int)((job_base + sw.steps - 1) / share - first) + 1;
        piece = (int)(my - first);
        sk = sw.sk;
        ctx = sk - sw.sq;
        q0 = sw.q0;
        nrows = min(C::kRows, g * sw.sq - r0);
        i_first = r0 / g;
        h_first = r0 - i_first * g;      // position and head of the tile's first row
        // Keys any row of the tile sees, and the piece's steps among them.
        vis_end = causal ? min(sk, (r0 + nrows - 1) / g + ctx + 1) : sk;
        vis_beg = window ? max(0, i_first + ctx - p.window + 1) : 0;
        step0 = max(vis_beg / kStep, sw.beg + (int)(pos - job_base));
        steps = max(0, min((vis_end + kStep - 1) / kStep, sw.beg + (int)(end - job_base)) - step0);
        nblk = (sk + b - 1) >> b_log2;
        bt = p.block_table + (int64_t)s * p.bt_stride;
        cache = static_cast<const uint8_t*>(op ? p.v_cache : p.k_cache) + hkv * page_bytes +
                (b == 64 && run ? b * C::kCodeRow : 0);
        pos = end;
        id_next = block_of(0);
        // Q (eight lanes a row) is fetched while the block ids are on their way,
        // where the registers allow it beside the last piece's o.
        constexpr int kPer = D / 8, kIter = C::kRows / 4;
        constexpr bool kEarly = NT * D <= 256;
        uint4 w[kEarly ? kIter : 1][kPer / 8];
        auto load_q = [&](int r, uint4 (&x)[kPer / 8]) {
#pragma unroll
            for (int c = 0; c < kPer / 8; ++c)
                x[c] = r < nrows ? __ldg(reinterpret_cast<const uint4*>(p.q + out_row(r) * D + (lane & 7) * kPer) + c)
                                 : make_uint4(0, 0, 0, 0);
        };
        if constexpr (kEarly) {
#pragma unroll
            for (int i = 0; i < kIter; ++i) load_q(4 * i + (lane >> 3), w[i]);
        }
#pragma unroll
        for (int i = 0; i < kDepth; ++i) issue(i);
        // Q as f16 in fragment order, each row scaled by a power of two so that
        // its largest magnitude lies in [1, 2) (f16 covers 2^-24 below that; the
        // factor goes into the row's score scale).
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int r = 4 * i + (lane >> 3), e0 = (lane & 7) * kPer;
            uint4 (&x)[kPer / 8] = w[kEarly ? i : 0];
            if constexpr (!kEarly) load_q(r, x);
            uint32_t amax = 0;
#pragma unroll
            for (int c = 0; c < kPer / 8; ++c)
                amax = __vmaxu2(amax, __vmaxu2(__vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu),
                                               __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu)));
            amax = max(amax & 0xffffu, amax >> 16);
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
            // Exponent field of the largest magnitude, kept where 2^-e is
            // normal (zeros, infinities and NaN: unscaled).
            const int ef = (int)(amax >> 7);
            const int e = (amax == 0 || ef == 255) ? 0 : min(max(ef, 1), 253) - 127;
            const float down = __int_as_float((127 - e) << 23);
            if ((lane & 7) == 0) q_scale[r] = __int_as_float((127 + e) << 23);
#pragma unroll
            for (int c = 0; c < kPer / 8; ++c) {
                const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    int step, tt, half;
                    q_place<D>(e0 + c * 8 + k * 2, step, tt, half);
                    reinterpret_cast<uint2*>(q_frag)[((r >> 3) * C::kKS + step) * 32 + (r & 7) * 4 + tt] =
                        make_uint2(pack_f16x2(bf16_lo(v[k]) * down, bf16_hi(v[k]) * down),
                                   pack_f16x2(bf16_lo(v[k + 1]) * down, bf16_hi(v[k + 1]) * down));
                }
            }
        }
        __syncwarp();
    };

    take();
    for (;;) {
        // ---- per-lane row constants: rows 8 n + 2t + c (mu: m, or 0 while m is
        // -inf).  Rows that do not exist see what the last row sees: their
        // results are never stored, and tile-wide tests stay simple.
        float m[NT][2], mu[NT][2], l[NT][2], fac[NT][2], slope[NT][2];
        int rlo[NT][2], rhi[NT][2], ri[NT][2];
        int full_lo = 0, full_hi = 0x7fffffff;       // keys every row of the tile sees
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 8 * j + 2 * t + c;
                const int i = pos_of(min(r, nrows - 1));
                m[j][c] = -INFINITY;
                mu[j][c] = l[j][c] = 0.f;
                ri[j][c] = i;
                rhi[j][c] = causal ? min(i + ctx, sk - 1) : sk - 1;
                rlo[j][c] = window ? max(0, i + ctx - p.window + 1) : 0;
                full_lo = max(full_lo, rlo[j][c]);
                full_hi = min(full_hi, rhi[j][c]);
                const float tau = p.scale * p.k_scale * q_scale[r];
                fac[j][c] = tau * (GEN ? cap_inv : kLog2e);
                slope[j][c] = alibi && r < nrows ? __ldg(p.alibi + head_of(r)) * kLog2e : 0.f;
            }
        full_lo = max(full_lo, __shfl_xor_sync(0xffffffffu, full_lo, 1));
        full_lo = max(full_lo, __shfl_xor_sync(0xffffffffu, full_lo, 2));
        full_hi = min(full_hi, __shfl_xor_sync(0xffffffffu, full_hi, 1));
        full_hi = min(full_hi, __shfl_xor_sync(0xffffffffu, full_hi, 2));

        float* scores[NT][2];            // EMIT: the rows' scores at the lane's first key
        if constexpr (EMIT) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    scores[j][c] = p.scores + out_row(min(8 * j + 2 * t + c, nrows - 1)) * p.score_stride + rho(u);
        }
        float o[C::kKS][NT][4];
#pragma unroll
        for (int i = 0; i < C::kKS; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][j][c] = 0.f;
        const uint2* qf = reinterpret_cast<const uint2*>(q_frag) + lane;

        if (p.stall && !__all_sync(0xffffffffu, mbar_wait_bounded(never, 0, (uint64_t)p.stall_ns))) {
            // Testing hook: a K/V wait that nothing completes has given up.
            give_up(p, bar0, it, min(steps, kDepth));
            return;
        }
        for (int i = 0; i < steps; ++i) {
            const int slot = (it + i) % kDepth;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + 8 * slot, ((it + i) / kDepth) & 1))) {
                give_up(p, bar0, it + i, min(steps - i, kDepth));
                return;
            }
            uint8_t* kst = ring + slot * C::kStage;
            uint8_t* vst = kst + C::kOp;
            const int key0 = step_key(i);
            if (key0 < full_lo || key0 + kStep - 1 > full_hi) {
                // Keys that some row does not see.  Those that no row of the tile
                // sees (past the end, before the window): their V scales become
                // 0, so that whatever the slots hold cannot reach O (0 * NaN is
                // NaN; codes are always finite).  Those that only some rows see:
                // NaN scales become 0 too, and the rows that see them take the
                // NaN here.
                const int key = key0 + lane;
                uint8_t* sc = vst + scale_0 + (lane >> 4) * scale_kt + (lane & 15) * C::kScaleRow;
                uint32_t bad = 0;                    // the key's NaN scales, one bit per 16 dims
                if (key < vis_beg || key >= vis_end) {
#pragma unroll
                    for (int e = 0; e < C::kScaleRow; e += 4) *reinterpret_cast<uint32_t*>(sc + e) = 0;
                    fence_proxy_async_smem();
                } else if (key < full_lo || key > full_hi) {
#pragma unroll 1
                    for (int e = 0; e < C::kScaleRow; ++e)
                        if ((sc[e] & 0x7f) == 0x7f) {
                            sc[e] = 0;
                            bad |= 1u << e;
                        }
                    if (bad) fence_proxy_async_smem();
                }
                __syncwarp();
                for (unsigned some = __ballot_sync(0xffffffffu, bad != 0); some; some &= some - 1) {
                    const int from = __ffs(some) - 1;
                    const uint32_t groups = __shfl_sync(0xffffffffu, bad, from);
#pragma unroll
                    for (int k = 0; k < C::kKS; ++k) {
                        if (!(groups >> ((u * (D / 8) + (k >> 2) * 8) >> 4) & 1)) continue;
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (key0 + from >= rlo[j][c] && key0 + from <= rhi[j][c])
                                    o[k][j][c] = o[k][j][c + 2] = __int_as_float(0x7fffffff);
                    }
                }
            }

            // S^T = K Q^T for two 16-key tiles.
            float sacc[2][NT][4];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) sacc[kt][j][c] = 0.f;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const uint8_t* codes = kst + kt * code_kt + rho(u) * C::kCodeRow;
                const uint8_t* scales = kst + scale_0 + kt * scale_kt + rho(u) * C::kScaleRow;
                uint32_t wa[D / 32], wb[D / 32], sa[D / 64], sb[D / 64];
                load_k_words<D>(codes, t, wa);
                load_k_words<D>(codes + 8 * C::kCodeRow, t, wb);
                load_k_scales<D>(scales, t, sa);
                load_k_scales<D>(scales + 8 * C::kScaleRow, t, sb);
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
                        for (int j = 0; j < NT; ++j) {
                            const uint2 qv = qf[(j * C::kKS + 2 * w + k) * 32];
                            mma_f16(sacc[kt][j], ha[2 * k], hb[2 * k], ha[2 * k + 1], hb[2 * k + 1], qv.x, qv.y);
                        }
                }
            }

            // Score chain, masks, running maximum.
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4) {
                        const int c = c4 & 1;
                        float x = sacc[kt][j][c4] * fac[j][c];
                        if constexpr (GEN) {
                            const int key = key0 + kt * 16 + rho(u) + (c4 >> 1) * 8;
                            if (softcap) x = cap * tanh_from_exp2(x);
                            if (alibi) x += slope[j][c] * (float)(key - ctx);
                            if (qq && key >= ctx && key <= rhi[j][c])
                                x += __ldg(p.qq_bias + (int64_t)ri[j][c] * p.qq_stride + (key - ctx)) * kLog2e;
                        }
                        sacc[kt][j][c4] = x;
                    }
            if (key0 < full_lo || key0 + kStep - 1 > full_hi) {
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int c4 = 0; c4 < 4; ++c4) {
                            const int key = key0 + kt * 16 + rho(u) + (c4 >> 1) * 8;
                            if (key < rlo[j][c4 & 1] || key > rhi[j][c4 & 1]) sacc[kt][j][c4] = -INFINITY;
                        }
            }
            if constexpr (EMIT) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (8 * j + 2 * t + c >= nrows) continue;
                        float* dst = scores[j][c] + key0;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (key0 + rho(u) + 8 * k < sk) dst[8 * k] = sacc[k >> 1][j][c + 2 * (k & 1)];
                    }
            }
            float tmax[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    tmax[j][c] = fmaxf(fmaxf(sacc[0][j][c], sacc[0][j][c + 2]), fmaxf(sacc[1][j][c], sacc[1][j][c + 2]));
            bool up = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) up |= tmax[j][c] > m[j][c] + kLazy4;
            if (__any_sync(0xffffffffu, up)) {
                // Re-anchor rows whose step maximum (over the 8 lanes that share
                // the row) exceeds m by more than the threshold.
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = tmax[j][c];
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        if (v > m[j][c] + kLazy4) {
                            const float a = fast_exp2(m[j][c] - v);
                            m[j][c] = mu[j][c] = v;
                            l[j][c] *= a;
#pragma unroll
                            for (int k = 0; k < C::kKS; ++k) {
                                o[k][j][c] *= a;
                                o[k][j][c + 2] *= a;
                            }
                        }
                    }
            }

            // P = 2^(x - m): fp32 into the row sums, f16 into the MMA (11 bits;
            // m trails the maximum by at most 8, so P <= 2^8.  P below 2^-14 is off
            // by up to 2^-25, of a row sum that is at least 1).
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float e[4];
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4) {
                        e[c4] = fast_exp2(sacc[kt][j][c4] - mu[j][c4 & 1]);
                        l[j][c4 & 1] += e[c4];
                    }
                    pb[kt][j][0] = transpose8(pack_f16x2(e[0], e[1]));
                    pb[kt][j][1] = transpose8(pack_f16x2(e[2], e[3]));
                }

            // O^T += V^T P^T.
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const int k0 = t, k1 = (t + 4) ^ 1;  // key indexes 2t, 2t + 1; + 8: the others
                uint32_t wv[4][D / 64];              // keys k0, k1, k0 + 8, k1 + 8: words of 8 dims
                const uint8_t* codes = vst + kt * code_kt;
                load_v_words<D>(codes + k0 * C::kCodeRow, u, wv[0]);
                load_v_words<D>(codes + k1 * C::kCodeRow, u, wv[1]);
                load_v_words<D>(codes + (k0 + 8) * C::kCodeRow, u, wv[2]);
                load_v_words<D>(codes + (k1 + 8) * C::kCodeRow, u, wv[3]);
                const uint8_t* sc = vst + scale_0 + kt * scale_kt;
                uint32_t sp[2] = {0, 0};             // scales of the two keys of a pair, f16x2
#pragma unroll
                for (int w = 0; w < D / 64; ++w) {
                    if (w % 2 == 0) {                // a scale covers two words
                        const int gi = (u * (D / 8) + w * 8) / 16;
#pragma unroll
                        for (int pr = 0; pr < 2; ++pr)
                            sp[pr] = e4m3x2_to_f16((uint32_t)sc[(k0 + 8 * pr) * C::kScaleRow + gi] |
                                                   ((uint32_t)sc[(k1 + 8 * pr) * C::kScaleRow + gi] << 8));
                    }
                    uint32_t h[2][2][4];             // [key pair][dim parity][byte]
#pragma unroll
                    for (int pr = 0; pr < 2; ++pr) {
                        const uint32_t a = wv[2 * pr][w], c = wv[2 * pr + 1][w];
                        e2m1x8_to_f16((a & 0x0f0f0f0fu) | ((c << 4) & 0xf0f0f0f0u), h[pr][0]);
                        e2m1x8_to_f16(((a >> 4) & 0x0f0f0f0fu) | (c & 0xf0f0f0f0u), h[pr][1]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            h[pr][0][k] = mul_f16x2(h[pr][0][k], sp[pr]);
                            h[pr][1][k] = mul_f16x2(h[pr][1][k], sp[pr]);
                        }
                    }
                    // M tile (w, k): row u = dim 8w + 2k of the lane's run, row u + 8 the next.
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            mma_f16(o[w * 4 + k][j], h[0][0][k], h[0][1][k], h[1][0][k], h[1][1][k], pb[kt][j][0],
                                    pb[kt][j][1]);
                }
            }
            __syncwarp();
            issue(i + kDepth);
        }
        it += steps;

        // ---- store: (m, l, o) of the piece, or the finished rows of a job in
        // one piece.  The next piece's copies start first.
        const int e_pieces = pieces, e_piece = piece, e_rows = nrows;
        int64_t e_row[NT][2];
        int e_head[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = min(8 * j + 2 * t + c, nrows - 1);
                e_row[j][c] = out_row(r);
                e_head[j][c] = head_of(r);
            }
        const bool more = pos < pos_end;
        if (more) take();
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = l[j][c];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (8 * j + 2 * t + c >= e_rows) continue;
                const int64_t row = e_row[j][c];
                const float2 ml = make_float2(stored_max(m[j][c], v), v);
                if (e_piece == 0 && u == 0) p.row_pieces[row] = make_int4(e_pieces, e_pieces, e_pieces, e_pieces);
                if (e_pieces == 1) {
                    if (EMIT && u == 0) *reinterpret_cast<float2*>(p.part_ml + row * 2) = ml;
                    const float f = row_factor(p, e_head[j][c], m[j][c], v);
                    uint2* dst = reinterpret_cast<uint2*>(p.out + row * D + u * (D / 8));
#pragma unroll
                    for (int k = 0; k < C::kKS; k += 2)
                        dst[k / 2] = make_uint2(pack_bf16x2(o[k][j][c] * f, o[k][j][c + 2] * f),
                                                pack_bf16x2(o[k + 1][j][c] * f, o[k + 1][j][c + 2] * f));
                    continue;
                }
                const int64_t at = row * p.splits + e_piece;
                if (u == 0) *reinterpret_cast<float2*>(p.piece_ml + at * 2) = ml;
#pragma unroll
                for (int k = 0; k < C::kKS; k += 2) {
                    const int64_t e = at * D + u * (D / 8) + 2 * k;
                    if (p.part_bf16)
                        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.part_o) + e) =
                            make_uint2(pack_bf16x2(o[k][j][c], o[k][j][c + 2]),
                                       pack_bf16x2(o[k + 1][j][c], o[k + 1][j][c + 2]));
                    else
                        *reinterpret_cast<float4*>(p.part_o + e) =
                            make_float4(o[k][j][c], o[k][j][c + 2], o[k + 1][j][c], o[k + 1][j][c + 2]);
                }
            }
        if (!more) return;
    }
}

// Joins the pieces of the rows that have more than one, in piece order, and
// leaves row_pieces at 0.  TEAM: a CTA of eight warps per row and 64 dims, each
// warp an eighth of the pieces (few rows, cut into many pieces: 150 at most on
// the four-request batch at d = 256, joined in 5 us); else a warp per row.
// kAhead pieces' loads are in flight at a time, and their statistics with them:
// the running maximum is re-anchored once per batch.
constexpr int kAhead = 8;

template <int D, bool EMIT, bool TEAM>
__global__ void __launch_bounds__(256) merge_kernel(const FwdParams p) {
    constexpr int kPer = TEAM ? 2 : D / 32;  // dims per lane
    constexpr int kParts = TEAM ? D / 64 : 1;
    __shared__ float2 s_ml[8];
    __shared__ float2 s_o[TEAM ? 8 : 1][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = TEAM ? (int64_t)blockIdx.x / kParts : (int64_t)blockIdx.x * 8 + warp;
    const int part = TEAM ? blockIdx.x % kParts : 0;
    griddep_wait();
    if (row >= p.total_q * p.hq) return;
    // Each part of a row has its own copy of the count to read and clear.
    int n;
    if constexpr (TEAM) {
        int* count = reinterpret_cast<int*>(p.row_pieces + row) + part;
        n = *count;
        __syncthreads();
        if (threadIdx.x == 0) *count = 0;
    } else {
        n = p.row_pieces[row].x;
        __syncwarp();
        if (lane == 0) p.row_pieces[row] = make_int4(0, 0, 0, 0);
    }
    if (n <= 1) return;
    const int per = TEAM ? (n + 7) / 8 : n;
    const int k0 = TEAM ? min(n, warp * per) : 0, k1 = min(n, k0 + per);
    const float2* st = reinterpret_cast<const float2*>(p.piece_ml) + row * p.splits;
    const int64_t o0 = row * p.splits * D + part * 64 + lane * kPer;
    float M = -INFINITY, L = 0.f, acc[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
    auto join = [&](auto bf16_parts) {
        constexpr bool kBf16 = decltype(bf16_parts)::value;
        constexpr int kWords = kBf16 ? kPer / 2 : kPer;
        for (int kk = k0; kk < k1; kk += kAhead) {
            float2 v[kAhead];
            uint32_t x[kAhead][kWords];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int k = min(kk + q, k1 - 1);
                v[q] = st[k];
                const uint32_t* src =
                    kBf16 ? reinterpret_cast<const uint32_t*>(reinterpret_cast<const __nv_bfloat16*>(p.part_o) + o0 +
                                                              (int64_t)k * D)
                          : reinterpret_cast<const uint32_t*>(p.part_o + o0 + (int64_t)k * D);
#pragma unroll
                for (int e = 0; e < kWords; ++e) x[q][e] = src[e];
            }
            float top = M;
#pragma unroll
            for (int q = 0; q < kAhead; ++q) top = fmaxf(top, v[q].x);
            if (top == -INFINITY) continue;              // pieces the row sees no key of
            const float back = fast_exp2(M - top);
            M = top;
            L *= back;
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] *= back;
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                if (kk + q >= k1) break;
                const float a = fast_exp2(v[q].x - M);
                L = fmaf(a, v[q].y, L);
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const uint32_t w = x[q][kBf16 ? e / 2 : e];
                    acc[e] = fmaf(a, kBf16 ? (e & 1 ? bf16_hi(w) : bf16_lo(w)) : __uint_as_float(w), acc[e]);
                }
            }
        }
    };
    if (p.part_bf16) join(std::true_type{});
    else join(std::false_type{});
    if constexpr (TEAM) {
        if (lane == 0) s_ml[warp] = make_float2(M, L);
        s_o[warp][lane] = make_float2(acc[0], acc[1]);
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int q = 1; q < 8; ++q) M = fmaxf(M, s_ml[q].x);
        L = acc[0] = acc[1] = 0.f;
        if (M != -INFINITY)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float a = fast_exp2(s_ml[q].x - M);
                L = fmaf(a, s_ml[q].y, L);
                acc[0] = fmaf(a, s_o[q][lane].x, acc[0]);
                acc[1] = fmaf(a, s_o[q][lane].y, acc[1]);
            }
    }
    if (EMIT && lane == 0 && part == 0) *reinterpret_cast<float2*>(p.part_ml + row * 2) = make_float2(M, L);
    const float f = row_factor(p, (int)(row % p.hq), M, L);
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(p.out + row * D + part * 64 + lane * kPer + e) =
            pack_bf16x2(acc[e] * f, acc[e + 1] * f);
}

template <int D, int NT, bool GEN, bool EMIT>
cudaError_t launch_t(const Fp4Plan& plan, const FwdParams& p, cudaStream_t stream) {
    using C = FCfg<D, NT>;
    auto kern = fp4_kernel<D, NT, GEN, EMIT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)plan.ctas, kW * 32, C::kSmem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The merge may be scheduled while the last pieces finish; it waits for
    // them (griddep_wait) before it reads anything.
    const int64_t rows = p.total_q * p.hq;
    const bool team = rows <= kTeamRows;
    const dim3 grid((unsigned)(team ? rows * (D / 64) : (rows + 7) / 8));
    return launch_early(team ? merge_kernel<D, EMIT, true> : merge_kernel<D, EMIT, false>, grid, 256, 0, stream, p);
}

template <int D>
cudaError_t launch_d(const Fp4Plan& plan, const FwdParams& p, cudaStream_t stream) {
    const bool gen = (p.flags & (UA_FLAG_SOFTCAP | UA_FLAG_ALIBI | UA_FLAG_QQ_BIAS)) != 0;
    const bool emit = p.scores != nullptr;
    if (plan.rows == 8) {
        if (emit) return gen ? launch_t<D, 1, true, true>(plan, p, stream) : launch_t<D, 1, false, true>(plan, p, stream);
        return gen ? launch_t<D, 1, true, false>(plan, p, stream) : launch_t<D, 1, false, false>(plan, p, stream);
    }
    if (emit) return gen ? launch_t<D, 2, true, true>(plan, p, stream) : launch_t<D, 2, false, true>(plan, p, stream);
    return gen ? launch_t<D, 2, true, false>(plan, p, stream) : launch_t<D, 2, false, false>(plan, p, stream);
}

int resident_ctas(int d, int rows) {
    if (rows == 8) return d == 64 ? kCtas<64, 1> : d == 128 ? kCtas<128, 1> : kCtas<256, 1>;
    return d == 64 ? kCtas<64, 2> : d == 128 ? kCtas<128, 2> : kCtas<256, 2>;
}

}  // namespace

size_t fp4_workspace_bytes(int64_t rows, int d) { return (size_t)rows * (d + 2) * sizeof(float); }

bool plan_fp4(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4Plan* plan) {
    *plan = Fp4Plan();
    const int64_t rows = (int64_t)p.g * p.max_seqlen_q;
    if (rows >= 1 << 30 || p.max_seqlen_k > 1 << 30 || p.total_q * p.hq >= int64_t(1) << 32) return false;
    plan->rows = rows <= 8 ? 8 : 16;
    // The batch's steps stay below 2^31; no more CTAs than it can have steps.
    const int64_t steps = (p.max_seqlen_k + (int64_t)kStep - 1) / kStep;
    const int64_t tiles = std::min((rows + plan->rows - 1) / plan->rows * p.num_seqs,
                                   p.total_q * p.g / plan->rows + p.num_seqs);
    if ((double)steps * tiles * p.hk >= 2147483647.0) return false;
    const int64_t most = (int64_t)num_sms * resident_ctas(p.d, plan->rows);
    plan->ctas = (int)std::max<int64_t>(1, std::min<int64_t>(most, (steps * tiles * p.hk + kW - 1) / kW));
    // Pieces per job: what the workspace holds, at least two of which the
    // problem's creation guarantees; a job of `steps` steps in shares of at
    // least `chunk` has at most ceil(steps / chunk) + 1 pieces.
    const size_t per_split = fp4_workspace_bytes(p.total_q * p.hq, p.d);
    const int64_t slots = std::min<int64_t>((int64_t)(workspace_bytes / per_split), steps + 1);
    if (slots < 2) return false;
    plan->splits = (int)slots;
    plan->chunk = (int)std::max<int64_t>(1, (steps + slots - 2) / (slots - 1));
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
