// ua_evict.cu -- eviction by accumulated attention weight: per (sequence, KV
// head) the `budget` kept keys are found (select_kernel) and their cache rows
// moved to the front of the destination table (move_kernel).
//
// Select: a cluster of 1, 2, 4 or 8 CTAs per (sequence, KV head), each with a
// run of the keys (up to 8192 of them stay in shared memory; a longer run, past
// 65536 keys, is read again in every pass).  A weight's bits, flipped so that
// unsigned order is float order, are searched for the m-th largest of the n candidates by three radix passes
// (11 + 11 + 10 bits) over shared-memory histograms, of which the cluster's CTAs
// read 32 sums and 64 bins from one another; one pass in key order then writes the kept positions,
// taking keys above the threshold, the first `need` of those equal to it, and
// the recent tail.
//
// Move: a CTA takes a run of 256 ranks, a warp 32 neighbouring ones, looks its
// rows' pages up once (lane = rank) and copies them in 16-byte pieces, eight
// loads per thread in flight before the first store.  A kept key's new position is never
// behind its old one, so in place a CTA that walks the ranks in order and has
// read a whole round before it writes any of it overwrites nothing unread.
//
// Measured: 512 heads of up to 8191 weights 24 us (a CTA each), 8 heads of up to
// 65535 14.5 us (clusters of eight; a pass is 1 us of counting and 1.3 of barrier
// and exchange); moving 2048 bf16 rows of each of the 512 163 us, 6.3 TB/s of reads
// and writes.
#include <algorithm>
#include <cstdint>

#include "ua_cache.h"
#include "ua_fp4.cuh"
#include "ua_launch.h"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kSelKeys = 8192;  // keys a cluster's CTA should have, kept in shared memory
constexpr int kBins = 2048;
constexpr int kMove = 256;      // threads of move_kernel
constexpr int kHold = 8;        // 16-byte pieces a move thread holds at a time
constexpr int kRanks = kMove;   // ranks of a CTA's round: 32 per warp

// Order-preserving bits: NaN first (0), -0 with +0, +inf last.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_incl_scan(uint32_t v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// A 32-bit word, or two, of the same shared-memory variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_word(const uint32_t* local, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}

__device__ __forceinline__ uint2 cluster_pair(const uint2* local, uint32_t rank) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}

template <int CL>
__device__ __forceinline__ void team_sync() {
    if constexpr (CL == 1) __syncthreads();
    else cluster_sync_all();
}

// Threads: 512 where a CTA works alone (three share an SM at 40 registers; four,
// at 32, spill: 199 against 193 us for the 64-request eviction), 1024 in a cluster
// (few CTAs, each should be quick).
template <int CL>
constexpr int kSelThreads = CL == 1 ? 512 : 1024;

// Dynamic shared memory: the run's weights, the histogram, its copy in pairs of
// bins from the top (in a cluster of two passes: another CTA may still read the
// last one's).
template <int CL>
constexpr int kPairs = CL == 1 ? 1 : 2;
template <int CL>
constexpr int kSelSmem = (kSelKeys + kBins) * 4 + kPairs<CL> * (kBins / 2) * 8;

template <int CL>
__global__ void __launch_bounds__(kSelThreads<CL>, CL == 1 ? 3 : 1) select_kernel(const EvictParams p) {
    constexpr int kSel = kSelThreads<CL>;
    constexpr int kKeep = kSelKeys / kSel;    // weights a thread holds of a run (or of 8192 keys of it)
    extern __shared__ __align__(16) float keep[];   // [kSelKeys], weight of key j0 + i at i
    uint32_t* hist = reinterpret_cast<uint32_t*>(keep + kSelKeys);
    uint2* pairs = reinterpret_cast<uint2*>(hist + kBins);
    __shared__ uint32_t sums[kPairs<CL>][32];       // of 64 bins each, from the top
    __shared__ uint32_t counts[kKeep * (kSel / 32) + 1];
    __shared__ uint32_t found[2];
    __shared__ uint32_t mine[2];              // this CTA's keys above and equal to the threshold
    const uint32_t rank = CL == 1 ? 0u : cluster_ctarank();
    const int h = blockIdx.x / CL, s = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const CacheParams& c = p.c;
    griddep_launch();
    const int sk = __ldg(c.seqused_k + s);
    const int64_t head = (int64_t)s * c.hk + h;
    int32_t* kept = p.kept + head * p.budget;
    const bool bad = sk < 0 || sk > p.max_seqlen_k || (int64_t)sk > (int64_t)c.bt_stride * c.b;
    if (bad && h == 0 && rank == 0 && tid == 0) atomicOr(c.err, (int)UA_DEVERR_BOUNDS);
    const int count = bad ? 0 : min(sk, p.budget);
    const int64_t step = kSel * CL, first = (int64_t)rank * kSel + tid;
    for (int64_t r = count + first; r < p.budget; r += step) kept[r] = -1;
    const float* wi = p.w_in + head * p.w_stride;
    float* wo = p.w_out + head * p.w_stride;
    if (bad || sk <= p.budget) {
        for (int64_t j = first; j < count; j += step) {
            kept[j] = (int32_t)j;
            if (wo != wi) wo[j] = wi[j];
        }
        return;                               // the whole cluster does
    }
    const int n = sk - p.recent;              // candidates
    const uint32_t m = (uint32_t)(p.budget - p.recent);
    // This CTA's run of them, a multiple of the threads long.
    const int run = (n + CL * kSel - 1) / (CL * kSel) * kSel;
    const int lo = min(n, (int)rank * run), hi = min(n, lo + run);
    uint32_t thr = 0;                         // found high bits of the threshold
    uint32_t need = m;                        // keys equal to the threshold to take
    const bool cached = run <= kSelKeys;
    // A thread reads back only what it wrote itself, keys j0 + q * kSel + tid.
    auto load = [&](int j0) {
        float v[kKeep];
#pragma unroll
        for (int q = 0; q < kKeep; ++q) v[q] = j0 + q * kSel + tid < hi ? wi[j0 + q * kSel + tid] : 0.f;
#pragma unroll
        for (int q = 0; q < kKeep; ++q) keep[q * kSel + tid] = v[q];
    };
    if (cached) load(lo);
    for (int i = tid; i < kBins; i += kSel) hist[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 3 && m > 0; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int bits = pass == 2 ? 10 : 11;
        uint2* pair = pairs + (pass & (kPairs<CL> - 1)) * (kBins / 2);
        uint32_t* sum64 = sums[pass & (kPairs<CL> - 1)];
        for (int j0 = lo; j0 < hi; j0 += kSelKeys) {
            if (!cached) load(j0);
#pragma unroll 4
            for (int q = 0; q < kKeep; ++q) {
                const uint32_t k = weight_key(keep[q * kSel + tid]);
                if (j0 + q * kSel + tid < hi && (pass == 0 || (k >> (shift + bits)) == thr))
                    atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
            }
        }
        __syncthreads();
        // Bins 2047 - 2 i and 2046 - 2 i are pair i; a warp has 32 of them at a time.
#pragma unroll
        for (int i = tid; i < kBins / 2; i += kSel) {
            const uint2 v = *reinterpret_cast<const uint2*>(hist + kBins - 2 - 2 * i);
            pair[i] = make_uint2(v.y, v.x);
            const uint32_t sum = __reduce_add_sync(0xffffffffu, v.x + v.y);
            if (lane == 0) sum64[i >> 5] = sum;
        }
        team_sync<CL>();
        if (warp == 0) {
            // Over the cluster: the 64 bins that hold the `need`-th key, then its bin.
            uint32_t v[CL], sum = 0;
#pragma unroll
            for (int q = 0; q < CL; ++q) v[q] = CL == 1 ? sum64[lane] : cluster_word(sum64 + lane, q);
#pragma unroll
            for (int q = 0; q < CL; ++q) sum += v[q];
            uint32_t incl = warp_incl_scan(sum, lane);
            const int at = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
            const uint32_t over = __shfl_sync(0xffffffffu, incl - sum, at);   // keys in higher bins
            uint2 w[CL], c = make_uint2(0, 0);
#pragma unroll
            for (int q = 0; q < CL; ++q) w[q] = CL == 1 ? pair[at * 32 + lane] : cluster_pair(pair + at * 32 + lane, q);
#pragma unroll
            for (int q = 0; q < CL; ++q) {
                c.x += w[q].x;
                c.y += w[q].y;
            }
            incl = over + warp_incl_scan(c.x + c.y, lane);
            const int in = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
            if (lane == in) {
                const uint32_t before = incl - c.x - c.y;
                const bool second = before + c.x < need;
                found[0] = (uint32_t)(kBins - 1 - 2 * (at * 32 + in) - second);
                found[1] = need - before - (second ? c.x : 0u);
            }
        } else if (pass < 2) {
            for (int i = tid - 32; i < kBins; i += kSel - 32) hist[i] = 0;
        }
        __syncthreads();
        thr = (thr << bits) | found[0];
        need = found[1];
    }
    // Kept positions in key order: rank = (keys above) + min(equal ones, need).
    uint32_t above0 = 0, equal0 = 0;          // before this CTA's run, then before the chunk
    if (CL > 1 && m > 0) {
        uint32_t na = 0, ne = 0;
        for (int j0 = lo; j0 < hi; j0 += kSelKeys) {
            if (!cached) load(j0);
#pragma unroll 4
            for (int q = 0; q < kKeep; ++q) {
                const uint32_t k = weight_key(keep[q * kSel + tid]);
                const bool in = j0 + q * kSel + tid < hi;
                na += in && k > thr;
                ne += in && k == thr;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            na += __shfl_xor_sync(0xffffffffu, na, o);
            ne += __shfl_xor_sync(0xffffffffu, ne, o);
        }
        if (tid < 2) mine[tid] = 0;
        __syncthreads();
        if (lane == 0) {
            atomicAdd(&mine[0], na);
            atomicAdd(&mine[1], ne);
        }
    }
    // From here on weights_out may overwrite weights_in; cached weights are in
    // shared memory by now.
    team_sync<CL>();
    if constexpr (CL > 1) {
        if (m > 0 && lane < (int)rank) {
            above0 = cluster_word(&mine[0], lane);
            equal0 = cluster_word(&mine[1], lane);
        }
        above0 = __reduce_add_sync(0xffffffffu, above0);
        equal0 = __reduce_add_sync(0xffffffffu, equal0);
    }
    // A CTA writes at or below its own keys, possibly in an earlier CTA's run:
    // where weights are moved in place and read again, the CTAs take turns.
    const bool turns = CL > 1 && wo == wi && !cached;
    for (int turn = 0; turn < (turns ? CL : 1); ++turn) {
        if (!turns || turn == (int)rank) {
            for (int j0 = lo; m > 0 && j0 < hi; j0 += kSelKeys) {
                if (!cached) load(j0);
                // Counts of every (row of kSel keys, warp), scanned by warp 0 in
                // key order; equal and above packed in one word (8192 at most).
#pragma unroll 4
                for (int q = 0; q < kKeep; ++q) {
                    const uint32_t k = weight_key(keep[q * kSel + tid]);
                    const bool in = j0 + q * kSel + tid < hi;
                    const unsigned ba = __ballot_sync(0xffffffffu, in && k > thr);
                    const unsigned be = __ballot_sync(0xffffffffu, in && k == thr);
                    if (lane == 0) counts[q * (kSel / 32) + warp] = (uint32_t)__popc(ba) << 16 | __popc(be);
                }
                __syncthreads();
                if (warp == 0) {
                    constexpr int kEach = kKeep * (kSel / 32) / 32;
                    uint32_t c0[kEach], sum = 0;
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        c0[e] = sum;
                        sum += counts[lane * kEach + e];
                    }
                    const uint32_t incl = warp_incl_scan(sum, lane);
#pragma unroll
                    for (int e = 0; e < kEach; ++e) counts[lane * kEach + e] = incl - sum + c0[e];
                    if (lane == 31) counts[kKeep * (kSel / 32)] = incl;
                }
                __syncthreads();
#pragma unroll 4
                for (int q = 0; q < kKeep; ++q) {
                    const int j = j0 + q * kSel + tid;
                    const uint32_t k = weight_key(keep[q * kSel + tid]);
                    const bool above = j < hi && k > thr, equal = j < hi && k == thr;
                    const unsigned ba = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
                    const uint32_t before = counts[q * (kSel / 32) + warp];
                    const unsigned lt = (1u << lane) - 1;
                    const uint32_t ra = above0 + (before >> 16) + __popc(ba & lt);
                    const uint32_t re = equal0 + (before & 0xffffu) + __popc(be & lt);
                    if (above || (equal && re < need)) {
                        const uint32_t to = ra + min(re, need);
                        kept[to] = j;
                        wo[to] = keep[q * kSel + tid];
                    }
                }
                const uint32_t all = counts[kKeep * (kSel / 32)];
                above0 += all >> 16;
                equal0 += all & 0xffffu;
                __syncthreads();
            }
            if (rank == CL - 1) {
                // The recent tail; in place a chunk is read before it is written.
                for (int j0 = n; j0 < sk; j0 += kSel) {
                    const int j = j0 + tid;
                    const float w = j < sk ? wi[j] : 0.f;
                    __syncthreads();
                    if (j < sk) {
                        kept[m + (uint32_t)(j - n)] = j;
                        wo[m + (uint32_t)(j - n)] = w;
                    }
                    __syncthreads();
                }
            }
        }
        if (turns) {
            __threadfence();
            cluster_sync_all();
        }
    }
    // No CTA ends while another may still read its shared memory.
    if (CL > 1 && !turns) cluster_sync_all();
}

// Pieces of a row, 16 bytes each; a 4-bit row ends with a piece of d / 16
// scale bytes.  Address of piece `x` of (block, slot, head).
__device__ __forceinline__ uint8_t* piece_at(const CacheParams& c, uint8_t* cache, int64_t block, int slot, int h, int x) {
    if (c.kv_dtype == UA_DTYPE_FP4_E2M1) {
        uint8_t* page = cache + (block * c.hk + h) * fp4_page_bytes(c.b, c.d);
        const int codes = c.d / 2;
        return x * 16 < codes ? page + slot * codes + x * 16 : page + c.b * codes + slot * (c.d / 16);
    }
    const int rb = c.kv_dtype == UA_DTYPE_BF16 ? 2 * c.d : c.d;
    return cache + ((block * c.b + slot) * c.hk + h) * rb + x * 16;
}

// grid: x = rank runs (1 in place) x piece slices x (K, V), y = KV head, z =
// sequence.  A warp has 32 neighbouring ranks of its CTA's 256; slices of `slice`
// pieces of a row go to different CTAs.
__global__ void __launch_bounds__(kMove, 3) move_kernel(const EvictParams p, int pieces, int slice) {
    const CacheParams& c = p.c;
    const int slices = (pieces + slice - 1) / slice;
    const bool v = blockIdx.x & 1;
    const int sl = (blockIdx.x >> 1) % slices, run = (blockIdx.x >> 1) / slices;
    const int h = blockIdx.y, s = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    const int32_t* kept = p.kept + ((int64_t)s * c.hk + h) * p.budget;
    const int32_t* src_table = c.block_table + (int64_t)s * c.bt_stride;
    const int32_t* dst_table = p.dst_table + (int64_t)s * c.bt_stride;
    uint8_t* cache = v ? c.v_cache : c.k_cache;
    const int x0 = sl * slice, nx = min(slice, pieces - x0);
    const uint32_t nx_inv = 0xffffffffu / (uint32_t)nx + 1u;   // e / nx = umulhi(e, nx_inv) for e < 2^16, nx > 1
    const int b_log2 = 31 - __clz(c.b);
    const bool fp4 = c.kv_dtype == UA_DTYPE_FP4_E2M1;
    for (int64_t r0 = (int64_t)run * kRanks; r0 < p.budget; r0 += kRanks) {
        if (kept[r0] < 0) break;
        // Lane = rank: the row's old and new place; j < 0: nothing to move.
        const int64_t r = r0 + warp * 32 + lane;
        int32_t j = r < p.budget ? kept[r] : -1, sb = -1, db = -1;
        if (j >= 0) {
            if (h == 0 && !v && sl == 0 && (r + 1 == p.budget || kept[r + 1] < 0)) p.seqused_out[s] = (int)r + 1;
            if (p.in_place && j == r) {
                j = -1;                       // already there
            } else {
                sb = __ldg(src_table + (j >> b_log2));
                db = __ldg(dst_table + (r >> b_log2));
                if (sb < 0 || (int64_t)sb >= c.num_blocks || db < 0 || (int64_t)db >= c.num_blocks) {
                    atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
                    j = -1;
                }
            }
        }
        // The warp's pieces, row by row, kHold per lane at a time (one turn in
        // place: the launcher's slices see to that).
        for (int i0 = 0; i0 < 32 * nx; i0 += 32 * kHold) {
            uint4 hold[kHold];
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const int e = i0 + k * 32 + lane;
                const int row = nx == 1 ? e : (int)__umulhi((uint32_t)e, nx_inv), x = x0 + e - row * nx;
                const int jj = __shfl_sync(0xffffffffu, j, row & 31), bb = __shfl_sync(0xffffffffu, sb, row & 31);
                if (row >= 32 || jj < 0) continue;
                const uint8_t* src = piece_at(c, cache, bb, jj & (c.b - 1), h, x);
                if (!fp4 || x < pieces - 1 || c.d == 256) hold[k] = *reinterpret_cast<const uint4*>(src);
                else if (c.d == 128) *reinterpret_cast<uint2*>(&hold[k]) = *reinterpret_cast<const uint2*>(src);
                else hold[k].x = *reinterpret_cast<const uint32_t*>(src);
            }
            if (p.in_place) __syncthreads();
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const int e = i0 + k * 32 + lane;
                const int row = nx == 1 ? e : (int)__umulhi((uint32_t)e, nx_inv), x = x0 + e - row * nx;
                const int jj = __shfl_sync(0xffffffffu, j, row & 31), dd = __shfl_sync(0xffffffffu, db, row & 31);
                if (row >= 32 || jj < 0) continue;
                uint8_t* to = piece_at(c, cache, dd, (int)(r0 + warp * 32 + row) & (c.b - 1), h, x);
                if (!fp4 || x < pieces - 1 || c.d == 256) *reinterpret_cast<uint4*>(to) = hold[k];
                else if (c.d == 128) *reinterpret_cast<uint2*>(to) = make_uint2(hold[k].x, hold[k].y);
                else *reinterpret_cast<uint32_t*>(to) = hold[k].x;
            }
        }
        if (!p.in_place) break;               // one round per run
    }
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && kept[0] < 0) p.seqused_out[s] = 0;
}

template <int CL>
cudaError_t launch_select(const EvictParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CL;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.c.hk * CL), (unsigned)p.c.num_seqs);
    cfg.blockDim = dim3(kSelThreads<CL>);
    cfg.dynamicSmemBytes = kSelSmem<CL>;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = CL > 1 ? 1 : 0;
    cudaError_t e = cudaFuncSetAttribute(select_kernel<CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)cfg.dynamicSmemBytes);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, select_kernel<CL>, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
    const CacheParams& c = p.c;
    const int ctas = (p.max_seqlen_k + kSelKeys - 1) / kSelKeys;
    cudaError_t e = ctas <= 1   ? launch_select<1>(p, stream)
                    : ctas <= 2 ? launch_select<2>(p, stream)
                    : ctas <= 4 ? launch_select<4>(p, stream)
                                : launch_select<8>(p, stream);
    if (e != cudaSuccess) return e;
    const int pieces = c.kv_dtype == UA_DTYPE_FP4_E2M1 ? c.d / 32 + 1
                     : c.kv_dtype == UA_DTYPE_BF16     ? c.d / 8
                                                       : c.d / 16;
    // In place one CTA walks all ranks of its slice: a slice's pieces fit one
    // turn of loads, and slices go down to two pieces where there are few
    // (sequence, KV head) pairs.
    int slice = pieces;
    const int64_t base = (int64_t)c.hk * 2 * c.num_seqs;
    if (p.in_place) {
        slice = std::min(slice, kHold);
        while (slice > 2 && base * ((pieces + slice - 1) / slice) < 2LL * num_sms) slice = (slice + 1) / 2;
    }
    const int slices = (pieces + slice - 1) / slice;
    const int64_t n = std::max(1, std::min(p.budget, p.max_seqlen_k));
    const int64_t runs = p.in_place ? 1 : (n + kRanks - 1) / kRanks;
    dim3 grid((unsigned)(runs * slices * 2), (unsigned)c.hk, (unsigned)c.num_seqs);
    return launch_early(move_kernel, grid, kMove, 0, stream, p, pieces, slice);
}

}  // namespace ua
