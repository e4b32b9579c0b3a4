// ua_evict.cu -- eviction by accumulated attention weight: per (sequence, KV
// head) the `budget` kept keys are found (select_kernel) and their cache rows
// moved to the front of the destination table (move_kernel).
//
// Select: one CTA per (sequence, KV head).  A weight's bits, flipped so that
// unsigned order is float order, are searched for the m-th largest of the n
// candidates by three radix passes (11 + 11 + 10 bits) over a shared-memory
// histogram; one pass in key order then writes the kept positions, taking keys
// above the threshold, the first `need` of those equal to it, and the recent
// tail.  Reading the weights four times costs L2 reads only (32 KB for 8192
// keys).  Move: rows in chunks of rank order; a kept key's new position is never
// behind its old one, so an in-place CTA that has read a whole chunk before it
// writes any of it overwrites nothing unread.
#include <algorithm>
#include <cstdint>

#include "ua_cache.h"
#include "ua_fp4.cuh"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kSel = 1024;      // threads of select_kernel
constexpr int kBins = 2048;
constexpr int kMove = 256;      // threads of move_kernel
constexpr int kBatch = 4;       // 16-byte pieces a move thread holds at a time

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

__global__ void __launch_bounds__(kSel) select_kernel(const EvictParams p) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wsum[32], wsum2[32];
    __shared__ uint32_t found[2];
    const int h = blockIdx.x, s = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const CacheParams& c = p.c;
    const int sk = __ldg(c.seqused_k + s);
    const int64_t head = (int64_t)s * c.hk + h;
    int32_t* kept = p.kept + head * p.budget;
    const bool bad = sk < 0 || sk > p.max_seqlen_k || (int64_t)sk > (int64_t)c.bt_stride * c.b;
    if (bad && h == 0 && tid == 0) atomicOr(c.err, (int)UA_DEVERR_BOUNDS);
    const int count = bad ? 0 : min(sk, p.budget);
    for (int64_t r = (int64_t)count + tid; r < p.budget; r += kSel) kept[r] = -1;
    const float* wi = p.w_in + head * p.w_stride;
    float* wo = p.w_out + head * p.w_stride;
    if (bad || sk <= p.budget) {
        for (int j = tid; j < count; j += kSel) {
            kept[j] = j;
            if (wo != wi) wo[j] = wi[j];
        }
        return;
    }
    const int n = sk - p.recent;              // candidates
    uint32_t m = (uint32_t)(p.budget - p.recent);
    uint32_t prefix = 0;                      // found high bits of the threshold
    uint32_t need = 0;                        // keys equal to the threshold to take
    if (m > 0) {
        need = m;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < kBins; i += kSel) hist[i] = 0;
            __syncthreads();
            for (int j = tid; j < n; j += kSel) {
                const uint32_t k = weight_key(wi[j]);
                if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            // Bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t.
            const uint32_t c0 = hist[kBins - 1 - 2 * tid], c1 = hist[kBins - 2 - 2 * tid];
            const uint32_t incl = warp_incl_scan(c0 + c1, lane);
            if (lane == 31) wsum[warp] = incl;
            __syncthreads();
            if (warp == 0) wsum2[lane] = warp_incl_scan(wsum[lane], lane);
            __syncthreads();
            const uint32_t before = (warp ? wsum2[warp - 1] : 0u) + incl - (c0 + c1);   // keys in higher bins
            if (before < need && before + c0 + c1 >= need) {
                const bool first = before + c0 >= need;
                found[0] = (uint32_t)(kBins - 1 - 2 * tid - (first ? 0 : 1));
                found[1] = need - before - (first ? 0u : c0);
            }
            __syncthreads();
            prefix = (prefix << bits) | found[0];
            need = found[1];
            __syncthreads();
        }
    }
    // Kept positions in key order: rank = (keys above) + min(equal ones, need).
    const uint32_t thr = prefix;
    uint32_t above0 = 0, equal0 = 0;          // before this chunk
    for (int j0 = 0; m > 0 && j0 < n; j0 += kSel) {
        const int j = j0 + tid;
        float w = 0.f;
        bool above = false, equal = false;
        if (j < n) {
            w = wi[j];
            const uint32_t k = weight_key(w);
            above = k > thr;
            equal = k == thr;
        }
        const unsigned ba = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
        if (lane == 0) {
            wsum[warp] = __popc(ba);
            wsum2[warp] = __popc(be);
        }
        __syncthreads();
        uint32_t na = 0, ne = 0, ta = 0, te = 0;
        for (int k = 0; k < 32; ++k) {
            if (k == warp) {
                na = ta;
                ne = te;
            }
            ta += wsum[k];
            te += wsum2[k];
        }
        const unsigned lt = (1u << lane) - 1;
        const uint32_t ra = above0 + na + __popc(ba & lt), re = equal0 + ne + __popc(be & lt);
        if (above || (equal && re < need)) {
            const uint32_t rank = ra + min(re, need);
            kept[rank] = j;
            wo[rank] = w;
        }
        above0 += ta;
        equal0 += te;
        __syncthreads();
    }
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

// grid: x = rank chunks (out of place; 1 in place) x piece slices, y = K / V of
// each KV head, z = sequence.
__global__ void __launch_bounds__(kMove) move_kernel(const EvictParams p, int pieces, int slice, int chunk) {
    const CacheParams& c = p.c;
    const int slices = (pieces + slice - 1) / slice;
    const int sl = blockIdx.x % slices, ch = blockIdx.x / slices;
    const int h = blockIdx.y >> 1;
    const bool v = blockIdx.y & 1;
    const int s = blockIdx.z;
    const int32_t* kept = p.kept + ((int64_t)s * c.hk + h) * p.budget;
    const int32_t* st = c.block_table + (int64_t)s * c.bt_stride;
    const int32_t* dt = p.dst_table + (int64_t)s * c.bt_stride;
    uint8_t* cache = v ? c.v_cache : c.k_cache;
    const int x0 = sl * slice, nx = min(slice, pieces - x0);
    const int rows = kMove / slice * kBatch;                 // ranks per round
    const int lane_row = threadIdx.x / slice, lane_x = threadIdx.x % slice;
    const int small = c.kv_dtype == UA_DTYPE_FP4_E2M1 && x0 + lane_x == pieces - 1 ? c.d / 16 : 16;
    const int r_end = (int)min((int64_t)p.budget, ((int64_t)ch + 1) * chunk);
    if (h == 0 && !v && sl == 0) {
        // New length: one past the last kept rank (every sequence has one such
        // rank, or none and length 0).
        for (int r = ch * chunk + threadIdx.x; r < r_end; r += kMove)
            if (kept[r] >= 0 && (r + 1 == p.budget || kept[r + 1] < 0)) p.seqused_out[s] = r + 1;
        if (ch == 0 && threadIdx.x == 0 && kept[0] < 0) p.seqused_out[s] = 0;
    }
    for (int r0 = ch * chunk; r0 < r_end; r0 += rows) {
        if (kept[r0] < 0) return;
        uint4 hold[kBatch];
        uint8_t* to[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = r0 + lane_row + k * (kMove / slice);
            to[k] = nullptr;
            if (lane_row >= kMove / slice || lane_x >= nx || r >= r_end) continue;
            const int j = kept[r];
            if (j < 0 || (p.in_place && j == r)) continue;
            const int32_t sb = __ldg(st + j / c.b), db = __ldg(dt + r / c.b);
            if (sb < 0 || (int64_t)sb >= c.num_blocks || db < 0 || (int64_t)db >= c.num_blocks) {
                atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
                continue;
            }
            const uint8_t* src = piece_at(c, cache, sb, j % c.b, h, x0 + lane_x);
            to[k] = piece_at(c, cache, db, r % c.b, h, x0 + lane_x);
            if (small == 16) hold[k] = *reinterpret_cast<const uint4*>(src);
            else if (small == 8) *reinterpret_cast<uint2*>(&hold[k]) = *reinterpret_cast<const uint2*>(src);
            else hold[k].x = *reinterpret_cast<const uint32_t*>(src);
        }
        if (p.in_place) __syncthreads();
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!to[k]) continue;
            if (small == 16) *reinterpret_cast<uint4*>(to[k]) = hold[k];
            else if (small == 8) *reinterpret_cast<uint2*>(to[k]) = make_uint2(hold[k].x, hold[k].y);
            else *reinterpret_cast<uint32_t*>(to[k]) = hold[k].x;
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
    const CacheParams& c = p.c;
    select_kernel<<<dim3((unsigned)c.hk, (unsigned)c.num_seqs), kSel, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int pieces = c.kv_dtype == UA_DTYPE_FP4_E2M1 ? c.d / 32 + 1
                     : c.kv_dtype == UA_DTYPE_BF16     ? c.d / 8
                                                       : c.d / 16;
    // In place one CTA walks all ranks of its slice; slices down to two pieces
    // keep the SMs busy when there are few (sequence, KV head) pairs.
    int slice = pieces;
    const int64_t base = (int64_t)c.hk * 2 * c.num_seqs;
    if (p.in_place)
        while (slice > 2 && base * ((pieces + slice - 1) / slice) < 2LL * num_sms) slice = (slice + 1) / 2;
    const int slices = (pieces + slice - 1) / slice;
    const int n = std::max(1, std::min(p.budget, p.max_seqlen_k));
    const int chunk = p.in_place ? p.budget : kMove / slice * kBatch;
    const int64_t chunks = p.in_place ? 1 : (n + (int64_t)chunk - 1) / chunk;
    move_kernel<<<dim3((unsigned)(chunks * slices), (unsigned)(c.hk * 2), (unsigned)c.num_seqs), kMove, 0, stream>>>(
        p, pieces, slice, chunk);
    return cudaGetLastError();
}

}  // namespace ua
