// ua_accept.cu -- the rows of a draft tree's accepted branch moved to the positions
// right behind the context.
//
// With the branch r_0 < r_1 < ... (node numbers from the root on), row r_t moves to
// position ctx + t.  A parent stands in front of its children, so r_t >= t: in ascending
// t a row is always read before a move overwrites it.  A thread owns one 16-byte column
// (4 bytes in the 4-bit format, whose scale rows are that short) of the rows of all
// heads and walks up t by itself, a few loads ahead of the stores, so that no two
// threads touch the same bytes and nothing waits for a neighbour.
//
// One CTA per sequence; bound by launch and load latency (parents, block ids, rows):
// 64 trees of up to 32 nodes, 8 heads of 128: 3.1 us a call in a row of them; 256
// trees, 8 heads of 256: 4.2 us.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ua_accept.h"
#include "ua_fp4.cuh"
#include "ua_launch.h"
#include "ua_plan.h"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kAhead = 8;

template <bool FP4>
__global__ void __launch_bounds__(1024) accept_kernel(const AcceptParams p) {
    using Word = typename std::conditional<FP4, uint32_t, uint4>::type;
    __shared__ int32_t node[kMaxTree];     // parents, then the branch's node numbers from the root on
    __shared__ int64_t from[kMaxTree], to[kMaxTree];    // block * b + slot; from < 0: stays
    __shared__ int len, start;
    const CacheParams& c = p.c;
    const int s = blockIdx.x, tid = threadIdx.x, b_log2 = 31 - __clz(c.b);
    griddep_wait();
    const int32_t a = p.cu_seqlens_q[s], z = p.cu_seqlens_q[s + 1];
    const int32_t sk = c.seqused_k[s], last = p.last[s];
    const int sq = z - a;
    uint32_t st = 0;
    if (a < 0 || z < a || (int64_t)z > p.total_q) {
        st = UA_DEVERR_CU_SEQLENS;
    } else {
        if (sk < sq) st |= UA_DEVERR_CONTEXT;
        if (sq > p.max_seqlen_q || sk > p.max_seqlen_k || (int64_t)sk > (int64_t)c.bt_stride * c.b)
            st |= UA_DEVERR_BOUNDS;
    }
    // Without query rows nothing was drafted, and `last` says nothing.
    const bool tree = last >= -1 && last < sq;
    const int up = st || sq == 0 || !tree ? -1 : last;
    for (int i = tid; i <= up; i += blockDim.x) node[i] = p.parents[(int64_t)s * p.parents_stride + i];
    __syncthreads();
    if (tid == 0) {
        // The branch from its end on, packed at the upper end of the nodes passed: the
        // walk's next node is always below where it writes.
        int at = up, w = up;
        uint32_t bad = st ? st : sq > 0 && !tree ? (uint32_t)UA_DEVERR_TREE : 0u;
        while (at >= 0) {
            const int q = node[at];
            node[w--] = at;
            if (q < -1 || q >= at) {
                bad |= UA_DEVERR_TREE;
                w = up;
                break;
            }
            at = q;
        }
        if (up - w > p.path_stride) {
            bad |= UA_DEVERR_BOUNDS;
            w = up;
        }
        start = w + 1;
        len = up - w;
        if (bad) atomicOr(c.err, (int)bad);
    }
    __syncthreads();
    const int n = len, base = start, ctx = sk - sq;
    const int32_t* table = c.block_table + (int64_t)s * c.bt_stride;
    for (int t = tid; t < n; t += blockDim.x) {
        const int r = node[base + t];
        from[t] = -1;
        if (r == t) continue;
        const int32_t x = table[((ctx + r) >> b_log2)], y = table[((ctx + t) >> b_log2)];
        if (x < 0 || y < 0 || (int64_t)x >= c.num_blocks || (int64_t)y >= c.num_blocks) {
            atomicOr(c.err, (int)UA_DEVERR_BLOCK_ID);
            continue;
        }
        from[t] = (int64_t)x * c.b + ((ctx + r) & (c.b - 1));
        to[t] = (int64_t)y * c.b + ((ctx + t) & (c.b - 1));
    }
    for (int t = tid; t < p.path_stride; t += blockDim.x) p.path[(int64_t)s * p.path_stride + t] = t < n ? node[base + t] : -1;
    if (tid == 0) {
        p.accepted[s] = n;
        // (Every thread has read seqused_k before the barriers above.)
        p.seqused_out[s] = st ? 0 : ctx + n;
    }
    __syncthreads();
    if (n == 0) return;
    // Columns of a token's rows: K's, then V's.
    const int d = c.d, head_words = FP4 ? (d / 2 + d / 16) / 4 : 0;
    const int cols = FP4 ? c.hk * head_words : c.hk * d * (c.kv_dtype == UA_DTYPE_BF16 ? 2 : 1) / 16;
    for (int64_t col = tid; col < 2 * (int64_t)cols; col += blockDim.x) {
        const int x = (int)(col < cols ? col : col - cols);
        uint8_t* cache = col < cols ? c.k_cache : c.v_cache;
        auto addr = [&](int64_t row) -> Word* {
            if constexpr (FP4) {
                const int h = x / head_words, w = x % head_words, codes = d / 8;
                const int slot = (int)(row & (c.b - 1));
                uint8_t* page = cache + ((row >> b_log2) * c.hk + h) * fp4_page_bytes(c.b, d);
                return reinterpret_cast<Word*>(w < codes ? page + slot * (d / 2) + w * 4
                                                         : page + c.b * (d / 2) + slot * (d / 16) + (w - codes) * 4);
            } else {
                return reinterpret_cast<Word*>(cache) + row * cols + x;
            }
        };
        for (int t0 = 0; t0 < n; t0 += kAhead) {
            Word v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (t0 + k < n && from[t0 + k] >= 0) v[k] = *addr(from[t0 + k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (t0 + k < n && from[t0 + k] >= 0) *addr(to[t0 + k]) = v[k];
        }
    }
}

}  // namespace

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t stream) {
    const bool fp4 = p.c.kv_dtype == UA_DTYPE_FP4_E2M1;
    const int64_t cols = 2LL * p.c.hk * (fp4 ? (p.c.d / 2 + p.c.d / 16) / 4
                                             : p.c.d * (p.c.kv_dtype == UA_DTYPE_BF16 ? 2 : 1) / 16);
    const int threads = (int)std::min<int64_t>(1024, std::max<int64_t>(64, (cols + 31) / 32 * 32));
    return launch_early(fp4 ? accept_kernel<true> : accept_kernel<false>, dim3((unsigned)p.c.num_seqs), threads, 0, stream, p);
}

}  // namespace ua
