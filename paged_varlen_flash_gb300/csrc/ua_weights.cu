// ua_weights.cu -- accumulated attention weight of every cached key.
//
// The attention kernel has stored each row's scores x (log2 units, masks
// applied) and, per KV segment, (m, l).  With M = max m and
// L = sum 2^(m - M) l (the sink joins L like a key), the row's weight on key j
// is 2^(x_j - M - log2 L); a thread owns four keys of one (sequence, KV head)
// and adds those of all its rows in row order: no atomics, one order.  Scores
// instead of a second Q K^T: 8 g bytes per (key, KV head) against the 2 d bytes
// of the key's row, a few rows per KV head at a decode step (64 requests, 250 us
// with the attention, of which 21 here and 6 in the join).  Calls of many rows over
// a 4-bit cache compute the scores again: ua_fp4_weights.cu.
#include <cstdint>

#include "ua_common.cuh"
#include "ua_launch.h"
#include "ua_ptx.cuh"
#include "ua_weights.h"

namespace ua {
namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 4 * kThreads;   // keys per CTA: a thread has four neighbours
constexpr int kAhead = 8;             // rows loaded ahead
constexpr int kBatch = 64;            // rows whose constants are in shared memory at a time

__global__ void __launch_bounds__(kThreads)
weights_kernel(const FwdParams p, const float* in_w, float* out_w, int64_t stride, float decay, bool merged) {
    __shared__ float lse[kBatch];         // log2 of the row's denominator; +inf: a row without weight
    __shared__ int lo[kBatch], hi[kBatch];
    __shared__ int64_t at_row[kBatch];
    const int s = blockIdx.z, hkv = blockIdx.y;
    // After the merge kernel, which writes the statistics, or beside the combine
    // kernel, which only reads them.
    if (merged) griddep_wait();
    int sq, sk;
    int64_t q0;
    const uint32_t st = seq_status(p, s, sq, sk, q0);
    const int64_t first = (int64_t)blockIdx.x * kKeys;
    if (st || sq <= 0 || first >= sk) {
        griddep_wait();
        return;
    }
    const int key = (int)first + threadIdx.x * 4;
    const int ctx = sk - sq, g = p.g;
    const int n = seq_segments(p, st, sk);
    const bool causal = (p.flags & UA_FLAG_CAUSAL) != 0;
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;
    const int64_t rows = (int64_t)g * sq;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t r0 = 0; r0 < rows; r0 += kBatch) {
        const int nb = (int)min((int64_t)kBatch, rows - r0);
        __syncthreads();
        if (threadIdx.x < nb) {
            const int r = (int)(r0 + threadIdx.x), i = r / g;
            const int h = hkv * g + r % g;
            const int64_t row = (q0 + i) * p.hq + h;
            lse[threadIdx.x] = row_lse(p, row, h, n);
            hi[threadIdx.x] = causal ? min(i + ctx, sk - 1) : sk - 1;
            lo[threadIdx.x] = window ? max(0, i + ctx - p.window + 1) : 0;
            at_row[threadIdx.x] = row * p.score_stride;
        }
        __syncthreads();
        if (key >= sk) continue;
        // Eight rows' loads in flight (32 to 128 rows per KV head, 8 sequences of
        // 1000 to 12000 keys: 79 -> 43 us).  Scores are stored for the keys a row sees (and masked
        // ones of the same step); the padded row stride keeps a load of four in
        // bounds.
        for (int k0 = 0; k0 < nb; k0 += kAhead) {
            float4 x[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int k = k0 + q;
                if (k < nb && key <= hi[k] && key + 3 >= lo[k])
                    x[q] = __ldcs(reinterpret_cast<const float4*>(p.scores + at_row[k] + key));
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int k = k0 + q;
                if (k >= nb || key > hi[k] || key + 3 < lo[k] || lse[k] == INFINITY) continue;
                const float v[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key + e >= lo[k] && key + e <= hi[k]) w[e] += fast_exp2(v[e] - lse[k]);
            }
        }
    }
    const int64_t at = ((int64_t)s * p.hk + hkv) * stride + key;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (key + e >= sk) break;
        if (in_w && decay != 0.f && key + e < ctx) w[e] = fmaf(decay, in_w[at + e], w[e]);
        out_w[at + e] = w[e];
    }
    griddep_wait();
}

}  // namespace

cudaError_t launch_weights(const FwdParams& p, const float* in_w, float* out_w, int64_t stride, float decay,
                           bool merged, cudaStream_t stream) {
    dim3 grid((unsigned)((p.max_seqlen_k + (int64_t)kKeys - 1) / kKeys), (unsigned)p.hk, (unsigned)p.num_seqs);
    return launch_early(weights_kernel, grid, kThreads, 0, stream, p, in_w, out_w, stride, decay, merged);
}

}  // namespace ua
