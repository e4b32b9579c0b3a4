// ua_weights.cu -- accumulated attention weight of every cached key.
//
// The attention kernel has stored each row's scores x (log2 units, masks
// applied) and, per KV segment, (m, l).  With M = max m and
// L = sum 2^(m - M) l (the sink joins L like a key), the row's weight on key j
// is 2^(x_j - M - log2 L); a thread owns one key of one (sequence, KV head)
// and adds those of all its rows in row order: no atomics, one order.  Scores
// instead of a second Q K^T: 8 g bytes per (key, KV head) against the 2 d bytes
// of the key's row.
#include <cstdint>

#include "ua_common.cuh"
#include "ua_ptx.cuh"
#include "ua_weights.h"

namespace ua {
namespace {

constexpr int kKeys = 256;   // keys (threads) per CTA
constexpr int kBatch = 64;   // rows whose normalisers are in shared memory at a time

__global__ void __launch_bounds__(kKeys)
weights_kernel(const FwdParams p, const float* in_w, float* out_w, int64_t stride, float decay) {
    __shared__ float lse[kBatch];
    const int s = blockIdx.z, hkv = blockIdx.y;
    int sq, sk;
    int64_t q0;
    const uint32_t st = seq_status(p, s, sq, sk, q0);
    const int64_t key0 = (int64_t)blockIdx.x * kKeys;
    if (st || sq <= 0 || key0 >= sk) return;
    const int key = (int)key0 + threadIdx.x;
    const int ctx = sk - sq, g = p.g;
    const int n = seq_segments(p, st, sk);
    const bool causal = (p.flags & UA_FLAG_CAUSAL) != 0;
    const bool window = (p.flags & UA_FLAG_WINDOW) != 0;
    const int64_t rows = (int64_t)g * sq;
    float w = 0.f;
    for (int64_t r0 = 0; r0 < rows; r0 += kBatch) {
        const int nb = (int)min((int64_t)kBatch, rows - r0);
        __syncthreads();
        if (threadIdx.x < nb) {
            const int64_t r = r0 + threadIdx.x;
            const int h = hkv * g + (int)(r % g);
            const float* ml = p.part_ml + ((q0 + r / g) * p.hq + h) * p.splits * 2;
            float M = -INFINITY, L = 0.f;
            for (int k = 0; k < n; ++k) M = fmaxf(M, ml[2 * k]);
            if (M != -INFINITY)
                for (int k = 0; k < n; ++k) L = fmaf(fast_exp2(ml[2 * k] - M), ml[2 * k + 1], L);
            if (p.flags & UA_FLAG_SINKS) {
                const float s2 = __ldg(p.sinks + h) * kLog2e;
                if (s2 == INFINITY) {
                    L = INFINITY;                 // the sink takes the whole row
                } else if (s2 > M) {
                    L = (M == -INFINITY ? 0.f : L * fast_exp2(M - s2)) + 1.f;
                    M = s2;
                } else if (s2 != -INFINITY) {
                    L += fast_exp2(s2 - M);
                }
            }
            // +inf: a row without weight (no visible key, or an infinite sink).
            lse[threadIdx.x] = (M == -INFINITY || L == INFINITY || L == 0.f) ? INFINITY : M + log2f(L);
        }
        __syncthreads();
        if (key < sk)
            for (int k = 0; k < nb; ++k) {
                const int64_t r = r0 + k;
                const int i = (int)(r / g);
                const int hi = causal ? min(i + ctx, sk - 1) : sk - 1;
                const int lo = window ? max(0, i + ctx - p.window + 1) : 0;
                if (key < lo || key > hi) continue;
                const float x = p.scores[((q0 + i) * p.hq + (int64_t)hkv * g + r % g) * p.score_stride + key];
                w += lse[k] == INFINITY ? 0.f : fast_exp2(x - lse[k]);
            }
    }
    if (key >= sk) return;
    const int64_t at = ((int64_t)s * p.hk + hkv) * stride + key;
    if (in_w && decay != 0.f && key < ctx) w = fmaf(decay, in_w[at], w);
    out_w[at] = w;
}

}  // namespace

cudaError_t launch_weights(const FwdParams& p, const float* in_w, float* out_w, int64_t stride, float decay,
                           cudaStream_t stream) {
    dim3 grid((unsigned)((p.max_seqlen_k + kKeys - 1) / kKeys), (unsigned)p.hk, (unsigned)p.num_seqs);
    weights_kernel<<<grid, kKeys, 0, stream>>>(p, in_w, out_w, stride, decay);
    return cudaGetLastError();
}

}  // namespace ua
