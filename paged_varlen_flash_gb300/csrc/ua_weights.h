// ua_weights.h -- launcher of the key-weight accumulation (internal).
#pragma once

#include "ua_common.cuh"
#include "ua_ptx.cuh"

namespace ua {

// out_w = decay * in_w (keys of the context) + the rows' softmax weights, from
// the scores in p.scores and the segment statistics in p.part_ml.  in_w may be
// null (zeros) or out_w itself; rows of `stride` floats per (sequence, KV head).
// Runs beside the combine kernel in front of it or, `merged`, after the merge kernel.
cudaError_t launch_weights(const FwdParams& p, const float* in_w, float* out_w, int64_t stride, float decay,
                           bool merged, cudaStream_t stream);

// The same for a 4-bit cache and calls of the tcgen05 attention kernel: scores
// are computed again (p.scores is not read).  Runs beside the combine kernel.
cudaError_t launch_fp4_weights(const FwdParams& p, int num_sms, const float* in_w, float* out_w, int64_t stride,
                               float decay, cudaStream_t stream);

// log2 of the denominator of a row (query head h) from its n segments' (m, l),
// the sink joined like a key: 2^(x - lse) is the weight of a key with score x.
// +inf for a row without weight.
__device__ __forceinline__ float row_lse(const FwdParams& p, int64_t row, int h, int n) {
    const float* ml = p.part_ml + row * p.splits * 2;
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
    return M == -INFINITY || L == INFINITY || L == 0.f ? INFINITY : M + log2f(L);
}

}  // namespace ua
