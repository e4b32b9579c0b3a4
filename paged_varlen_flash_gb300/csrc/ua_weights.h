// ua_weights.h -- launcher of the key-weight accumulation (internal).
#pragma once

#include "ua_common.cuh"

namespace ua {

// out_w = decay * in_w (keys of the context) + the rows' softmax weights, from
// the scores in p.scores and the segment statistics in p.part_ml.  in_w may be
// null (zeros) or out_w itself; rows of `stride` floats per (sequence, KV head).
cudaError_t launch_weights(const FwdParams& p, const float* in_w, float* out_w, int64_t stride, float decay,
                           cudaStream_t stream);

}  // namespace ua
