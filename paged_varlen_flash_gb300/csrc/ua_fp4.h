// ua_fp4.h -- launcher of the attention kernel over 4-bit (e2m1) caches (internal).
#pragma once

#include "ua_common.cuh"

namespace ua {

struct Fp4Plan {
    int rows = 16;      // packed rows per tile (8 or 16)
    int splits = 1;     // KV segments per (sequence, kv head, row tile)
    int chunk = 0;      // keys per segment (a multiple of 128)
    int row_tiles = 1;  // row tiles per (sequence, kv head)
    int launches = 0;   // kernels enqueued per call (the combine among them)
};

// False when the call's grid does not fit.
bool plan_fp4(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4Plan* plan);

// Enqueue the kernel (p.splits / p.chunk / p.row_tiles / partial pointers set
// from the plan).  With p.scores set every row's scores are stored as well and
// partials are written even for one segment.
cudaError_t launch_fp4(const Fp4Plan& plan, const FwdParams& p, cudaStream_t stream);

}  // namespace ua
