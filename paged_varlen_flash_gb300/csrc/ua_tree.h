// ua_tree.h -- attention for trees of drafted tokens (internal).
#pragma once

#include "ua_common.cuh"

namespace ua {

struct TreePlan {
    int tiles = 0;         // row tiles per (sequence, KV head)
    int splits = 1;        // KV segments
    int chunk = 0;         // keys per segment
};

// Rows of a tile hold whole groups: g <= 128.
bool plan_tree(const FwdParams& p, int num_sms, size_t workspace_bytes, TreePlan* plan);

cudaError_t launch_tree(const TreePlan& plan, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const FwdParams& p,
                        cudaStream_t stream);

}  // namespace ua
