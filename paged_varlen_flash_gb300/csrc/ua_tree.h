// ua_tree.h -- attention for trees of drafted tokens (internal).
#pragma once

#include "ua_common.cuh"

namespace ua {

// An item that begins in a share and is cut by its end: its first partial's slot, the
// number of shares it touches, its rows.
struct TreeJoin {
    int64_t row0;          // first token
    int32_t pieces, slot, nodes, hkv;
};

// The work of a call, cut into equal shares (one per CTA).
struct TreeShares {
    TreeJoin* joins;       // one per share
    int32_t tiles;         // row tiles of the longest chunk
    int32_t slot_rows;     // rows of a partial; share i has slots 2 i and 2 i + 1
    int32_t least;         // steps of a share at least
    int32_t turn;          // steps that an item costs besides its key tiles
};

struct TreePlan {
    int ctas = 0;
    TreeShares shares{};
};

// What a problem's workspace holds for ua_forward_tree at full width.
size_t tree_workspace_bytes(const ua_problem_desc& d, int num_sms);

// Fill *plan and the partials' pointers in *p.  False for g > 128.
bool plan_tree(FwdParams* p, int num_sms, void* workspace, size_t workspace_bytes, TreePlan* plan);

cudaError_t launch_tree(const TreePlan& plan, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const FwdParams& p,
                        cudaStream_t stream);

}  // namespace ua
