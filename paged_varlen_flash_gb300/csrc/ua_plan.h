// ua_plan.h -- blocks, slots, positions and ancestor masks of a step (internal).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace ua {

constexpr int kMaxTree = 1024;      // nodes of a draft tree
constexpr int kMaxPlanSeqs = 16384; // prefix sums of all sequences fit a CTA's shared memory

struct PlanParams {
    int32_t* block_table;          // [num_seqs, bt_stride]
    int32_t* held;                 // [num_seqs] blocks of every sequence
    int32_t* pool;                 // free blocks, a stack of *pool_count
    int32_t* pool_count;
    const int32_t* ctx_lens;       // [num_seqs]
    const int32_t* new_lens;       // [num_seqs]
    const int32_t* parents;        // [num_seqs, parents_stride] or null (chains)
    int32_t* granted;              // [num_seqs]
    int32_t* cu;                   // [num_seqs + 1]
    int32_t* used;                 // [num_seqs], may be ctx_lens
    int32_t* positions;            // [max_tokens]
    int64_t* slots;                // [max_tokens]
    uint32_t* mask;                // [max_tokens, mask_stride] or null
    int32_t* err;                  // device error word
    int32_t* ticket;               // CTAs that are done, 0 between calls
    int64_t parents_stride;
    int64_t num_blocks;
    int64_t max_tokens;
    int32_t mask_stride;
    int32_t num_seqs, bt_stride, b_log2;
    int32_t aligned;               // positions and slots on 16-byte boundaries
};

cudaError_t launch_plan(const PlanParams& p, int num_sms, cudaStream_t stream);

}  // namespace ua
