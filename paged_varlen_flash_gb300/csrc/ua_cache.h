// ua_cache.h -- cache operators besides attention: store, expand, evict (internal).
#pragma once

#include "ua_common.cuh"

namespace ua {

// One paged cache format and one call's batch.
struct CacheParams {
    uint8_t* k_cache;
    uint8_t* v_cache;
    const int32_t* block_table;    // [num_seqs, bt_stride]
    const int32_t* seqused_k;      // [num_seqs]
    int32_t* err;                  // device error word
    int64_t num_blocks;
    int32_t num_seqs, bt_stride, hk, d, b;
    int32_t kv_dtype;              // UA_DTYPE_*
    float k_scale, v_scale;
};

struct StoreParams {
    CacheParams c;
    const __nv_bfloat16* k_new;    // token rows, `stride` elements apart
    const __nv_bfloat16* v_new;
    const int32_t* cu_seqlens_q;
    int64_t stride, total_q;
    int32_t max_seqlen_q, max_seqlen_k;
};

struct ExpandParams {
    CacheParams c;
    const int32_t* begin;          // [num_seqs] or null (0)
    __nv_bfloat16* k_out;          // [out_blocks, b, hk, d]
    __nv_bfloat16* v_out;
    const int32_t* out_table;      // [num_seqs, out_stride]
    int64_t out_blocks;
    int32_t out_stride, max_keys;
};

struct EvictParams {
    CacheParams c;
    const int32_t* dst_table;      // [num_seqs, bt_stride]
    const float* w_in;             // [num_seqs, hk, w_stride]
    float* w_out;
    int32_t* kept;                 // [num_seqs, hk, budget]
    int32_t* seqused_out;
    int64_t w_stride;
    int32_t max_seqlen_k, budget, recent;
    int32_t in_place;              // dst_table is block_table
};

cudaError_t launch_store(const StoreParams& p, cudaStream_t stream);
cudaError_t launch_expand(const ExpandParams& p, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream);

}  // namespace ua
