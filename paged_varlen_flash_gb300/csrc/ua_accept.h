// ua_accept.h -- the accepted branch of every draft tree moved behind its context (internal).
#pragma once

#include "ua_cache.h"

namespace ua {

struct AcceptParams {
    CacheParams c;
    const int32_t* cu_seqlens_q;
    const int32_t* parents;         // [num_seqs, parents_stride]
    const int32_t* last;            // [num_seqs] deepest accepted node, -1: none
    int32_t* path;                  // [num_seqs, path_stride]
    int32_t* accepted;              // [num_seqs]
    int32_t* seqused_out;           // [num_seqs], may be seqused_k
    int64_t parents_stride, total_q;
    int32_t path_stride, max_seqlen_q, max_seqlen_k;
};

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t stream);

}  // namespace ua
