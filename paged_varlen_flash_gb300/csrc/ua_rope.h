// ua_rope.h -- rotary positions and the store of the rotated keys (internal).
#pragma once

#include <cstdint>

#include "ua_cache.h"

namespace ua {

constexpr int kMaxFreq = 128;       // rotated pairs of a head (d / 2 at most)

// Angle per position of every pair, as a fraction of a turn times 2^64.  Passed to
// the kernel by value: a captured call keeps the frequencies that it was made with.
struct RopeTable {
    uint64_t turn[kMaxFreq];
    int32_t n;                      // pairs; dims from 2 n on are not rotated
    int32_t pairs;                  // 1: dims (2i, 2i + 1), 0: dims (i, i + n)
    float magnitude;                // factor of cos and sin
};

struct RopeParams {
    CacheParams c;
    const __nv_bfloat16* q;         // token rows, q_stride elements apart
    const __nv_bfloat16* k_new;     // token rows, kv_stride elements apart
    const __nv_bfloat16* v_new;
    __nv_bfloat16* q_out;           // token rows, out_stride elements apart
    const int32_t* positions;       // [total_q]
    const int64_t* slots;           // [total_q], block * b + slot; below 0: not stored
    int64_t q_stride, kv_stride, out_stride, total_q;
    int32_t hq;
};

cudaError_t launch_rope_store(const RopeParams& p, const RopeTable& t, cudaStream_t stream);

}  // namespace ua
