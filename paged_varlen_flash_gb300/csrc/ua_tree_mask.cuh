// ua_tree_mask.cuh -- which keys a row of a draft tree sees.
#pragma once

#include <cstdint>

#include "ua_common.cuh"

namespace ua {

// The position of the chunk's key c, within the range that a tree can have.
__device__ __forceinline__ int node_position(const FwdParams& p, int64_t q0, int c, int ctx, int sk) {
    return min(max(p.positions[q0 + c], ctx), sk - 1);
}

// Which of the 32 keys from kb on a row sees (bit e: key kb + e).  lo: the first
// position inside the row's window.
__device__ __forceinline__ uint32_t seen_keys(const FwdParams& p, const uint32_t* row, int64_t q0, int kb, int ctx, int sq,
                                              int sk, int lo) {
    const int c0 = kb - ctx;
    if (c0 >= sq) return 0u;
    uint32_t bits = 0xffffffffu;
    if (c0 > -32) {
        const int w = c0 >> 5;             // -1: the words in front of the chunk are all ones
        const uint32_t a = w < 0 ? 0xffffffffu : row[w];
        const uint32_t b = w + 1 < p.mask_stride ? row[w + 1] : 0u;
        bits = __funnelshift_r(a, b, c0 & 31);
        if (sq - c0 < 32) bits &= (1u << (sq - c0)) - 1u;
    }
    const int low = min(lo, ctx) - kb;     // context keys in front of the window
    if (low > 0) bits &= low >= 32 ? 0u : 0xffffffffu << low;
    if (lo > ctx)                          // a window shorter than the branch
        for (int e = max(0, -c0); e < 32; ++e)
            if ((bits >> e & 1u) && node_position(p, q0, c0 + e, ctx, sk) < lo) bits &= ~(1u << e);
    return bits;
}

}  // namespace ua
