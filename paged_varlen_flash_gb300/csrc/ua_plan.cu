// ua_plan.cu -- block tables, slots, positions and ancestor masks of a step, from the
// requests' lengths and a pool of free blocks.
//
// A sequence needs ceil((ctx + new) / b) blocks.  Those that hold more give the last
// ones back; those that hold fewer take the difference from the pool, in their order,
// as long as the running demand is covered.  With T blocks taken and R returned, and
// the pool a stack of n blocks, taken block k (counted over the sequences) is
//     returned block k          for k < R,
//     pool[n + R - 1 - k]       otherwise,
// and the returned blocks from T on stay, block r at pool[n + R - 1 - r]: the returned
// blocks lie on the stack with the first one on top.  (A step that is taken back leaves
// the pool as it was.)  So every id follows from prefix sums over the sequences, and no
// write of the call touches a pool entry that it reads.
//
// Every CTA computes the prefix sums itself (12 bytes a sequence, from L2), then takes
// its share of the tokens, the taken blocks and the returned ones; the last CTA to finish
// writes what replaces an input (held, pool_count, used), when nobody reads it any more.
//
// Bound by latency: 64 sequences of one token 5.0 us a call in a row of them (two rounds of
// loads, the prefix sums' barriers, the last CTA's ticket; 8.2 when the CTAs started behind
// the kernel in front).  128 prompts of 1.08 million tokens in all and the way back: 22 us
// for the two calls, 12 bytes written per token.
#include <algorithm>
#include <cstdint>

#include "../../include/ua.h"
#include "ua_launch.h"
#include "ua_plan.h"
#include "ua_ptx.cuh"

namespace ua {
namespace {

constexpr int kThreads = 1024;     // at most
constexpr int kFew = 256;          // threads of a CTA where they hold all sequences

struct Sums {          // of the sequences in front of a thread's, or of all
    int64_t a, b, c;
};

// Exclusive prefix over the CTA's threads; *total gets the sum.
__device__ __forceinline__ Sums prefix(Sums v, Sums* warp_sums, Sums* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, x.a, o), b = __shfl_up_sync(0xffffffffu, x.b, o),
                      c = __shfl_up_sync(0xffffffffu, x.c, o);
        if (lane >= o) {
            x.a += a;
            x.b += b;
            x.c += c;
        }
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    Sums before{0, 0, 0}, all{0, 0, 0};
    const int warps = blockDim.x >> 5;
    for (int w = 0; w < warps; ++w) {
        const Sums y = warp_sums[w];
        if (w < warp) {
            before.a += y.a;
            before.b += y.b;
            before.c += y.c;
        }
        all.a += y.a;
        all.b += y.b;
        all.c += y.c;
    }
    *total = all;
    return {before.a + x.a - v.a, before.b + x.b - v.b, before.c + x.c - v.c};
}

// What a sequence asks for.  Malformed lengths ask for nothing and give nothing back.
struct Ask {
    int ctx, fresh, held, more, back;
    bool bad;
};

__device__ __forceinline__ Ask ask_of(const PlanParams& p, int s) {
    Ask a{p.ctx_lens[s], p.new_lens[s], p.held[s], 0, 0, false};
    const int64_t end = (int64_t)a.ctx + a.fresh;
    a.bad = a.ctx < 0 || a.fresh < 0 || a.held < 0 || a.held > p.bt_stride || end > (int64_t)p.bt_stride << p.b_log2 ||
            (p.parents && a.fresh > p.parents_stride) || (p.mask && (int64_t)a.fresh > 32LL * p.mask_stride);
    if (a.bad) {
        a.ctx = a.fresh = 0;
        return a;
    }
    const int need = (int)((end + (1 << p.b_log2) - 1) >> p.b_log2);
    a.more = max(need - a.held, 0);
    a.back = max(a.held - need, 0);
    return a;
}

// Last s with first[s] <= x (first[0] = 0, x < first[n]).
__device__ __forceinline__ int owner_of(const int32_t* first, int n, int32_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The slot of sequence s's key `place`; -1 and an error bit for a bad block id.
template <typename Taken>
__device__ __forceinline__ int64_t slot_of(const PlanParams& p, const int32_t* take, const Taken& taken, int s, int place,
                                           uint32_t& err) {
    const int blk = place >> p.b_log2, held = p.held[s];
    const int32_t id = blk < held ? p.block_table[(int64_t)s * p.bt_stride + blk] : taken(take[s] + blk - held);
    if (id < 0 || (int64_t)id >= p.num_blocks) {
        err |= UA_DEVERR_BLOCK_ID;
        return -1;
    }
    return ((int64_t)id << p.b_log2) + (place & ((1 << p.b_log2) - 1));
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanParams p) {
    extern __shared__ int32_t smem[];
    __shared__ Sums warp_sums[2][kThreads / 32];
    __shared__ int last;
    const int n = p.num_seqs, tid = threadIdx.x, threads = blockDim.x;
    int32_t* tok = smem;             // tokens in front of a sequence
    int32_t* take = tok + n + 1;     // blocks taken in front of it
    int32_t* give = take + n + 1;    // blocks returned in front of it
    const int per = (n + threads - 1) / threads;
    griddep_wait();
    const int s0 = min(n, tid * per), s1 = min(n, s0 + per);
    int64_t count = *p.pool_count;

    // 1. What is asked for, and which sequences get it.  (A thread's first sequence stays in
    // registers; only batches of more sequences than threads have others.)
    Ask own{0, 0, 0, 0, 0, false};
    if (s0 < s1) own = ask_of(p, s0);
    auto ask = [&](int s) { return s == s0 ? own : ask_of(p, s); };
    Sums mine{0, 0, 0}, all;
    uint32_t err = 0;
    for (int s = s0; s < s1; ++s) {
        const Ask a = ask(s);
        if (a.bad) err |= UA_DEVERR_BOUNDS;
        mine.a += a.more;
        mine.b += a.back;
        mine.c += a.fresh;
    }
    const Sums before = prefix(mine, warp_sums[0], &all);
    // A pool of another size than the cache's, or more blocks given back than there are:
    // nothing is taken or nothing is given back.
    const bool sane = count >= 0 && count <= p.num_blocks;
    const bool returns = sane && count + all.b <= p.num_blocks;
    if (!sane) count = 0;
    if (!returns) err |= UA_DEVERR_POOL;
    const int64_t R = returns ? all.b : 0;
    // 2. Prefix sums of what is given out.  Places are asked for by the sequences that the
    // pool serves.  (Where it serves all of them, or there are places for all tokens, the sums
    // above will do: the same for the whole CTA.)
    const bool dry = all.a > count + R && all.c > p.max_tokens;
    int64_t fresh_before = before.c;
    if (dry) {
        Sums served{0, 0, 0}, unused;
        int64_t more = before.a;
        for (int s = s0; s < s1; ++s) {
            const Ask a = ask(s);
            more += a.more;
            if (a.more == 0 || more <= count + R) served.c += a.fresh;
        }
        fresh_before = prefix(served, warp_sums[1], &unused).c;
    }
    Sums got{0, 0, 0}, sum;
    auto each = [&](auto&& f) {
        int64_t more = before.a, fresh = fresh_before;
        for (int s = s0; s < s1; ++s) {
            const Ask a = ask(s);
            more += a.more;
            const bool served = a.more == 0 || more <= count + R;
            if (served) fresh += a.fresh;
            const bool fits = fresh <= p.max_tokens, ok = fits && served;
            if (served && !fits && a.fresh) err |= UA_DEVERR_BOUNDS;
            f(s, ok ? a.more : 0, returns ? a.back : 0, ok ? a.fresh : 0);
        }
    };
    each([&](int, int more, int back, int fresh) {
        got.a += more;
        got.b += back;
        got.c += fresh;
    });
    // (Every thread is past the first sums when the second ones have been joined.)
    Sums at = prefix(got, warp_sums[dry ? 0 : 1], &sum);
    each([&](int s, int more, int back, int fresh) {
        take[s] = (int32_t)at.a;
        give[s] = (int32_t)at.b;
        tok[s] = (int32_t)at.c;
        at.a += more;
        at.b += back;
        at.c += fresh;
    });
    if (tid == 0) {
        take[n] = (int32_t)sum.a;
        give[n] = (int32_t)sum.b;
        tok[n] = (int32_t)sum.c;
    }
    __syncthreads();
    const int T = (int)sum.a, total = (int)sum.c;
    const int64_t first = (int64_t)blockIdx.x * threads + tid, step = (int64_t)gridDim.x * threads;

    auto returned = [&](int r) -> int32_t {
        const int s = owner_of(give, n, r);
        const int keep = p.held[s] - (give[s + 1] - give[s]);
        return p.block_table[(int64_t)s * p.bt_stride + keep + (r - give[s])];
    };
    auto taken = [&](int k) -> int32_t { return k < R ? returned(k) : p.pool[count + R - 1 - k]; };

    // 3. Taken blocks into the tables, returned ones that nobody took onto the pool.
    for (int64_t k = first; k < T; k += step) {
        const int s = owner_of(take, n, (int)k);
        const int32_t id = taken((int)k);
        if (id < 0 || (int64_t)id >= p.num_blocks) err |= UA_DEVERR_BLOCK_ID;
        p.block_table[(int64_t)s * p.bt_stride + p.held[s] + ((int)k - take[s])] = id;
    }
    for (int64_t r = T + first; r < R; r += step) {
        const int32_t id = returned((int)r);
        if (id < 0 || (int64_t)id >= p.num_blocks) err |= UA_DEVERR_BLOCK_ID;
        p.pool[count + R - 1 - r] = id;
    }

    // 4. Tokens.  Chains without a mask four at a time, which nearly always are neighbours
    // in one block.
    const bool fours = !p.parents && !p.mask && p.aligned;
    if (fours) {
        for (int64_t t = 4 * first; t < p.max_tokens; t += 4 * step) {
            int pos[4];
            int64_t slot[4];
            const int s = t < total ? owner_of(tok, n, (int)t) : 0;
            const int place = t < total ? p.ctx_lens[s] + ((int)t - tok[s]) : 0;
            if (t < total && t + 3 < tok[s + 1] && (place & ((1 << p.b_log2) - 1)) <= (1 << p.b_log2) - 4) {
                const int64_t at_slot = slot_of(p, take, taken, s, place, err);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    pos[k] = place + k;
                    slot[k] = at_slot < 0 ? -1 : at_slot + k;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    pos[k] = 0;
                    slot[k] = -1;
                    if (t + k >= total) continue;
                    const int sk = owner_of(tok, n, (int)t + k);
                    pos[k] = p.ctx_lens[sk] + ((int)t + k - tok[sk]);
                    slot[k] = slot_of(p, take, taken, sk, pos[k], err);
                }
            }
            if (t + 3 < p.max_tokens) {
                *reinterpret_cast<int4*>(p.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
                *reinterpret_cast<longlong2*>(p.slots + t) = make_longlong2(slot[0], slot[1]);
                *reinterpret_cast<longlong2*>(p.slots + t + 2) = make_longlong2(slot[2], slot[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (t + k < p.max_tokens) {
                        p.positions[t + k] = pos[k];
                        p.slots[t + k] = slot[k];
                    }
            }
        }
    }
    for (int64_t t = first; !fours && t < p.max_tokens; t += step) {
        if (t >= total) {
            p.positions[t] = 0;
            p.slots[t] = -1;
            continue;
        }
        const int s = owner_of(tok, n, (int)t);
        const int i = (int)t - tok[s], ctx = p.ctx_lens[s];
        p.slots[t] = slot_of(p, take, taken, s, ctx + i, err);
        int depth = i;
        if (p.parents) {
            // Up to the root; the bits of a word of the mask are complete when the
            // walk leaves it, since parents stand in front of their children.
            const int32_t* up = p.parents + (int64_t)s * p.parents_stride;
            uint32_t* row = p.mask ? p.mask + t * p.mask_stride : nullptr;
            int w = p.mask_stride - 1, node = i;
            uint32_t bits = 0;
            depth = -1;
            while (node >= 0) {
                if (row) {
                    for (; w > node >> 5; --w) {
                        row[w] = bits;
                        bits = 0;
                    }
                    bits |= 1u << (node & 31);
                }
                ++depth;
                const int q = up[node];
                if (q < -1 || q >= node) {
                    err |= UA_DEVERR_TREE;
                    break;
                }
                node = q;
            }
            if (row)
                for (; w >= 0; --w) {
                    row[w] = bits;
                    bits = 0;
                }
        } else if (p.mask) {
            for (int w = 0; w < p.mask_stride; ++w) {
                const int over = i + 1 - 32 * w;
                p.mask[t * p.mask_stride + w] = over >= 32 ? 0xffffffffu : over > 0 ? (1u << over) - 1 : 0u;
            }
        }
        p.positions[t] = ctx + depth;
    }
    if (err) atomicOr(p.err, (int)err);

    // 5. The last CTA replaces the state.
    if (gridDim.x > 1) {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            last = atomicAdd(p.ticket, 1) == (int)gridDim.x - 1;
        }
        __syncthreads();
        if (!last) return;
        __threadfence();
        if (tid == 0) *p.ticket = 0;
    } else {
        __syncthreads();
    }
    for (int s = tid; s < n; s += threads) {
        const Ask a = s == s0 && per == 1 ? own : ask_of(p, s);
        const int fresh = tok[s + 1] - tok[s];
        p.granted[s] = fresh;
        p.cu[s] = tok[s];
        p.used[s] = a.ctx + fresh;
        if (!a.bad) p.held[s] = a.held + (take[s + 1] - take[s]) - (give[s + 1] - give[s]);
    }
    if (tid == 0) {
        p.cu[n] = total;
        if (sane) *p.pool_count = (int32_t)(count + R - T);
    }
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, int num_sms, cudaStream_t stream) {
    const size_t smem = (size_t)3 * (p.num_seqs + 1) * sizeof(int32_t);
    if (smem > 48 * 1024 - 2048) {
        const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    // Few sequences: smaller CTAs, whose sums are quicker, and more of them.
    const int threads = p.num_seqs <= kFew ? kFew : kThreads;
    const int64_t each = (p.parents || p.mask ? 1 : 4) * (int64_t)threads;
    const int64_t most = (int64_t)num_sms * (threads == kFew ? 4 : 1);
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(most, (p.max_tokens + each - 1) / each));
    PlanParams q = p;
    q.aligned = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15u) == 0;
    return launch_early(plan_kernel, dim3((unsigned)ctas), threads, smem, stream, q);
}

}  // namespace ua
