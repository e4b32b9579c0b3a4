// ua_api.cu -- the C ABI of include/ua.h: argument validation, the problem-
// owned workspace, tensor-map encoding, and the host planner that picks the
// execution path and launch shape for each call (gfx950 "Unified paged
// attention on gfx950, from the math up", section 6: choose between a path
// whose query-tile grid already fills the device and a split-KV path plus a
// reduction when it does not).
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "ua_accept.h"
#include "ua_cache.h"
#include "ua_common.cuh"
#include "ua_decode_tc.h"
#include "ua_fp4.cuh"
#include "ua_fp4.h"
#include "ua_plan.h"
#include "ua_prefill.h"
#include "ua_rope.h"
#include "ua_split.h"
#include "ua_tmap.h"
#include "ua_topk.h"
#include "ua_tree.h"
#include "ua_weights.h"

namespace {

thread_local char g_cuda_err[256] = "";

void note_cuda(cudaError_t e, const char* where) {
    std::snprintf(g_cuda_err, sizeof g_cuda_err, "%s: %s", where, cudaGetErrorString(e));
}

constexpr int kMaxSplits = 64;
constexpr size_t kWorkspaceCap = size_t(128) << 20;  // bytes of split partials

// Cache map of the problem's caches with boxes of `box_rows` slots.
bool encode_cache_map(CUtensorMap* m, const void* base, const ua_problem_desc& d, int box_rows) {
    return ua::encode_cache_map(m, base, d.head_size, d.num_kv_heads, d.block_size, d.num_blocks,
                                d.kv_dtype == UA_DTYPE_FP8_E4M3, box_rows);
}

// Two fresh buffers as zeros, complete on return: the problem's first call may
// come on any stream.  cudaMemset only queues its work on the legacy default
// stream, which a non-blocking stream does not wait for; a stream of its own
// does not wait for what the default stream still has to do either.
cudaError_t clear_now(void* a, size_t a_bytes, void* b, size_t b_bytes) {
    cudaStream_t st;
    cudaError_t e = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking);
    if (e != cudaSuccess) return e;
    e = cudaMemsetAsync(a, 0, a_bytes, st);
    if (e == cudaSuccess && b_bytes) e = cudaMemsetAsync(b, 0, b_bytes, st);
    const cudaError_t done = cudaStreamSynchronize(st);
    cudaStreamDestroy(st);
    return e == cudaSuccess ? done : e;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

struct ua_problem {
    ua_problem_desc desc;
    int device = 0;
    int num_sms = 0;
    int32_t* d_err = nullptr;      // the error word, then ua_plan_step's count of finished CTAs
    float* d_ws = nullptr;
    size_t ws_bytes = 0;
    size_t tree_bytes = 0;         // of the same buffer, what ua_forward_tree may use
    // scores of ua_forward_weights (UA_FLAG_KEY_WEIGHTS problems only)
    float* d_scores = nullptr;
    size_t scores_elems = 0;
    // pieces of every row of a call on a 4-bit cache (fp4 problems only)
    int4* d_pieces = nullptr;
    // work list of the persistent prefill kernel: entries, then the
    // per-sequence prefix, then [entries, claim counter]
    void* d_work = nullptr;
    int32_t work_cap = 0;
    // staging buffers of ua_forward_host (allocated on first use)
    void* st_q = nullptr;
    void* st_out = nullptr;
    int32_t* st_bt = nullptr;
    int32_t* st_cu = nullptr;
    int32_t* st_su = nullptr;
    float* st_sinks = nullptr;
    float* st_alibi = nullptr;
    // query-query bias set by ua_set_qq_bias (caller-owned device memory)
    const float* qq_bias = nullptr;
    int64_t qq_n = 0;
    int64_t qq_stride = 0;
    // rotary frequencies set by ua_set_rope (n = 0: none)
    ua::RopeTable rope{};
    // tensor maps of the most recent caches (re-encoded when the pointers change)
    const void* map_k_ptr = nullptr;
    const void* map_v_ptr = nullptr;
    CUtensorMap map_k16, map_v16;       // 16-slot boxes (split path)
    CUtensorMap map_kp, map_vp;         // prefill-path boxes
    int map_p_rows = 0;
    const void* map_g_k_ptr = nullptr;  // row-gather views of the caches (top-k calls)
    const void* map_g_v_ptr = nullptr;
    CUtensorMap map_kg, map_vg;
    int last_launches = 0;
    const char* last_path = "none";
    cudaEvent_t prof_begin = nullptr;
    cudaEvent_t prof_end = nullptr;
    // testing hook of ua_debug_stall_data_waits
    int32_t stall = 0;
    int64_t stall_ns = 0;
};

namespace {
void prof_mark(const ua_problem* p, bool begin, cudaStream_t st) {
    if (p->prof_begin && p->prof_end) cudaEventRecord(begin ? p->prof_begin : p->prof_end, st);
}
}  // namespace

extern "C" {

const char* ua_status_string(ua_status s) {
    switch (s) {
        case UA_OK: return "ok";
        case UA_ERR_INVALID_ARG: return "invalid argument";
        case UA_ERR_UNSUPPORTED: return "unsupported configuration";
        case UA_ERR_CUDA: return "CUDA error";
        case UA_ERR_OUT_OF_MEMORY: return "out of device memory";
        case UA_ERR_DEVICE: return "device reported an input error";
    }
    return "unknown status";
}

const char* ua_last_cuda_error(void) { return g_cuda_err; }

ua_status ua_problem_create(const ua_problem_desc* d, ua_problem** out) {
    if (!d || !out) return UA_ERR_INVALID_ARG;
    *out = nullptr;
    const uint32_t known = UA_FLAG_CAUSAL | UA_FLAG_SOFTCAP | UA_FLAG_ALIBI | UA_FLAG_WINDOW |
                           UA_FLAG_SINKS | UA_FLAG_QQ_BIAS | UA_FLAG_KEY_WEIGHTS;
    if (d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->num_q_heads % d->num_kv_heads != 0)
        return UA_ERR_INVALID_ARG;
    if (d->num_blocks <= 0 || d->max_num_seqs <= 0 || d->max_blocks_per_seq <= 0 ||
        d->max_total_q <= 0 || d->head_size <= 0 || d->block_size <= 0)
        return UA_ERR_INVALID_ARG;
    if (d->flags & ~known) return UA_ERR_INVALID_ARG;
    if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return UA_ERR_INVALID_ARG;
    if ((d->flags & UA_FLAG_SOFTCAP) && !(d->softcap > 0.f && std::isfinite(d->softcap)))
        return UA_ERR_INVALID_ARG;
    if ((d->flags & UA_FLAG_WINDOW) && (d->window < 1 || !(d->flags & UA_FLAG_CAUSAL)))
        return UA_ERR_INVALID_ARG;
    if (d->dtype != UA_DTYPE_BF16) return UA_ERR_UNSUPPORTED;
    if (d->kv_dtype != UA_DTYPE_BF16 && d->kv_dtype != UA_DTYPE_FP8_E4M3 &&
        d->kv_dtype != UA_DTYPE_FP4_E2M1)
        return UA_ERR_INVALID_ARG;
    if (d->kv_dtype != UA_DTYPE_BF16 &&
        (!(d->k_scale > 0.f) || !std::isfinite(d->k_scale) || !(d->v_scale > 0.f) ||
         !std::isfinite(d->v_scale)))
        return UA_ERR_INVALID_ARG;
    // One kernel family reads a 4-bit cache, whatever the call's shape.
    if (d->kv_dtype == UA_DTYPE_FP4_E2M1 && d->path != UA_PATH_AUTO)
        return d->path > UA_PATH_DECODE_TC ? UA_ERR_INVALID_ARG : UA_ERR_UNSUPPORTED;
    if (d->kv_dtype == UA_DTYPE_FP8_E4M3) {
        // The decode tensor-core kernel and the one of draft trees read an fp8 cache, at d = 128.
        if (d->head_size != 128) return UA_ERR_UNSUPPORTED;
        if (d->path != UA_PATH_AUTO && d->path != UA_PATH_DECODE_TC) return UA_ERR_UNSUPPORTED;
    }
    if (d->head_size != 64 && d->head_size != 128 && d->head_size != 256) return UA_ERR_UNSUPPORTED;
    if (d->block_size != 16 && d->block_size != 32 && d->block_size != 64) return UA_ERR_UNSUPPORTED;
    if (d->num_blocks > (int64_t(1) << 31) - 1) return UA_ERR_UNSUPPORTED;
    if (d->path > UA_PATH_DECODE_TC) return UA_ERR_INVALID_ARG;
    if (d->split_partials != UA_PARTIALS_F32 && d->split_partials != UA_PARTIALS_BF16)
        return UA_ERR_INVALID_ARG;

    // Rows that the workspace is sized for, and the bytes of one partial.  Sizes
    // that 64 bits could not count are more than any device holds.
    const double rows = (double)d->max_total_q * d->num_q_heads;
    const size_t row_bytes = size_t(d->head_size + 2) * sizeof(float);
    const size_t keys = ((size_t)d->max_blocks_per_seq * d->block_size + 127) / 128 * 128;
    if (((d->flags & UA_FLAG_KEY_WEIGHTS) && rows * std::max((double)row_bytes, 4. * keys) >= 0x1p62) ||
        (d->kv_dtype == UA_DTYPE_FP4_E2M1 && rows * row_bytes * 512 >= 0x1p62))
        return UA_ERR_OUT_OF_MEMORY;

    ua_problem* p = new (std::nothrow) ua_problem();
    if (!p) return UA_ERR_OUT_OF_MEMORY;
    p->desc = *d;
    cudaError_t e = cudaGetDevice(&p->device);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, p->device);
    if (e != cudaSuccess) {
        note_cuda(e, "ua_problem_create");
        delete p;
        return UA_ERR_CUDA;
    }
    const bool capped = rows * row_bytes * 16 >= (double)kWorkspaceCap;
    p->ws_bytes = capped ? kWorkspaceCap : size_t(d->max_total_q) * d->num_q_heads * row_bytes * 16;
    if (d->flags & UA_FLAG_KEY_WEIGHTS) {
        // Key weights always go through partials: room for one segment of every
        // row, and the rows' scores.
        p->ws_bytes = std::max(p->ws_bytes, size_t(d->max_total_q) * d->num_q_heads * row_bytes);
        p->scores_elems = size_t(d->max_total_q) * d->num_q_heads * keys;
    }
    size_t piece_bytes = 0;
    if (d->kv_dtype == UA_DTYPE_FP4_E2M1) {
        // A row may have as many pieces as warps share its keys: slots under the
        // cap, two at least, and the rows' statistics.
        const size_t slot = ua::fp4_workspace_bytes(d->max_total_q * d->num_q_heads, d->head_size);
        p->ws_bytes = std::max(std::min(slot * 512, kWorkspaceCap), slot * 2) +
                      size_t(d->max_total_q) * d->num_q_heads * 2 * sizeof(float) + 16;
        piece_bytes = size_t(d->max_total_q) * d->num_q_heads * sizeof(int4);
    }
    // Draft trees cut their work into one share per CTA of the device, with two partials
    // each.  (Key-weight problems have the size that is documented for them, and fewer
    // shares.)
    p->tree_bytes = p->ws_bytes;
    if (d->kv_dtype == UA_DTYPE_BF16 && !(d->flags & UA_FLAG_KEY_WEIGHTS))
        p->tree_bytes = std::max(p->ws_bytes, ua::tree_workspace_bytes(*d, p->num_sms));
    // Work-list entries: every call's (total_q / (2 ppt) + num_seqs) entries
    // without a KV split, and room for the splits the planner makes when the
    // grid is small (about 4 x 152 units per KV head x up to 64 segments).
    const int64_t cap = std::min<int64_t>(d->max_total_q + d->max_num_seqs + 64 * 4 * 160,
                                          int64_t(1) << 30);
    p->work_cap = (int32_t)cap;
    const size_t work_bytes = (size_t)cap * sizeof(int2) + (size_t)(d->max_num_seqs + 1) * 4 + 16;
    if (cudaMalloc(&p->d_err, 2 * sizeof(int32_t)) != cudaSuccess ||
        cudaMalloc(&p->d_ws, p->tree_bytes) != cudaSuccess ||
        cudaMalloc(&p->d_work, work_bytes) != cudaSuccess ||
        (piece_bytes && cudaMalloc(&p->d_pieces, piece_bytes) != cudaSuccess) ||
        (p->scores_elems && cudaMalloc(&p->d_scores, p->scores_elems * sizeof(float)) != cudaSuccess)) {
        cudaGetLastError();
        cudaFree(p->d_err);
        cudaFree(p->d_ws);
        cudaFree(p->d_work);
        cudaFree(p->d_pieces);
        delete p;
        return UA_ERR_OUT_OF_MEMORY;
    }
    e = clear_now(p->d_err, 2 * sizeof(int32_t), p->d_pieces, piece_bytes);
    if (e != cudaSuccess) {
        note_cuda(e, "ua_problem_create");
        cudaFree(p->d_err);
        cudaFree(p->d_ws);
        cudaFree(p->d_work);
        cudaFree(p->d_scores);
        cudaFree(p->d_pieces);
        delete p;
        return UA_ERR_CUDA;
    }
    *out = p;
    return UA_OK;
}

void ua_destroy(ua_problem* p) {
    if (!p) return;
    cudaFree(p->d_err);
    cudaFree(p->d_ws);
    cudaFree(p->d_work);
    cudaFree(p->d_scores);
    cudaFree(p->d_pieces);
    cudaFree(p->st_q);
    cudaFree(p->st_out);
    cudaFree(p->st_bt);
    cudaFree(p->st_cu);
    cudaFree(p->st_su);
    cudaFree(p->st_sinks);
    cudaFree(p->st_alibi);
    delete p;
}

int32_t ua_last_launch_count(const ua_problem* p) { return p ? p->last_launches : 0; }

const char* ua_last_path(const ua_problem* p) { return p ? p->last_path : "none"; }

ua_status ua_set_qq_bias(ua_problem* p, const float* bias, int64_t n, int64_t row_stride) {
    if (!p || !(p->desc.flags & UA_FLAG_QQ_BIAS)) return UA_ERR_INVALID_ARG;
    if (!bias) {
        p->qq_bias = nullptr;
        p->qq_n = p->qq_stride = 0;
        return UA_OK;
    }
    if (n < 1 || row_stride < n || (reinterpret_cast<uintptr_t>(bias) & 3u) != 0)
        return UA_ERR_INVALID_ARG;
    p->qq_bias = bias;
    p->qq_n = n;
    p->qq_stride = row_stride;
    return UA_OK;
}

ua_status ua_debug_stall_data_waits(ua_problem* p, int32_t enable, int64_t limit_ns) {
    if (!p) return UA_ERR_INVALID_ARG;
    if (enable && (limit_ns < 1000 || limit_ns > 1000000000)) return UA_ERR_INVALID_ARG;
    p->stall = enable ? 1 : 0;
    p->stall_ns = enable ? limit_ns : 0;
    return UA_OK;
}

ua_status ua_set_profile_events(ua_problem* p, void* ev_begin, void* ev_end) {
    if (!p || ((ev_begin == nullptr) != (ev_end == nullptr))) return UA_ERR_INVALID_ARG;
    p->prof_begin = reinterpret_cast<cudaEvent_t>(ev_begin);
    p->prof_end = reinterpret_cast<cudaEvent_t>(ev_end);
    return UA_OK;
}

}  // extern "C"

namespace {

// Every pointer is null or aligned to 4 bytes (the kernels' int32 and fp32 arrays).
template <typename... P>
bool words(const P*... ptr) {
    return ((reinterpret_cast<uintptr_t>(ptr) | ...) & 3u) == 0;
}

// Host checks shared by the forward entry points, then the kernel parameters.
// Returns UA_OK with *skip set when the call has nothing to compute.
ua_status prepare_call(ua_problem* p, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* cu_seqlens_q,
                       const int32_t* seqused_k, int32_t num_seqs, int64_t total_q,
                       int32_t max_seqlen_q, int32_t max_seqlen_k, uint32_t flags,
                       const float* sinks, const float* alibi_slopes, void* out,
                       ua::FwdParams* fpp, bool* skip) {
    *skip = false;
    if (!p) return UA_ERR_INVALID_ARG;
    p->last_launches = 0;
    p->last_path = "none";
    const ua_problem_desc& d = p->desc;
    if (num_seqs < 0 || num_seqs > d.max_num_seqs || total_q < 0 || total_q > d.max_total_q)
        return UA_ERR_INVALID_ARG;
    if (max_seqlen_q < 0 || max_seqlen_k < 0 || max_seqlen_q > max_seqlen_k ||
        (int64_t)max_seqlen_k > (int64_t)d.max_blocks_per_seq * d.block_size)
        return UA_ERR_INVALID_ARG;
    if ((flags & ~(d.flags & ~(uint32_t)UA_FLAG_KEY_WEIGHTS)) != 0) return UA_ERR_INVALID_ARG;
    if ((flags & UA_FLAG_WINDOW) && !(flags & UA_FLAG_CAUSAL)) return UA_ERR_INVALID_ARG;
    if (((flags & UA_FLAG_SINKS) != 0) != (sinks != nullptr)) return UA_ERR_INVALID_ARG;
    if (((flags & UA_FLAG_ALIBI) != 0) != (alibi_slopes != nullptr)) return UA_ERR_INVALID_ARG;
    if ((flags & UA_FLAG_QQ_BIAS) && (!p->qq_bias || (int64_t)max_seqlen_q > p->qq_n))
        return UA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_q == 0) {
        *skip = true;
        return UA_OK;
    }
    if (num_seqs > 65535) return UA_ERR_UNSUPPORTED;   // grids index sequences on gridDim.z
    if (!q || !k_cache || !v_cache || !block_table || !cu_seqlens_q || !seqused_k || !out)
        return UA_ERR_INVALID_ARG;
    if (!words(block_table, cu_seqlens_q, seqused_k, sinks, alibi_slopes)) return UA_ERR_INVALID_ARG;
    auto misaligned = [](const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) != 0; };
    if (misaligned(q) || misaligned(out) || misaligned(k_cache) || misaligned(v_cache))
        return UA_ERR_INVALID_ARG;
    if (max_seqlen_k == 0) {
        // Only empty sequences can be well formed; nothing to compute.
        max_seqlen_k = 1;
        if (max_seqlen_q > 1) return UA_ERR_INVALID_ARG;
    }

    ua::FwdParams& fp = *fpp;
    std::memset(&fp, 0, sizeof fp);
    fp.q = static_cast<const __nv_bfloat16*>(q);
    fp.k_cache = k_cache;
    fp.v_cache = v_cache;
    fp.block_table = block_table;
    fp.cu_seqlens_q = cu_seqlens_q;
    fp.seqused_k = seqused_k;
    fp.sinks = sinks;
    fp.alibi = alibi_slopes;
    fp.out = static_cast<__nv_bfloat16*>(out);
    fp.err = p->d_err;
    fp.total_q = total_q;
    fp.num_blocks = d.num_blocks;
    fp.num_seqs = num_seqs;
    fp.bt_stride = d.max_blocks_per_seq;
    fp.max_seqlen_q = max_seqlen_q;
    fp.max_seqlen_k = max_seqlen_k;
    fp.hq = d.num_q_heads;
    fp.hk = d.num_kv_heads;
    fp.g = d.num_q_heads / d.num_kv_heads;
    fp.d = d.head_size;
    fp.b = d.block_size;
    fp.flags = flags;
    fp.scale = d.scale;
    fp.softcap = d.softcap;
    fp.window = d.window;
    fp.kv_fp8 = d.kv_dtype == UA_DTYPE_FP8_E4M3 ? 1 : 0;
    fp.k_scale = d.kv_dtype != UA_DTYPE_BF16 ? d.k_scale : 1.f;
    fp.v_scale = d.kv_dtype != UA_DTYPE_BF16 ? d.v_scale : 1.f;
    fp.part_bf16 = d.split_partials == UA_PARTIALS_BF16 ? 1 : 0;
    fp.work_list = static_cast<int2*>(p->d_work);
    fp.seq_prefix = reinterpret_cast<int32_t*>(fp.work_list + p->work_cap);
    fp.work_info = fp.seq_prefix + (d.max_num_seqs + 1);
    fp.work_cap = p->work_cap;
    fp.stall = p->stall;
    fp.stall_ns = p->stall_ns;
    if (flags & UA_FLAG_QQ_BIAS) {
        fp.qq_bias = p->qq_bias;
        fp.qq_stride = p->qq_stride;
    }
    return UA_OK;
}

// The cache's tensor maps with 16-slot boxes (re-encoded when the caches
// change), and with boxes of b slots for the tensor-core kernels.
ua_status encode_maps(ua_problem* p, const void* k_cache, const void* v_cache, bool block_boxes) {
    const ua_problem_desc& d = p->desc;
    if (k_cache != p->map_k_ptr || v_cache != p->map_v_ptr) {
        if (!encode_cache_map(&p->map_k16, k_cache, d, 16) ||
            !encode_cache_map(&p->map_v16, v_cache, d, 16)) {
            p->map_k_ptr = p->map_v_ptr = nullptr;
            std::snprintf(g_cuda_err, sizeof g_cuda_err, "cuTensorMapEncodeTiled failed");
            return UA_ERR_CUDA;
        }
        p->map_k_ptr = k_cache;
        p->map_v_ptr = v_cache;
        p->map_p_rows = 0;
    }
    if (block_boxes && p->map_p_rows != d.block_size) {
        if (!encode_cache_map(&p->map_kp, k_cache, d, d.block_size) ||
            !encode_cache_map(&p->map_vp, v_cache, d, d.block_size)) {
            std::snprintf(g_cuda_err, sizeof g_cuda_err, "cuTensorMapEncodeTiled failed");
            p->map_p_rows = 0;
            return UA_ERR_CUDA;
        }
        p->map_p_rows = d.block_size;
    }
    return UA_OK;
}

// The call's partials behind each other in the problem's workspace.
void set_partials(const ua_problem* p, ua::FwdParams* fp, int splits, int chunk) {
    fp->splits = splits;
    fp->chunk = chunk;
    fp->part_o = p->d_ws;
    fp->part_ml = p->d_ws + (size_t)fp->total_q * p->desc.num_q_heads * splits * p->desc.head_size;
}

ua_status run_combine(const ua::FwdParams& fp, cudaStream_t st) {
    const cudaError_t e = ua::launch_combine(fp, st);
    if (e == cudaSuccess) return UA_OK;
    note_cuda(e, "combine kernel launch");
    return UA_ERR_CUDA;
}

// Attention over a 4-bit cache, or of draft trees over an fp8 one.  With fp->scores the
// rows' final (m, l) go to the front of the workspace, laid out like the partials of one
// segment.
ua_status run_fp4(ua_problem* p, ua::FwdParams* fp, cudaStream_t st) {
    const size_t rows = (size_t)fp->total_q * p->desc.num_q_heads;
    ua::Fp4RowsPlan tiles;
    if (ua::plan_fp4_rows(*fp, p->num_sms, p->ws_bytes, &tiles)) {
        set_partials(p, fp, tiles.splits, tiles.chunk);
        prof_mark(p, true, st);
        const cudaError_t e = fp->kv_fp8 ? ua::launch_fp8_tree(tiles, p->map_kp, p->map_vp, *fp, st)
                                         : ua::launch_fp4_rows(tiles, *fp, st);
        prof_mark(p, false, st);
        if (e != cudaSuccess) {
            note_cuda(e, "quantised rows kernel launch");
            return UA_ERR_CUDA;
        }
        const bool combine = tiles.splits > 1 || fp->scores;
        p->last_launches = combine ? 2 : 1;
        p->last_path = fp->kv_fp8 ? (combine ? "fp8_tree+combine" : "fp8_tree")
                                  : (combine ? "fp4_rows+combine" : "fp4_rows");
        return combine ? run_combine(*fp, st) : UA_OK;
    }
    // The kernel below knows no tree masks and reads 4-bit pages alone.
    if (fp->tree_mask || fp->kv_fp8) return UA_ERR_UNSUPPORTED;
    const size_t stats = fp->scores ? rows * 2 : 0;
    ua::Fp4Plan plan;
    if (!ua::plan_fp4(*fp, p->num_sms, p->ws_bytes - stats * sizeof(float) - 16, &plan)) return UA_ERR_UNSUPPORTED;
    fp->splits = plan.splits;
    fp->chunk = plan.chunk;
    fp->part_ml = p->d_ws;
    fp->part_o = p->d_ws + (stats + 3) / 4 * 4;
    fp->piece_ml = fp->part_o + rows * plan.splits * p->desc.head_size;
    fp->row_pieces = p->d_pieces;
    prof_mark(p, true, st);
    cudaError_t e = ua::launch_fp4(plan, *fp, st);
    prof_mark(p, false, st);
    if (e != cudaSuccess) {
        note_cuda(e, "fp4 kernel launch");
        return UA_ERR_CUDA;
    }
    fp->splits = 1;                      // what part_ml holds, for the key-weight kernel
    fp->chunk = 1 << 30;
    p->last_launches = 2;
    p->last_path = "fp4+merge";
    return UA_OK;
}

// The problem's device is the current one (the cache operators launch on it).
bool on_device(const ua_problem* p) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return dev == p->device;
}

// f / 2 pi (0 <= f <= 6: below one turn) times 2^64, to the nearest integer: the double's 53 bits
// times 1 / 2 pi to 128 bits.  (A product of doubles is off by up to 2^11, which at position
// 2^31 are 2^-22 of a turn.)
uint64_t turn_of(double f) {
    using U128 = unsigned __int128;
    constexpr uint64_t hi = 0x28be60db9391054au, lo = 0x7f09d5f47d4d3770u;    // 2^128 / 2 pi
    int e = 0;
    const uint64_t m = (uint64_t)std::ldexp(std::frexp(f, &e), 53);
    const U128 x = (U128)m * hi + (uint64_t)((U128)m * lo >> 64);              // m 2^64 / 2 pi, below 2^115
    const int shift = 53 - e;                                                  // f = m 2^-shift; 50 at least, or m = 0
    return shift < 50 || shift > 127 ? 0 : (uint64_t)((x + ((U128)1 << (shift - 1))) >> shift);
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

ua::CacheParams cache_params(const ua_problem* p, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* seqused_k, int32_t num_seqs) {
    const ua_problem_desc& d = p->desc;
    ua::CacheParams c{};
    c.k_cache = static_cast<uint8_t*>(const_cast<void*>(k_cache));
    c.v_cache = static_cast<uint8_t*>(const_cast<void*>(v_cache));
    c.block_table = block_table;
    c.seqused_k = seqused_k;
    c.err = p->d_err;
    c.num_blocks = d.num_blocks;
    c.num_seqs = num_seqs;
    c.bt_stride = d.max_blocks_per_seq;
    c.hk = d.num_kv_heads;
    c.d = d.head_size;
    c.b = d.block_size;
    c.kv_dtype = d.kv_dtype;
    c.k_scale = d.kv_dtype != UA_DTYPE_BF16 ? d.k_scale : 1.f;
    c.v_scale = d.kv_dtype != UA_DTYPE_BF16 ? d.v_scale : 1.f;
    return c;
}

}  // namespace

extern "C" {

ua_status ua_forward(ua_problem* p, const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_table, const int32_t* cu_seqlens_q,
                     const int32_t* seqused_k, int32_t num_seqs, int64_t total_q,
                     int32_t max_seqlen_q, int32_t max_seqlen_k, uint32_t flags,
                     const float* sinks, const float* alibi_slopes, void* out, void* stream) {
    ua::FwdParams fp;
    bool skip = false;
    ua_status rs = prepare_call(p, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                                num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags, sinks,
                                alibi_slopes, out, &fp, &skip);
    if (rs != UA_OK || skip) return rs;
    const ua_problem_desc& d = p->desc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int g = fp.g;
    max_seqlen_k = fp.max_seqlen_k;

    if (d.kv_dtype == UA_DTYPE_FP4_E2M1) return on_device(p) ? run_fp4(p, &fp, st) : UA_ERR_INVALID_ARG;
    rs = encode_maps(p, k_cache, v_cache, false);
    if (rs != UA_OK) return rs;

    // ---- path choice ------------------------------------------------------
    const int64_t rows_per_kv = (int64_t)g * max_seqlen_q;
    const bool tc_ok = ua::prefill_shape_ok(fp);
    const bool dec_ok = ua::decode_tc_shape_ok(fp);
    bool use_dec = dec_ok;
    bool use_tc = !dec_ok && tc_ok && rows_per_kv > 16;
    if (d.path == UA_PATH_SPLIT_KV) use_dec = use_tc = false;
    if (d.path == UA_PATH_TENSOR_CORE) {
        if (!tc_ok) return UA_ERR_UNSUPPORTED;
        use_dec = false;
        use_tc = true;
    }
    if (d.path == UA_PATH_DECODE_TC || fp.kv_fp8) {
        if (!dec_ok) return UA_ERR_UNSUPPORTED;   // an fp8 cache is read by this kernel only
        use_dec = true;
        use_tc = false;
    }
    if (use_dec || use_tc) {
        // Both tensor-core kernels read the caches through boxes of b slots.
        rs = encode_maps(p, k_cache, v_cache, true);
        if (rs != UA_OK) return rs;
    }
    if (use_dec) {
        ua::DecodePlan plan;
        ua::plan_decode_tc(fp, p->num_sms, p->ws_bytes, &plan);
        fp.splits = plan.splits;
        fp.chunk = plan.chunk;
        fp.part_o = p->d_ws;
        fp.part_ml = p->d_ws + (size_t)total_q * d.num_q_heads * plan.splits * d.head_size;
        prof_mark(p, true, st);
        cudaError_t e = ua::launch_decode_tc(plan, p->map_kp, p->map_vp, fp, st);
        prof_mark(p, false, st);
        if (e != cudaSuccess) {
            note_cuda(e, "decode kernel launch");
            return UA_ERR_CUDA;
        }
        if (plan.splits > 1) {
            e = ua::launch_combine(fp, st);
            if (e != cudaSuccess) {
                note_cuda(e, "combine kernel launch");
                return UA_ERR_CUDA;
            }
        }
        p->last_launches = plan.launches;
        p->last_path = plan.splits > 1 ? "decode_tc+combine" : "decode_tc";
        return UA_OK;
    }
    if (use_tc) {
        ua::PrefillPlan plan;
        ua::plan_prefill(fp, p->num_sms, p->ws_bytes, &plan);
        fp.splits = plan.splits;
        fp.chunk = plan.chunk;
        fp.part_o = p->d_ws;
        fp.part_ml = p->d_ws + (size_t)total_q * d.num_q_heads * plan.splits * d.head_size;
        prof_mark(p, true, st);
        cudaError_t e = ua::launch_prefill(plan, p->map_kp, p->map_vp, fp, st);
        prof_mark(p, false, st);
        if (e != cudaSuccess) {
            note_cuda(e, "prefill kernel launch");
            return UA_ERR_CUDA;
        }
        if (plan.splits > 1) {
            e = ua::launch_combine(fp, st);
            if (e != cudaSuccess) {
                note_cuda(e, "combine kernel launch");
                return UA_ERR_CUDA;
            }
        }
        p->last_launches = plan.launches;
        if (ua::prefill_pair_supported(fp.d) && plan.dense)
            p->last_path = plan.splits > 1 ? "tensor_core_grid+combine" : "tensor_core_grid";
        else if (ua::prefill_pair_supported(fp.d))
            p->last_path = plan.splits > 1 ? "tensor_core_pair+combine" : "tensor_core_pair";
        else
            p->last_path = plan.splits > 1 ? "tensor_core_cta2+combine" : "tensor_core_cta2";
        return UA_OK;
    }

    int rows = 1;
    int row_tiles = 1;
    if (rows_per_kv <= 16) {
        while (rows < rows_per_kv) rows <<= 1;
    } else {
        rows = 16;
        row_tiles = ceil_div(rows_per_kv, 16);
    }
    const int smem = ua::split_smem_bytes(d.head_size, rows);
    const int cps = std::max(1, std::min(8, (228 * 1024) / (smem + 1024)));
    const int64_t base = (int64_t)num_seqs * d.num_kv_heads * row_tiles;
    const int64_t slots = (int64_t)p->num_sms * cps;
    int splits = (int)std::min<int64_t>(kMaxSplits, std::max<int64_t>(1, (4 * slots + base - 1) / base));
    splits = std::min(splits, std::max(1, ceil_div(max_seqlen_k, 256)));
    const size_t per_split = (size_t)total_q * d.num_q_heads * (d.head_size + 2) * sizeof(float);
    splits = (int)std::min<size_t>((size_t)splits, p->ws_bytes / per_split);
    if (splits < 1) splits = 1;
    int chunk = ceil_div(ceil_div(max_seqlen_k, splits), 64) * 64;
    splits = ceil_div(max_seqlen_k, chunk);
    if (row_tiles * (int64_t)d.num_kv_heads > 0x7fffffffLL || splits > 65535) return UA_ERR_UNSUPPORTED;
    fp.splits = splits;
    fp.chunk = chunk;
    fp.row_tiles = row_tiles;
    fp.part_o = p->d_ws;
    fp.part_ml = p->d_ws + (size_t)total_q * d.num_q_heads * splits * d.head_size;

    prof_mark(p, true, st);
    cudaError_t e = ua::launch_split(rows, p->map_k16, p->map_v16, fp, st);
    prof_mark(p, false, st);
    if (e != cudaSuccess) {
        note_cuda(e, "split kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 1;
    if (splits > 1) {
        e = ua::launch_combine(fp, st);
        if (e != cudaSuccess) {
            note_cuda(e, "combine kernel launch");
            return UA_ERR_CUDA;
        }
        p->last_launches = 2;
        p->last_path = "split_kv+combine";
    } else {
        p->last_path = "split_kv_direct";
    }
    return UA_OK;
}

ua_status ua_forward_topk(ua_problem* p, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* cu_seqlens_q,
                          const int32_t* seqused_k, int32_t num_seqs, int64_t total_q,
                          int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* topk_idx,
                          const int32_t* topk_len, int32_t topk_stride, uint32_t flags,
                          const float* sinks, const float* alibi_slopes, void* out, void* stream) {
    ua::FwdParams fp;
    bool skip = false;
    ua_status rs = prepare_call(p, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                                num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags, sinks,
                                alibi_slopes, out, &fp, &skip);
    if (rs != UA_OK) return rs;
    if (topk_stride < 1) return UA_ERR_INVALID_ARG;
    if (topk_stride > (1 << 30)) return UA_ERR_UNSUPPORTED;   // entry indices stay in int32
    if (skip) return UA_OK;
    if (!topk_idx || !topk_len) return UA_ERR_INVALID_ARG;
    const ua_problem_desc& d = p->desc;
    if (d.kv_dtype != UA_DTYPE_BF16) return UA_ERR_UNSUPPORTED;
    if (d.path != UA_PATH_AUTO && d.path != UA_PATH_DECODE_TC) return UA_ERR_UNSUPPORTED;
    fp.topk_idx = topk_idx;
    fp.topk_len = topk_len;
    fp.topk_stride = topk_stride;
    if (!ua::topk_shape_ok(fp)) return UA_ERR_UNSUPPORTED;
    if (k_cache != p->map_g_k_ptr || v_cache != p->map_g_v_ptr) {
        if (!ua::encode_gather_map(&p->map_kg, k_cache, d.num_blocks, d.block_size, d.num_kv_heads,
                                   d.head_size) ||
            !ua::encode_gather_map(&p->map_vg, v_cache, d.num_blocks, d.block_size, d.num_kv_heads,
                                   d.head_size)) {
            p->map_g_k_ptr = p->map_g_v_ptr = nullptr;
            // Either the cache's rows overflow the gather's 32-bit row index
            // or the encoder failed.
            if ((int64_t)d.num_blocks * d.block_size * d.num_kv_heads > 0x7fffffffLL)
                return UA_ERR_UNSUPPORTED;
            std::snprintf(g_cuda_err, sizeof g_cuda_err, "cuTensorMapEncodeTiled failed");
            return UA_ERR_CUDA;
        }
        p->map_g_k_ptr = k_cache;
        p->map_g_v_ptr = v_cache;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ua::TopkPlan plan;
    ua::plan_topk(fp, p->num_sms, p->ws_bytes, &plan);
    fp.splits = plan.splits;
    fp.chunk = plan.chunk;
    fp.part_o = p->d_ws;
    fp.part_ml = p->d_ws + (size_t)total_q * d.num_q_heads * plan.splits * d.head_size;
    prof_mark(p, true, st);
    cudaError_t e = ua::launch_topk(plan, p->map_kg, p->map_vg, fp, st);
    prof_mark(p, false, st);
    if (e != cudaSuccess) {
        note_cuda(e, "top-k kernel launch");
        return UA_ERR_CUDA;
    }
    if (plan.splits > 1) {
        e = ua::launch_combine(fp, st);
        if (e != cudaSuccess) {
            note_cuda(e, "combine kernel launch");
            return UA_ERR_CUDA;
        }
    }
    p->last_launches = plan.launches;
    p->last_path = plan.splits > 1 ? "topk_tc+combine" : "topk_tc";
    return UA_OK;
}

ua_status ua_forward_weights(ua_problem* p, const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_table, const int32_t* cu_seqlens_q,
                             const int32_t* seqused_k, int32_t num_seqs, int64_t total_q,
                             int32_t max_seqlen_q, int32_t max_seqlen_k, uint32_t flags,
                             const float* sinks, const float* alibi_slopes, const float* weights_in,
                             float* weights_out, int64_t weight_stride, float decay, void* out,
                             void* stream) {
    ua::FwdParams fp;
    bool skip = false;
    ua_status rs = prepare_call(p, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                                num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags, sinks,
                                alibi_slopes, out, &fp, &skip);
    if (rs != UA_OK) return rs;
    const ua_problem_desc& d = p->desc;
    if (!(d.flags & UA_FLAG_KEY_WEIGHTS) || !(decay >= 0.f) || !std::isfinite(decay) ||
        weight_stride < max_seqlen_k || !on_device(p))
        return UA_ERR_INVALID_ARG;
    if (skip) return UA_OK;
    if (!weights_out || !words(weights_in, weights_out)) return UA_ERR_INVALID_ARG;
    if (d.path != UA_PATH_AUTO || d.num_kv_heads > 65535 || max_seqlen_k > 1 << 30) return UA_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    fp.scores = p->d_scores;
    fp.score_stride = ((int64_t)fp.max_seqlen_k + 127) / 128 * 128;
    if (d.kv_dtype == UA_DTYPE_FP4_E2M1) {
        rs = run_fp4(p, &fp, st);
        if (rs != UA_OK) return rs;
        p->last_path = std::strncmp(p->last_path, "fp4_rows", 8) == 0 ? "fp4_rows+combine+weights"
                                                                      : "fp4+merge+weights";
    } else {
        if (!ua::decode_tc_shape_ok(fp)) return UA_ERR_UNSUPPORTED;
        rs = encode_maps(p, k_cache, v_cache, true);
        if (rs != UA_OK) return rs;
        ua::DecodePlan plan;
        ua::plan_decode_tc(fp, p->num_sms, p->ws_bytes, &plan);
        if ((int64_t)plan.splits * plan.row_tiles > 0x7fffffffLL) return UA_ERR_UNSUPPORTED;
        set_partials(p, &fp, plan.splits, plan.chunk);
        prof_mark(p, true, st);
        const cudaError_t e = ua::launch_decode_tc(plan, p->map_kp, p->map_vp, fp, st);
        prof_mark(p, false, st);
        if (e != cudaSuccess) {
            note_cuda(e, "decode kernel launch");
            return UA_ERR_CUDA;
        }
        rs = run_combine(fp, st);
        if (rs != UA_OK) return rs;
        p->last_path = "decode_tc+combine+weights";
    }
    const bool again = std::strncmp(p->last_path, "fp4_rows", 8) == 0;
    const cudaError_t e =
        again ? ua::launch_fp4_weights(fp, p->num_sms, weights_in, weights_out, weight_stride, decay, st)
              : ua::launch_weights(fp, weights_in, weights_out, weight_stride, decay,
                                   d.kv_dtype == UA_DTYPE_FP4_E2M1, st);
    if (e != cudaSuccess) {
        note_cuda(e, "weights kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 3;
    return UA_OK;
}

ua_status ua_cache_store(ua_problem* p, const void* k_new, const void* v_new, int64_t new_stride,
                         void* k_cache, void* v_cache, const int32_t* block_table,
                         const int32_t* cu_seqlens_q, const int32_t* seqused_k, int32_t num_seqs,
                         int64_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k, void* stream) {
    if (!p) return UA_ERR_INVALID_ARG;
    p->last_launches = 0;
    p->last_path = "none";
    const ua_problem_desc& d = p->desc;
    if (num_seqs < 0 || num_seqs > d.max_num_seqs || total_q < 0 || total_q > d.max_total_q ||
        max_seqlen_q < 0 || max_seqlen_k < max_seqlen_q ||
        (int64_t)max_seqlen_k > (int64_t)d.max_blocks_per_seq * d.block_size ||
        new_stride < (int64_t)d.num_kv_heads * d.head_size || new_stride % 8 != 0 || !on_device(p))
        return UA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return UA_OK;
    if (num_seqs > 65535) return UA_ERR_UNSUPPORTED;
    if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !cu_seqlens_q || !seqused_k ||
        !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !words(block_table, cu_seqlens_q, seqused_k))
        return UA_ERR_INVALID_ARG;
    ua::StoreParams sp{};
    sp.c = cache_params(p, k_cache, v_cache, block_table, seqused_k, num_seqs);
    sp.k_new = static_cast<const __nv_bfloat16*>(k_new);
    sp.v_new = static_cast<const __nv_bfloat16*>(v_new);
    sp.cu_seqlens_q = cu_seqlens_q;
    sp.stride = new_stride;
    sp.total_q = total_q;
    sp.max_seqlen_q = max_seqlen_q;
    sp.max_seqlen_k = max_seqlen_k;
    const cudaError_t e = ua::launch_store(sp, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        note_cuda(e, "store kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 1;
    p->last_path = "store";
    return UA_OK;
}

ua_status ua_cache_expand(ua_problem* p, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* seqused_k, const int32_t* begin,
                          int32_t num_seqs, int32_t max_keys, void* k_out, void* v_out,
                          const int32_t* out_block_table, int32_t out_table_stride,
                          int64_t out_num_blocks, void* stream) {
    if (!p) return UA_ERR_INVALID_ARG;
    p->last_launches = 0;
    p->last_path = "none";
    const ua_problem_desc& d = p->desc;
    if (num_seqs < 0 || num_seqs > d.max_num_seqs || max_keys < 0 || out_table_stride < 1 ||
        out_num_blocks < 1 || !on_device(p))
        return UA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_keys == 0) return UA_OK;
    if (num_seqs > 65535 || out_num_blocks > (int64_t(1) << 31) - 1) return UA_ERR_UNSUPPORTED;
    if (!k_cache || !v_cache || !block_table || !seqused_k || !k_out || !v_out || !out_block_table ||
        !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out) ||
        !words(block_table, seqused_k, begin, out_block_table))
        return UA_ERR_INVALID_ARG;
    ua::ExpandParams ep{};
    ep.c = cache_params(p, k_cache, v_cache, block_table, seqused_k, num_seqs);
    ep.begin = begin;
    ep.k_out = static_cast<__nv_bfloat16*>(k_out);
    ep.v_out = static_cast<__nv_bfloat16*>(v_out);
    ep.out_table = out_block_table;
    ep.out_blocks = out_num_blocks;
    ep.out_stride = out_table_stride;
    ep.max_keys = max_keys;
    const cudaError_t e = ua::launch_expand(ep, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        note_cuda(e, "expand kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 1;
    p->last_path = "expand";
    return UA_OK;
}

ua_status ua_cache_evict(ua_problem* p, void* k_cache, void* v_cache, const int32_t* block_table,
                         const int32_t* dst_block_table, const int32_t* seqused_k, int32_t num_seqs,
                         int32_t max_seqlen_k, const float* weights_in, float* weights_out,
                         int64_t weight_stride, int32_t budget, int32_t recent, int32_t* kept,
                         int32_t* seqused_out, void* stream) {
    if (!p) return UA_ERR_INVALID_ARG;
    p->last_launches = 0;
    p->last_path = "none";
    const ua_problem_desc& d = p->desc;
    if (num_seqs < 0 || num_seqs > d.max_num_seqs || max_seqlen_k < 0 ||
        (int64_t)max_seqlen_k > (int64_t)d.max_blocks_per_seq * d.block_size || budget < 1 ||
        recent < 0 || recent > budget || weight_stride < max_seqlen_k || !on_device(p))
        return UA_ERR_INVALID_ARG;
    if (num_seqs == 0) return UA_OK;
    if (num_seqs > 65535 || d.num_kv_heads > 32767 || max_seqlen_k > 1 << 30) return UA_ERR_UNSUPPORTED;
    if (!k_cache || !v_cache || !block_table || !seqused_k || !weights_in || !weights_out || !kept ||
        !seqused_out || !aligned16(k_cache) || !aligned16(v_cache) ||
        !words(block_table, dst_block_table, seqused_k, weights_in, weights_out, kept, seqused_out))
        return UA_ERR_INVALID_ARG;
    ua::EvictParams ep{};
    ep.c = cache_params(p, k_cache, v_cache, block_table, seqused_k, num_seqs);
    ep.in_place = !dst_block_table || dst_block_table == block_table;
    ep.dst_table = ep.in_place ? block_table : dst_block_table;
    ep.w_in = weights_in;
    ep.w_out = weights_out;
    ep.kept = kept;
    ep.seqused_out = seqused_out;
    ep.w_stride = weight_stride;
    ep.max_seqlen_k = max_seqlen_k;
    ep.budget = budget;
    ep.recent = recent;
    const cudaError_t e = ua::launch_evict(ep, p->num_sms, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        note_cuda(e, "evict kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 2;
    p->last_path = ep.in_place ? "evict_in_place" : "evict";
    return UA_OK;
}

ua_status ua_plan_step(ua_problem* p, int32_t* block_table, int32_t* blocks_held, int32_t* free_blocks,
                       int32_t* free_count, const int32_t* ctx_lens, const int32_t* new_lens,
                       const int32_t* parents, int64_t parents_stride, int32_t num_seqs, int64_t max_tokens,
                       int32_t* granted, int32_t* cu_seqlens_q, int32_t* seqused_k, int32_t* positions,
                       int64_t* slots, uint32_t* tree_mask, int32_t mask_stride, void* stream) {
    if (!p) return UA_ERR_INVALID_ARG;
    p->last_launches = 0;
    p->last_path = "none";
    const ua_problem_desc& d = p->desc;
    if (num_seqs < 0 || num_seqs > d.max_num_seqs || max_tokens < 0 || max_tokens > d.max_total_q ||
        (parents && parents_stride < 1) || (tree_mask && mask_stride < 1) || !on_device(p))
        return UA_ERR_INVALID_ARG;
    if (num_seqs == 0 && max_tokens == 0) return UA_OK;
    if (num_seqs > ua::kMaxPlanSeqs || max_tokens > 0x7fffffff || (parents && parents_stride > 0x7fffffff))
        return UA_ERR_UNSUPPORTED;
    if (!free_blocks || !free_count || !cu_seqlens_q || (max_tokens && (!positions || !slots)) ||
        (num_seqs && (!block_table || !blocks_held || !ctx_lens || !new_lens || !granted || !seqused_k)) ||
        !words(block_table, blocks_held, free_blocks, free_count, ctx_lens, new_lens, parents, granted, cu_seqlens_q,
               seqused_k, positions, tree_mask) ||
        (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
        return UA_ERR_INVALID_ARG;
    ua::PlanParams pp{};
    pp.block_table = block_table;
    pp.held = blocks_held;
    pp.pool = free_blocks;
    pp.pool_count = free_count;
    pp.ctx_lens = ctx_lens;
    pp.new_lens = new_lens;
    pp.parents = parents;
    pp.granted = granted;
    pp.cu = cu_seqlens_q;
    pp.used = seqused_k;
    pp.positions = positions;
    pp.slots = slots;
    pp.mask = tree_mask;
    pp.err = p->d_err;
    pp.ticket = p->d_err + 1;
    pp.parents_stride = parents_stride;
    pp.num_blocks = d.num_blocks;
    pp.max_tokens = max_tokens;
    pp.mask_stride = mask_stride;
    pp.num_seqs = num_seqs;
    pp.bt_stride = d.max_blocks_per_seq;
    pp.b_log2 = d.block_size == 16 ? 4 : d.block_size == 32 ? 5 : 6;
    const cudaError_t e = ua::launch_plan(pp, p->num_sms, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        note_cuda(e, "plan kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 1;
    p->last_path = "plan";
    return UA_OK;
}

ua_status ua_set_rope(ua_problem* p, const double* inv_freq, int32_t n, uint32_t layout, float magnitude) {
    if (!p || !inv_freq || n < 1 || layout > UA_ROPE_PAIRS || !std::isfinite(magnitude)) return UA_ERR_INVALID_ARG;
    if (2 * (int64_t)n > p->desc.head_size || n % 8 != 0) return UA_ERR_UNSUPPORTED;
    ua::RopeTable t{};
    for (int i = 0; i < n; ++i) {
        if (!(inv_freq[i] >= 0. && inv_freq[i] <= 6.)) return UA_ERR_INVALID_ARG;
        t.turn[i] = turn_of(inv_freq[i]);
    }
    t.n = n;
    t.pairs = layout == UA_ROPE_PAIRS;
    t.magnitude = magnitude;
    p->rope = t;
    return UA_OK;
}

ua_status ua_rope_store(ua_problem* p, const void* q, int64_t q_stride, const void* k_new, const void* v_new,
                        int64_t kv_stride, const int32_t* positions, const int64_t* slots, int64_t total_q,
                        void* q_out, int64_t out_stride, void* k_cache, void* v_cache, void* stream) {
    if (!p) return UA_ERR_INVALID_ARG;
    p->last_launches = 0;
    p->last_path = "none";
    const ua_problem_desc& d = p->desc;
    const int64_t q_row = (int64_t)d.num_q_heads * d.head_size, kv_row = (int64_t)d.num_kv_heads * d.head_size;
    if (total_q < 0 || total_q > d.max_total_q || q_stride < q_row || out_stride < q_row || kv_stride < kv_row ||
        q_stride % 8 != 0 || out_stride % 8 != 0 || kv_stride % 8 != 0 || p->rope.n == 0 || !on_device(p))
        return UA_ERR_INVALID_ARG;
    if (total_q == 0) return UA_OK;
    if (total_q > 0x7fffffff || q_row + 2 * kv_row > 0x3fffffff) return UA_ERR_UNSUPPORTED;
    if (!q || !k_new || !v_new || !positions || !slots || !q_out || !k_cache || !v_cache || !aligned16(q) ||
        !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !words(positions) || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0 || (q_out == q && out_stride != q_stride))
        return UA_ERR_INVALID_ARG;
    ua::RopeParams rp{};
    rp.c = cache_params(p, k_cache, v_cache, nullptr, nullptr, 0);
    rp.q = static_cast<const __nv_bfloat16*>(q);
    rp.k_new = static_cast<const __nv_bfloat16*>(k_new);
    rp.v_new = static_cast<const __nv_bfloat16*>(v_new);
    rp.q_out = static_cast<__nv_bfloat16*>(q_out);
    rp.positions = positions;
    rp.slots = slots;
    rp.q_stride = q_stride;
    rp.kv_stride = kv_stride;
    rp.out_stride = out_stride;
    rp.total_q = total_q;
    rp.hq = d.num_q_heads;
    const cudaError_t e = ua::launch_rope_store(rp, p->rope, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        note_cuda(e, "rope store kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 1;
    p->last_path = "rope_store";
    return UA_OK;
}

ua_status ua_forward_tree(ua_problem* p, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                          int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
                          const uint32_t* tree_mask, int32_t mask_stride, const int32_t* positions, uint32_t flags,
                          const float* sinks, const float* alibi_slopes, void* out, void* stream) {
    ua::FwdParams fp;
    bool skip = false;
    ua_status rs = prepare_call(p, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, num_seqs, total_q,
                                max_seqlen_q, max_seqlen_k, flags, sinks, alibi_slopes, out, &fp, &skip);
    if (rs != UA_OK) return rs;
    if (!(flags & UA_FLAG_CAUSAL) || mask_stride < 1 || 32LL * mask_stride < max_seqlen_q || !on_device(p))
        return UA_ERR_INVALID_ARG;
    const ua_problem_desc& d = p->desc;
    if ((flags & UA_FLAG_QQ_BIAS) || d.path != UA_PATH_AUTO ||
        max_seqlen_q > ua::kMaxTree || max_seqlen_k > 1 << 30 || d.num_kv_heads > 65535 ||
        d.num_q_heads / d.num_kv_heads > 128)
        return UA_ERR_UNSUPPORTED;
    if (skip) return UA_OK;
    const bool places = (flags & (UA_FLAG_WINDOW | UA_FLAG_ALIBI)) != 0;
    if (!tree_mask || (places && !positions) || !words(tree_mask, positions)) return UA_ERR_INVALID_ARG;
    fp.tree_mask = tree_mask;
    fp.mask_stride = mask_stride;
    fp.positions = positions;
    if (d.kv_dtype == UA_DTYPE_FP4_E2M1) return run_fp4(p, &fp, reinterpret_cast<cudaStream_t>(stream));
    rs = encode_maps(p, k_cache, v_cache, true);
    if (rs != UA_OK) return rs;
    if (fp.kv_fp8) return run_fp4(p, &fp, reinterpret_cast<cudaStream_t>(stream));
    ua::TreePlan plan;
    if (!ua::plan_tree(&fp, p->num_sms, p->d_ws, p->tree_bytes, &plan)) return UA_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    prof_mark(p, true, st);
    const cudaError_t e = ua::launch_tree(plan, p->map_kp, p->map_vp, fp, st);
    prof_mark(p, false, st);
    if (e != cudaSuccess) {
        note_cuda(e, "tree kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = plan.ctas > 1 ? 2 : 1;
    p->last_path = plan.ctas > 1 ? "tree+merge" : "tree";
    return UA_OK;
}

ua_status ua_cache_accept(ua_problem* p, void* k_cache, void* v_cache, const int32_t* block_table,
                          const int32_t* cu_seqlens_q, const int32_t* seqused_k, const int32_t* parents,
                          int64_t parents_stride, const int32_t* last, int32_t num_seqs, int64_t total_q,
                          int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t* path, int32_t path_stride,
                          int32_t* accepted, int32_t* seqused_out, void* stream) {
    if (!p) return UA_ERR_INVALID_ARG;
    p->last_launches = 0;
    p->last_path = "none";
    const ua_problem_desc& d = p->desc;
    if (num_seqs < 0 || num_seqs > d.max_num_seqs || total_q < 0 || total_q > d.max_total_q || max_seqlen_q < 0 ||
        max_seqlen_k < max_seqlen_q || (int64_t)max_seqlen_k > (int64_t)d.max_blocks_per_seq * d.block_size ||
        parents_stride < std::max(1, max_seqlen_q) || path_stride < 1 || !on_device(p))
        return UA_ERR_INVALID_ARG;
    if (num_seqs == 0) return UA_OK;
    if (max_seqlen_q > ua::kMaxTree) return UA_ERR_UNSUPPORTED;
    if (!k_cache || !v_cache || !block_table || !cu_seqlens_q || !seqused_k || !parents || !last || !path || !accepted ||
        !seqused_out || !aligned16(k_cache) || !aligned16(v_cache) ||
        !words(block_table, cu_seqlens_q, seqused_k, parents, last, path, accepted, seqused_out))
        return UA_ERR_INVALID_ARG;
    ua::AcceptParams ap{};
    ap.c = cache_params(p, k_cache, v_cache, block_table, seqused_k, num_seqs);
    ap.cu_seqlens_q = cu_seqlens_q;
    ap.parents = parents;
    ap.last = last;
    ap.path = path;
    ap.accepted = accepted;
    ap.seqused_out = seqused_out;
    ap.parents_stride = parents_stride;
    ap.total_q = total_q;
    ap.path_stride = path_stride;
    ap.max_seqlen_q = max_seqlen_q;
    ap.max_seqlen_k = max_seqlen_k;
    const cudaError_t e = ua::launch_accept(ap, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) {
        note_cuda(e, "accept kernel launch");
        return UA_ERR_CUDA;
    }
    p->last_launches = 1;
    p->last_path = "accept";
    return UA_OK;
}

ua_status ua_forward_host(ua_problem* p, const void* q_host, const void* k_cache,
                          const void* v_cache, const int32_t* block_table_host,
                          const int32_t* cu_seqlens_q_host, const int32_t* seqused_k_host,
                          int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q,
                          int32_t max_seqlen_k, uint32_t flags, const float* sinks_host,
                          const float* alibi_host, void* out_host, void* stream) {
    if (!p) return UA_ERR_INVALID_ARG;
    const ua_problem_desc& d = p->desc;
    if (num_seqs < 0 || num_seqs > d.max_num_seqs || total_q < 0 || total_q > d.max_total_q)
        return UA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_q == 0) return UA_OK;
    if (!q_host || !block_table_host || !cu_seqlens_q_host || !seqused_k_host || !out_host)
        return UA_ERR_INVALID_ARG;
    const size_t qbytes_max = (size_t)d.max_total_q * d.num_q_heads * d.head_size * 2;
    if (!p->st_q) {
        bool ok = cudaMalloc(&p->st_q, qbytes_max) == cudaSuccess &&
                  cudaMalloc(&p->st_out, qbytes_max) == cudaSuccess &&
                  cudaMalloc(&p->st_bt, (size_t)d.max_num_seqs * d.max_blocks_per_seq * 4) == cudaSuccess &&
                  cudaMalloc(&p->st_cu, (size_t)(d.max_num_seqs + 1) * 4) == cudaSuccess &&
                  cudaMalloc(&p->st_su, (size_t)d.max_num_seqs * 4) == cudaSuccess &&
                  cudaMalloc(&p->st_sinks, (size_t)d.num_q_heads * 4) == cudaSuccess &&
                  cudaMalloc(&p->st_alibi, (size_t)d.num_q_heads * 4) == cudaSuccess;
        if (!ok) {
            cudaGetLastError();
            cudaFree(p->st_q); cudaFree(p->st_out); cudaFree(p->st_bt); cudaFree(p->st_cu);
            cudaFree(p->st_su); cudaFree(p->st_sinks); cudaFree(p->st_alibi);
            p->st_q = p->st_out = nullptr;
            p->st_bt = p->st_cu = p->st_su = nullptr;
            p->st_sinks = p->st_alibi = nullptr;
            return UA_ERR_OUT_OF_MEMORY;
        }
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t qbytes = (size_t)total_q * d.num_q_heads * d.head_size * 2;
    cudaError_t e = cudaMemcpyAsync(p->st_q, q_host, qbytes, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(p->st_bt, block_table_host, (size_t)num_seqs * d.max_blocks_per_seq * 4,
                            cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(p->st_cu, cu_seqlens_q_host, (size_t)(num_seqs + 1) * 4,
                            cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(p->st_su, seqused_k_host, (size_t)num_seqs * 4, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess && sinks_host)
        e = cudaMemcpyAsync(p->st_sinks, sinks_host, (size_t)d.num_q_heads * 4, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess && alibi_host)
        e = cudaMemcpyAsync(p->st_alibi, alibi_host, (size_t)d.num_q_heads * 4, cudaMemcpyHostToDevice, st);
    if (e != cudaSuccess) {
        note_cuda(e, "ua_forward_host upload");
        return UA_ERR_CUDA;
    }
    ua_status s = ua_forward(p, p->st_q, k_cache, v_cache, p->st_bt, p->st_cu, p->st_su, num_seqs,
                             total_q, max_seqlen_q, max_seqlen_k, flags,
                             sinks_host ? p->st_sinks : nullptr, alibi_host ? p->st_alibi : nullptr,
                             p->st_out, stream);
    if (s != UA_OK) return s;
    e = cudaMemcpyAsync(out_host, p->st_out, qbytes, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) {
        note_cuda(e, "ua_forward_host download");
        return UA_ERR_CUDA;
    }
    return UA_OK;
}

ua_status ua_check_device_error(ua_problem* p, void* stream, int32_t* code) {
    if (!p || !code) return UA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int32_t h = 0;
    cudaError_t e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) e = cudaMemcpy(&h, p->d_err, sizeof h, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(p->d_err, 0, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        note_cuda(e, "ua_check_device_error");
        return UA_ERR_CUDA;
    }
    *code = h;
    return h ? UA_ERR_DEVICE : UA_OK;
}

}  // extern "C"
