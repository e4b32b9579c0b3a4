/*
 * ua.h -- C ABI of the unified paged varlen attention forward library
 * (libua.so, sm_103a).
 *
 * One forward call serves decode (S_q = 1), prefill (S_q = S_k) and chunked
 * prefill (1 < S_q < S_k) over a block-table-mapped bf16 KV cache.  For each
 * packed query row i of sequence s and query head h it computes
 *
 *     O_i = sum_j softmax(x)_j V_j   over the visible keys j of s,
 *
 * with the score transform applied in this fixed order (gfx950 "Unified paged
 * attention on gfx950, from the math up", section 1 "What unified attention
 * computes", steps 1-7):
 *
 *     x_j  = tau * <Q_i, K_j>                            scale
 *     x_j  = c * tanh(x_j / c)            UA_FLAG_SOFTCAP
 *     x_j += slope_h * (j - ctx)          UA_FLAG_ALIBI
 *     x_j += B[i][j - ctx] for j >= ctx   UA_FLAG_QQ_BIAS (see ua_set_qq_bias)
 *     drop j > i + ctx                    UA_FLAG_CAUSAL
 *     drop j < i + ctx - W + 1            UA_FLAG_WINDOW (requires CAUSAL)
 *     sink_h joins the denominator        UA_FLAG_SINKS (no value row)
 *
 * where ctx = S_k - S_q (the query chunk is the last S_q of the sequence's S_k
 * keys, and its K/V are already in the cache), GQA maps query head h to KV head
 * floor(h / g) with g = H_q / H_k (section 0, notation; section 4 on packing the
 * g heads of one KV head into one tile), and a row with an empty denominator
 * gets O_i = 0 (gfx1151 ALGORITHM.md section 6).
 *
 * Layouts (all row-major, contiguous, device memory owned by the caller):
 *   q, out        bf16  [total_q, H_q, d]        packed ragged batch
 *   k_cache,
 *   v_cache       bf16  [num_blocks, b, H_k, d]  paged cache (section 0)
 *   block_table   int32 [num_seqs, max_blocks_per_seq]; key j of sequence s
 *                       lives in block block_table[s][j / b], slot j % b
 *   cu_seqlens_q  int32 [num_seqs + 1]; sequence s owns rows
 *                       cu_seqlens_q[s] .. cu_seqlens_q[s+1]-1, cu_seqlens_q[0] = 0
 *   seqused_k     int32 [num_seqs]; S_k of each sequence
 *   sinks         fp32  [H_q] natural-log sink logits (UA_FLAG_SINKS only)
 *   alibi_slopes  fp32  [H_q] (UA_FLAG_ALIBI only)
 * Block-table entries past ceil(S_k / b) are never read.
 *
 * Every call is asynchronous on the given stream and never synchronises the
 * host.  Errors the host can see are returned as ua_status before anything is
 * launched; errors only the device can see (bad lengths or block ids inside
 * the metadata arrays) are recorded in a problem-owned device error word that
 * ua_check_device_error() reads -- the kernels never trap.
 */
#ifndef UA_H_
#define UA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ua_status {
    UA_OK = 0,
    UA_ERR_INVALID_ARG = 1,   /* a null or malformed argument; nothing launched */
    UA_ERR_UNSUPPORTED = 2,   /* valid, but outside what this build implements */
    UA_ERR_CUDA = 3,          /* a CUDA runtime call failed (see ua_last_cuda_error) */
    UA_ERR_OUT_OF_MEMORY = 4, /* device workspace allocation failed */
    UA_ERR_DEVICE = 5         /* the device error word was non-zero */
} ua_status;

/* Score-transform flags (section 1 of the spec above).  A problem is created
 * with the set it may use; each call passes a subset of it. */
enum {
    UA_FLAG_CAUSAL = 1u << 0,
    UA_FLAG_SOFTCAP = 1u << 1,
    UA_FLAG_ALIBI = 1u << 2,
    UA_FLAG_WINDOW = 1u << 3,
    UA_FLAG_SINKS = 1u << 4,
    UA_FLAG_QQ_BIAS = 1u << 5,
    /* Descriptor only: the problem may run ua_forward_weights (its score
     * workspace is allocated at creation); never part of a call's flags. */
    UA_FLAG_KEY_WEIGHTS = 1u << 6
};

/* Bits of the device error word. */
enum {
    UA_DEVERR_CONTEXT = 1u << 0,  /* seqused_k[s] < S_q(s): rows of s are written as 0 */
    UA_DEVERR_BLOCK_ID = 1u << 1, /* a block id outside [0, num_blocks): those keys read as 0 */
    UA_DEVERR_CU_SEQLENS = 1u << 2, /* cu_seqlens_q decreasing or past total_q: s skipped */
    UA_DEVERR_BOUNDS = 1u << 3,   /* S_q > max_seqlen_q or S_k > max_seqlen_k or
                                     S_k > max_blocks_per_seq * b: rows of s written as 0
                                     where addressable */
    UA_DEVERR_TIMEOUT = 1u << 4,  /* a bounded on-chip wait gave up; results unspecified */
    UA_DEVERR_TREE = 1u << 5,     /* a draft tree's parent, accepted node or position out of range */
    UA_DEVERR_POOL = 1u << 6      /* ua_plan_step: a pool count outside [0, num_blocks], or more
                                     blocks given back than the pool has room for */
};

/* Element types.  Q, O: bf16.  K/V caches: bf16, or fp8 e4m3 codes (one byte
 * each; OCP e4m3: bias 7, subnormals, no infinities, 0x7f / 0xff NaN) with one
 * scale per tensor, K = code * k_scale, V = code * v_scale (gfx950 page,
 * section 7.3 "fp8 KV cache (bf16-Q + fp8-KV)").  ua_forward reads an fp8
 * cache on its DECODE_TC path only; the other calls say what they need.
 *
 * UA_DTYPE_FP4_E2M1: caches in 4 bits, uint8 [num_blocks, H_k, P] with
 * P = b * (d / 2 + d / 16) bytes for one (block, KV head): first b rows of
 * d / 2 bytes holding e2m1 codes (dim 2i in the low nibble of byte i, dim
 * 2i + 1 in the high one; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign
 * bit), then b rows of d / 16 e4m3 scales, one per 16 consecutive dims.
 * K = code * scale * k_scale, V = code * scale * v_scale; ua_cache_store
 * writes this format, and a (block, KV head) is one contiguous, 16-byte
 * aligned run.  Any d, b, g and S_q; needs path AUTO and, for ua_forward, the
 * problem's device to be current (else UA_ERR_INVALID_ARG).  A NaN value
 * reaches the rows that see its key and no others.  The problem's workspace
 * holds two partials of every row at least: 8 * max_total_q * H_q * (d + 2)
 * bytes.  UA_ERR_UNSUPPORTED past
 * max_seqlen_k = 2^30, g * max_seqlen_q = 2^30, total_q * H_q = 2^32, or 2^31
 * steps of 32 keys over all (sequence, KV head, tile of 8 or 16 rows). */
enum { UA_DTYPE_BF16 = 0, UA_DTYPE_FP8_E4M3 = 1, UA_DTYPE_FP4_E2M1 = 2 };

/* Execution path (gfx950 spec section 6: a path whose query-tile grid fills
 * the device versus split-KV segments plus a reduction).
 *   SPLIT_KV     CUDA-core split-KV kernel + combine, any shape.
 *   TENSOR_CORE  tcgen05 kernels over tiles of 128 packed (position, head)
 *                rows (floor(128 / g) positions of the g heads of one KV
 *                head): two tiles per CTA at d = 64 and 128, two tiles per
 *                cluster of two CTAs at d = 256; KV-split + combine when the
 *                tile grid is small; needs g <= 128.
 *   DECODE_TC    tcgen05 kernel with the keys on the MMA M dimension for
 *                calls with at most 16 packed rows per KV head: needs
 *                g * max_seqlen_q <= 16 (d = 64, 128 or 256; an fp8 cache
 *                needs d = 128).
 *   AUTO         DECODE_TC when it applies, else TENSOR_CORE when it applies
 *                and a KV head has more than 16 packed rows, else SPLIT_KV.
 * A forced path that does not apply returns UA_ERR_UNSUPPORTED. */
enum { UA_PATH_AUTO = 0, UA_PATH_SPLIT_KV = 1, UA_PATH_TENSOR_CORE = 2, UA_PATH_DECODE_TC = 3 };

/* Storage of the per-segment o partials that a KV-split call writes and the
 * combine kernel reads (gfx950 spec section 5; storing them in bf16 halves
 * their bytes and stores, as the pages' sparse decode kernel does).  m and l
 * stay fp32 either way; bf16 rounds each partial o element once (relative
 * error <= 2^-9 of that element). */
enum { UA_PARTIALS_F32 = 0, UA_PARTIALS_BF16 = 1 };

/*
 * Static description of a problem family (UnifiedAttentionProblem in the
 * gfx950 spec: one flag per bias/mask term, section 1 last paragraph and
 * section 6).  Validated by ua_problem_create.
 */
typedef struct ua_problem_desc {
    int32_t num_q_heads;        /* H_q > 0 */
    int32_t num_kv_heads;       /* H_k > 0, H_q % H_k == 0 */
    int32_t head_size;          /* d in {64, 128, 256} */
    int32_t block_size;         /* b in {16, 32, 64} */
    int64_t num_blocks;         /* physical blocks in each cache, > 0 */
    int32_t max_num_seqs;       /* upper bound on num_seqs per call, > 0 */
    int32_t max_blocks_per_seq; /* row stride of block_table, > 0 */
    int64_t max_total_q;        /* upper bound on total_q per call, > 0 */
    int32_t dtype;              /* UA_DTYPE_BF16 */
    uint32_t flags;             /* UA_FLAG_* the calls may use */
    float scale;                /* tau > 0 (usually 1/sqrt(d)) */
    float softcap;              /* c > 0 when UA_FLAG_SOFTCAP, else ignored */
    int32_t window;             /* W >= 1 when UA_FLAG_WINDOW, else ignored */
    uint32_t path;              /* UA_PATH_*: which kernel family serves the calls */
    int32_t kv_dtype;           /* UA_DTYPE_BF16, or UA_DTYPE_FP8_E4M3 (needs d = 128 and
                                   path AUTO or DECODE_TC; a ua_forward call whose
                                   shape the decode kernel does not take returns
                                   UA_ERR_UNSUPPORTED), or UA_DTYPE_FP4_E2M1 (needs
                                   path AUTO) */
    float k_scale;              /* fp8 / fp4 caches: factor of every K value, > 0; else ignored */
    float v_scale;              /* fp8 / fp4 caches: factor of every V value, > 0; else ignored */
    int32_t split_partials;     /* UA_PARTIALS_F32 (0, the default) or UA_PARTIALS_BF16 */
} ua_problem_desc;

typedef struct ua_problem ua_problem;

/*
 * Validate *desc and create a problem bound to the current CUDA device.  The
 * problem owns a device workspace (split-KV partials of fp32 (m, l, o), the
 * device error word) that is allocated here, once; ua_forward allocates
 * nothing.  (Of a bf16 cache it has room for the partials of ua_forward_tree, whether
 * it is called or not: two tiles of up to 128 rows per share of the work, about 41 MB
 * at most.)  Returns UA_ERR_INVALID_ARG for malformed fields (e.g. H_q % H_k != 0,
 * WINDOW without CAUSAL), UA_ERR_UNSUPPORTED for d or b outside the sets above or a
 * non-bf16 dtype, UA_ERR_OUT_OF_MEMORY if the workspace cannot be allocated.  *out is
 * set only on UA_OK; free it with ua_destroy.
 */
ua_status ua_problem_create(const ua_problem_desc *desc, ua_problem **out);

/*
 * Forward pass, enqueued on `stream` (a cudaStream_t; NULL = legacy default
 * stream), without host synchronisation.
 *
 * num_seqs <= max_num_seqs and num_seqs <= 65535 (else UA_ERR_UNSUPPORTED);
 * total_q = cu_seqlens_q[num_seqs] <= max_total_q;
 * max_seqlen_q / max_seqlen_k are host-side upper bounds on S_q(s) / S_k(s)
 * used to size the launch (the device checks them and reports
 * UA_DEVERR_BOUNDS).  `flags` must be a subset of the problem's flags;
 * `sinks` / `alibi_slopes` must be non-null exactly when their flag is set.
 * All array pointers are device pointers with the layouts above, `out` must
 * not alias any input, and q / out / caches must be 16-byte aligned.  `out` is
 * fully written for every row of every well-formed sequence.
 *
 * Returns UA_ERR_INVALID_ARG (nothing launched) on a contract violation the
 * host can see, UA_ERR_CUDA if a launch fails.
 */
ua_status ua_forward(ua_problem *p, const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_table, const int32_t *cu_seqlens_q,
                     const int32_t *seqused_k, int32_t num_seqs, int64_t total_q,
                     int32_t max_seqlen_q, int32_t max_seqlen_k, uint32_t flags,
                     const float *sinks, const float *alibi_slopes, void *out,
                     void *stream);

/*
 * ua_forward_topk -- sparse top-k decode ("[Triton/Gluon] [GFX950] Sparse
 * paged attention and Sparse MLA", its token-granular top-k gather): each
 * query token t attends to its own list of key positions instead of to all
 * S_k keys of its sequence,
 *
 *     O_(t,h) = sum_e softmax(x)_e V_(j_e),  j_e = topk_idx[t][e], e < topk_len[t],
 *
 * where x_e is the score chain above evaluated for key j_e (the masks, ALiBi
 * and QQ-bias use the listed position j_e).  Entries outside [0, S_k) are
 * padding (-1 by convention) and are not keys; an entry listed twice counts
 * twice.  Same arguments as ua_forward plus:
 *   topk_idx     int32 [total_q, topk_stride] device, the lists (row t = token t)
 *   topk_len     int32 [total_q] device, list lengths in [0, topk_stride];
 *                a length outside it sets UA_DEVERR_BOUNDS and writes the
 *                token's rows as 0
 *   topk_stride  > 0, entries per list row (at most 2^30)
 * A listed key in a block whose id is out of range is dropped and sets
 * UA_DEVERR_BLOCK_ID.  Needs d = 128, g <= 16, a bf16 cache, path AUTO
 * or DECODE_TC and num_blocks * b * H_k < 2^31 (else UA_ERR_UNSUPPORTED).
 * The lists are split into segments of 128-entry tiles per token (one CTA
 * each, merged by the combine kernel), counted from each token's own length.
 */
ua_status ua_forward_topk(ua_problem *p, const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_table, const int32_t *cu_seqlens_q,
                          const int32_t *seqused_k, int32_t num_seqs, int64_t total_q,
                          int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t *topk_idx,
                          const int32_t *topk_len, int32_t topk_stride, uint32_t flags,
                          const float *sinks, const float *alibi_slopes, void *out,
                          void *stream);

/*
 * Same computation with the per-step inputs and the output in HOST memory:
 * q_host, block_table_host, cu_seqlens_q_host, seqused_k_host, sinks_host and
 * alibi_host are copied to problem-owned device staging buffers (allocated on
 * first use, sized by the problem's maxima), the forward runs on `stream`, the
 * result is copied into out_host, and the call returns after `stream` has
 * drained.  The caches stay device-resident (k_cache / v_cache are device
 * pointers).  Pinned host memory makes the copies asynchronous DMA.
 */
ua_status ua_forward_host(ua_problem *p, const void *q_host, const void *k_cache,
                          const void *v_cache, const int32_t *block_table_host,
                          const int32_t *cu_seqlens_q_host, const int32_t *seqused_k_host,
                          int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q,
                          int32_t max_seqlen_k, uint32_t flags, const float *sinks_host,
                          const float *alibi_host, void *out_host, void *stream);

/*
 * Synchronise `stream`, return the device error word (UA_DEVERR_* bits) in
 * *code and clear it.  Returns UA_ERR_DEVICE when *code != 0, UA_OK otherwise.
 */
ua_status ua_check_device_error(ua_problem *p, void *stream, int32_t *code);

/*
 * Number of kernel launches the most recent ua_forward, ua_forward_host,
 * ua_forward_topk, ua_forward_weights, ua_forward_tree, ua_plan_step, ua_rope_store
 * or ua_cache_* call enqueued (for launch accounting in benchmarks).
 */
int32_t ua_last_launch_count(const ua_problem *p);

/* Human-readable name of the execution path the last of those calls took. */
const char *ua_last_path(const ua_problem *p);

/*
 * Query-query bias (gfx950 page, section 1, step 4): with UA_FLAG_QQ_BIAS a
 * call adds B[i][j - ctx] to the score of query row i (the row's index inside
 * its sequence's query chunk, 0 <= i < S_q) and key j, for the keys of the
 * query section (ctx <= j < S_k), after softcap and ALiBi and before the
 * masks.  Keys of the context (j < ctx) get no bias.  B is one fp32 matrix in
 * natural-log units, shared by every sequence and every query head; its
 * element (a, c) is bias[a * row_stride + c].
 *
 * bias: device pointer, owned by the caller, read by every later call that
 *       passes UA_FLAG_QQ_BIAS until it is replaced; NULL clears it.
 * n:    rows and columns of B that may be read; a call with the flag needs
 *       max_seqlen_q <= n (else UA_ERR_INVALID_ARG, nothing launched).
 * row_stride: elements between rows, >= n.
 * The problem must have been created with UA_FLAG_QQ_BIAS in its flags.
 * Returns UA_ERR_INVALID_ARG for n < 1 or row_stride < n with a non-NULL bias.
 */
ua_status ua_set_qq_bias(ua_problem *p, const float *bias, int64_t n, int64_t row_stride);

/*
 * Profiling hook: when both events are non-null, every later forward call
 * records `ev_begin` on its stream immediately before launching its dominant
 * kernel (the attention kernel, not the split combine) and `ev_end`
 * immediately after it, so the caller can time that kernel alone with
 * cudaEventElapsedTime.  The events (cudaEvent_t) stay owned by the caller;
 * pass NULL, NULL to switch the hook off.
 */
ua_status ua_set_profile_events(ua_problem *p, void *ev_begin, void *ev_end);

/*
 * Testing hook for the bounded-wait abort path; not for production use.
 * Every on-chip wait of the kernels is bounded (about one second); when one
 * gives up, the kernel sets UA_DEVERR_TIMEOUT, raises a CTA-wide abort flag so
 * that every role leaves its loop, waits (bounded) for the copies and
 * tensor-core operations it issued, frees its tensor memory and returns.
 * While this hook is enabled, the split, decode tensor-core, 4-bit, two-tile and
 * CTA-pair prefill kernels of later forward calls make their first
 * consumer-side K/V data wait wait on a barrier that nothing completes,
 * bounded by limit_ns instead: the wait gives up, the call returns,
 * ua_check_device_error reports UA_DEVERR_TIMEOUT, and the outputs of that
 * call are unspecified.  (In the CTA-pair kernel only the MMA-issuing CTA
 * stalls; its partner's waits give up on their normal bound.)  The waits
 * that drain a CTA's own copies and MMAs keep their normal bound.
 * enable = 0 restores normal calls.  limit_ns must lie in [1e3, 1e9] when
 * enabling (else UA_ERR_INVALID_ARG).
 */
ua_status ua_debug_stall_data_waits(ua_problem *p, int32_t enable, int64_t limit_ns);

/*
 * ua_forward_noalloc -- the split-KV forward pass without any allocation.
 * (An addition of this library; the paper has no counterpart.)
 *
 * For callers that cannot call cudaMalloc: code that lives inside a memory
 * arena owning the whole device, code running inside stream capture where an
 * allocation would break the capture, plugins that are handed only the
 * tensors of the call, and latency paths that must not enter an allocator.
 * Such callers cannot use ua_problem_create, which allocates the workspace.
 *
 * It takes the problem description by value-pointer (no ua_problem) plus the
 * same inputs and output as ua_forward, and runs the same split kernel and
 * combine kernel.  Their fp32 partials live in a 16 MiB array that the
 * library declares statically in device memory: every GPU that loads
 * libua.so holds those 16 MiB until the process exits.  Calls whose partials
 * (total_q * H_q * (d + 2) * 4 bytes per segment) do not fit twice in that
 * array return UA_ERR_UNSUPPORTED and launch nothing, as do descriptions
 * with an fp8 cache (kv_dtype != UA_DTYPE_BF16) or with UA_FLAG_QQ_BIAS
 * (the bias matrix is bound to a ua_problem).
 *
 * device_error: optional caller-owned device int32 that receives the
 * UA_DEVERR_* bits (OR-ed in; the caller clears it).  When NULL the bits go to
 * a word inside the static array, cleared at the start of each call, and are
 * not reported.
 *
 * The first call in a CUDA context resolves the array's address in that
 * context (once per context; a caller that switches contexts on one device
 * gets each context's own address); make that first call before any stream
 * capture.  All calls on a device share the array and leave their partials in
 * it: calls whose kernels may overlap on the GPU race on it and must be
 * ordered by the caller.
 *
 * desc->path must be UA_PATH_AUTO or UA_PATH_SPLIT_KV (this entry point runs
 * the split kernel only; TENSOR_CORE or DECODE_TC return UA_ERR_UNSUPPORTED,
 * a value past UA_PATH_DECODE_TC UA_ERR_INVALID_ARG); desc->max_num_seqs and
 * desc->max_total_q are not used.  num_seqs above 65535 returns
 * UA_ERR_UNSUPPORTED.
 */
ua_status ua_forward_noalloc(const ua_problem_desc *desc, const void *q, const void *k_cache,
                             const void *v_cache, const int32_t *block_table,
                             const int32_t *cu_seqlens_q, const int32_t *seqused_k,
                             int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q,
                             int32_t max_seqlen_k, uint32_t flags, const float *sinks,
                             const float *alibi_slopes, void *out, int32_t *device_error,
                             void *stream);

/*
 * ---- the cache: writing, reading back, weighing and thinning it ----
 * (Additions of this library; the pages leave the cache's writer open.)
 *
 * The calls below are asynchronous on `stream`, allocate nothing, launch
 * nothing when they return an error, need the problem's device to be current
 * and int32 and fp32 arrays on 4-byte boundaries (else UA_ERR_INVALID_ARG), and
 * report malformed metadata through the
 * problem's device error word like ua_forward.  Calls on one problem share
 * its workspace: calls (or graph replays) that may overlap on the GPU need a
 * problem each.
 *
 * ua_cache_store -- write the chunk's K and V rows into the paged caches: row
 * i of sequence s goes to key position ctx + i (ctx = S_k - S_q, the place
 * ua_forward expects it), block block_table[s][j / b], slot j % b.
 *   k_new, v_new  bf16 [total_q, H_k, d], tokens new_stride elements apart
 *                 (>= H_k * d, a multiple of 8; a slice of a fused QKV
 *                 projection), 16-byte aligned
 * By the problem's kv_dtype, with scale = k_scale or v_scale and
 * y = x / scale rounded to fp32:
 *   BF16      the bits of x;
 *   FP8_E4M3  y rounded to nearest even, magnitudes above 448 (infinities
 *             too) to 448, NaN to 0x7f;
 *   FP4_E2M1  per 16 dims s = max|y| / 6 rounded to e4m3 (nearest even, at
 *             most 448), codes y / s rounded to nearest even, at most 6 (a
 *             negative value that rounds to 0 stores the code of 0); s = 0
 *             stores zero codes; a NaN among the 16 stores s = 0x7f and zero
 *             codes, so that all 16 read back as NaN.  The rounding is that of
 *             the exact quotients.
 * Malformed sequences are skipped; rows whose block id is out of range are
 * dropped (UA_DEVERR_BLOCK_ID).  No slot may be written by two rows of a call.
 */
ua_status ua_cache_store(ua_problem *p, const void *k_new, const void *v_new, int64_t new_stride,
                         void *k_cache, void *v_cache, const int32_t *block_table,
                         const int32_t *cu_seqlens_q, const int32_t *seqused_k, int32_t num_seqs,
                         int64_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
                         void *stream);

/*
 * ua_cache_expand -- the values of the cached keys begin[s] <= j < S_k of
 * every sequence (begin NULL: from 0), the fp32 product of code, scale and
 * k_scale or v_scale rounded to bf16, into bf16 pages
 * [out_num_blocks, b, H_k, d] at block out_block_table[s][j / b] (rows of
 * out_table_stride ids), slot j % b.  A bf16 problem with these pages runs the
 * prefill kernels over what a 4-bit or fp8 cache holds.  Exact when the scale
 * is a power of two.
 *   max_keys  host-side upper bound on S_k(s) - begin(s); a sequence above
 *             it, or with begin outside [0, S_k], is skipped
 *             (UA_DEVERR_BOUNDS)
 * Rows of other keys are left as they are.  Keys whose source or destination
 * block id is out of range are dropped (UA_DEVERR_BLOCK_ID).
 */
ua_status ua_cache_expand(ua_problem *p, const void *k_cache, const void *v_cache,
                          const int32_t *block_table, const int32_t *seqused_k,
                          const int32_t *begin, int32_t num_seqs, int32_t max_keys, void *k_out,
                          void *v_out, const int32_t *out_block_table, int32_t out_table_stride,
                          int64_t out_num_blocks, void *stream);

/*
 * ua_forward_weights -- ua_forward plus the accumulated attention weight of
 * every cached key.  For a sequence with S_q >= 1 query rows, KV head k and
 * key j < S_k
 *
 *     out_w[s][k][j] = decay * in_w[s][k][j] * [j < ctx]
 *                      + sum over the rows i and the g query heads h of k of
 *                        softmax(x_(i,h))_j
 *
 * (the sink's share of a row goes to no key; an empty row adds nothing; the
 * chunk's own keys start from zero, whatever in_w holds).  Entries j >= S_k,
 * and all entries of malformed sequences or of sequences without query rows,
 * are left as they are.  Every sum has one order, so equal calls give equal
 * bits.
 *   weights_in   fp32 [num_seqs, H_k, weight_stride], or NULL for zeros (not
 *                read when decay = 0)
 *   weights_out  same layout; may be weights_in itself (else disjoint)
 *   weight_stride >= max_seqlen_k
 *   decay        finite and >= 0
 * The problem must have been created with UA_FLAG_KEY_WEIGHTS, which
 * allocates 4 * max_total_q * H_q * (max_blocks_per_seq * b, rounded up to
 * 128) bytes for the scores: size max_total_q for the steps that are weighed
 * (a decode batch, a prompt's last tokens).  Needs g <= 16 on bf16 and fp8
 * caches, path AUTO, H_k <= 65535 and max_seqlen_k <= 2^30 (else
 * UA_ERR_UNSUPPORTED).  `out` is ua_forward's up to rounding; on bf16 and fp8
 * caches a NaN or infinite V value also reaches the rows of its tile (16 / g
 * neighbouring positions) that do not see its key.
 */
ua_status ua_forward_weights(ua_problem *p, const void *q, const void *k_cache,
                             const void *v_cache, const int32_t *block_table,
                             const int32_t *cu_seqlens_q, const int32_t *seqused_k,
                             int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q,
                             int32_t max_seqlen_k, uint32_t flags, const float *sinks,
                             const float *alibi_slopes, const float *weights_in,
                             float *weights_out, int64_t weight_stride, float decay, void *out,
                             void *stream);

/*
 * ua_cache_evict -- keep at most `budget` keys of every (sequence, KV head):
 * all of them when S_k <= budget, else the last `recent` keys and the
 * budget - recent heaviest of the keys before those (ties: the lowest
 * position; NaN weighs less than anything).  The kept keys move, in their
 * order, to positions 0, 1, ... of dst_block_table, each KV head with its own
 * choice; positions afterwards are ranks, not the original positions, so
 * ALiBi and windows no longer mean distances.
 *   dst_block_table  same layout as block_table, its row stride
 *                    (max_blocks_per_seq) too.  NULL or block_table itself
 *                    evicts in place; any other table must name blocks that
 *                    block_table does not name (the sources stay as they are,
 *                    so a prefix shared with another sequence survives).
 *                    Within a table no block may be named twice, or in place
 *                    be shared.
 *   weights_in       fp32 [num_seqs, H_k, weight_stride], the weights
 *   weights_out      the kept keys' weights at their new positions (entries
 *                    past them are left as they are); may be weights_in
 *   kept             int32 [num_seqs, H_k, budget]: the kept positions,
 *                    ascending, then -1
 *   seqused_out      int32 [num_seqs]: min(S_k, budget); may be seqused_k
 *   budget >= 1, 0 <= recent <= budget, weight_stride >= max_seqlen_k
 * Needs H_k <= 32767 and max_seqlen_k <= 2^30 (else UA_ERR_UNSUPPORTED).
 * A malformed length keeps nothing (kept -1, seqused_out 0, the cache and the
 * weights as they were; UA_DEVERR_BOUNDS).  Keys whose source or destination
 * block id is out of range are not moved (UA_DEVERR_BLOCK_ID).
 */
ua_status ua_cache_evict(ua_problem *p, void *k_cache, void *v_cache, const int32_t *block_table,
                         const int32_t *dst_block_table, const int32_t *seqused_k,
                         int32_t num_seqs, int32_t max_seqlen_k, const float *weights_in,
                         float *weights_out, int64_t weight_stride, int32_t budget,
                         int32_t recent, int32_t *kept, int32_t *seqused_out, void *stream);

/*
 * ---- a step of speculative decoding: blocks and slots, rotary store, draft trees ----
 * (Additions of this library.)
 *
 * A serving step hands out blocks and slots (ua_plan_step), rotates q and k and
 * stores k and v (ua_rope_store), attends (ua_forward, or ua_forward_tree for a tree
 * of drafted tokens), and keeps the accepted branch (ua_cache_accept).  What the
 * cache calls above say about streams, workspace, alignment and errors holds here.
 *
 * A draft tree is given by its nodes' parents: int32, one row per sequence,
 * parents[s * parents_stride + i] for node i, which is the i-th query row of sequence
 * s.  A parent stands in front of its children; -1 marks a node without one (there may
 * be several).  A tree has at most 1024 nodes.
 *
 * ua_plan_step -- give the sequences of a step their blocks and tokens.  Sequence s
 * has ctx_lens[s] cached keys and wants new_lens[s] more; it needs
 * ceil((ctx + new) / b) blocks.
 *   block_table    int32 [num_seqs, max_blocks_per_seq], in and out: ids of new blocks
 *                  are written behind the held ones
 *   blocks_held    int32 [num_seqs], in and out: blocks that the sequences have
 *   free_blocks    int32 [num_blocks], in and out: a stack of *free_count block ids
 *   free_count     int32 [1], in and out
 * Sequences that hold more than they need give their last blocks back, and these lie on
 * the stack with the first of them on top (first sequence, lowest position); then
 * sequences in their order take what they lack from the top.  A sequence that needs
 * more blocks than are left, counting what those in front of it asked for, gets no
 * tokens and keeps what it has; sequences that need no further block are served always.
 * Of the served ones those get tokens whose last one is within max_tokens, counting the
 * tokens of all served ones in front.
 * (A finished request passes ctx = new = 0, rejected drafts simply a smaller ctx in
 * the next step.  A step that is followed by one with new = 0 leaves the pool as it
 * was.)
 *   parents        draft trees of the new tokens, parents_stride >= their number; or
 *                  NULL: chains
 *   granted        int32 [num_seqs] out: new_lens[s], or 0; may be new_lens
 *   cu_seqlens_q   int32 [num_seqs + 1] out: prefix sums of granted
 *   seqused_k      int32 [num_seqs] out: ctx + granted; may be ctx_lens
 *   positions      int32 [max_tokens] out: ctx + depth in the tree (a chain: ctx + i) of
 *                  every packed token
 *   slots          int64 [max_tokens] out: block * b + slot of every packed token's key
 *   tree_mask      uint32 [max_tokens, mask_stride] out, or NULL: bit c % 32 of word
 *                  c / 32 of a token's row is set for the nodes c on its branch; rows of
 *                  tokens that are not there are left as they are
 *   max_tokens     host-side bound on the tokens, <= max_total_q; places behind the last
 *                  token get position 0 and slot -1
 * Malformed lengths (negative, past max_blocks_per_seq * b, past parents_stride or 32 *
 * mask_stride) get nothing and seqused_k = 0; these and tokens past max_tokens are
 * reported (UA_DEVERR_BOUNDS).  A bad block id gives the slot -1 and is reported, also
 * where it is given back (UA_DEVERR_BLOCK_ID; it goes to the pool all the same), a bad
 * parent ends its branch (UA_DEVERR_TREE).
 * Needs num_seqs <= 16384 (else UA_ERR_UNSUPPORTED).  Arrays may not overlap otherwise.
 */
ua_status ua_plan_step(ua_problem *p, int32_t *block_table, int32_t *blocks_held,
                       int32_t *free_blocks, int32_t *free_count, const int32_t *ctx_lens,
                       const int32_t *new_lens, const int32_t *parents, int64_t parents_stride,
                       int32_t num_seqs, int64_t max_tokens, int32_t *granted,
                       int32_t *cu_seqlens_q, int32_t *seqused_k, int32_t *positions,
                       int64_t *slots, uint32_t *tree_mask, int32_t mask_stride, void *stream);

/* Which dims of a head form a rotated pair, with n frequencies. */
enum {
    UA_ROPE_HALF = 0,    /* (i, i + n) */
    UA_ROPE_PAIRS = 1    /* (2i, 2i + 1) */
};

/*
 * ua_set_rope -- the rotary frequencies of later ua_rope_store calls: inv_freq[i]
 * (host array, radians per position, 0 <= inv_freq[i] <= 6) for pair i < n, where 2n is
 * the number of rotated dims: a multiple of 16, at most d (else UA_ERR_UNSUPPORTED).
 * Scalings for long contexts are other frequencies and, where they have one, a factor
 * `magnitude` (finite) on cos and sin.  The values are copied; calls that were captured
 * into a graph keep those they were captured with.
 */
ua_status ua_set_rope(ua_problem *p, const double *inv_freq, int32_t n, uint32_t layout,
                      float magnitude);

/*
 * ua_rope_store -- rotate q and k by the tokens' positions and write k and v into the
 * caches.  A pair (x, y) with angle phi = position * inv_freq[i] becomes
 *     magnitude * (x cos phi - y sin phi, x sin phi + y cos phi)
 * in fp32, rounded once to bf16; other dims stay.  The angle's fraction of a turn is off
 * by 2^-25 at most, at any position (the frequency is taken to 2^-65 of a turn per
 * position, the fraction becomes an fp32 number).  Keys are then stored like
 * ua_cache_store does, from the rounded values.
 *   q              bf16 [total_q, H_q, d], tokens q_stride elements apart
 *   k_new, v_new   bf16 [total_q, H_k, d], tokens kv_stride elements apart
 *   q_out          bf16 [total_q, H_q, d], tokens out_stride elements apart; q itself
 *                  with the same stride, or disjoint from every input
 *   positions      int32 [total_q]
 *   slots          int64 [total_q]: block * b + slot; negative: k and v are not stored
 *                  (q is rotated all the same).  A slot past the cache is dropped
 *                  (UA_DEVERR_BLOCK_ID); no slot may be named twice
 * Strides are multiples of 8 and at least a token's row; q, k_new, v_new, q_out and the
 * caches are 16-byte aligned.  ua_set_rope comes first (else UA_ERR_INVALID_ARG).
 */
ua_status ua_rope_store(ua_problem *p, const void *q, int64_t q_stride, const void *k_new,
                        const void *v_new, int64_t kv_stride, const int32_t *positions,
                        const int64_t *slots, int64_t total_q, void *q_out, int64_t out_stride,
                        void *k_cache, void *v_cache, void *stream);

/*
 * ua_forward_tree -- ua_forward where a query row sees all ctx keys of its context and,
 * of its chunk's own keys, those that its row of tree_mask names: bit c % 32 of word
 * c / 32 stands for key ctx + c, c < S_q.  Any mask will do; a row that sees nothing
 * gets O = 0.
 *   tree_mask      uint32 [total_q, mask_stride], 32 * mask_stride >= max_seqlen_q
 *   positions      int32 [total_q], positions of the query rows, within [ctx, S_k)
 *                  (others are moved there, UA_DEVERR_TREE); needed with
 *                  UA_FLAG_WINDOW or UA_FLAG_ALIBI, else not read.  A context key's
 *                  position is j, a chunk key's that of its row: the window keeps keys
 *                  from position(row) - W + 1 on, ALiBi adds slope * (position - ctx)
 * The mask takes the place of the causal rule: flags must have UA_FLAG_CAUSAL (else
 * UA_ERR_INVALID_ARG); UA_FLAG_QQ_BIAS is not served (UA_ERR_UNSUPPORTED).  Needs path
 * AUTO, g <= 128, max_seqlen_q <= 1024, max_seqlen_k <= 2^30 and H_k <= 65535 (else
 * UA_ERR_UNSUPPORTED).  A value that is not finite reaches the rows that see its key and
 * no others.  Equal calls give equal bits.
 */
ua_status ua_forward_tree(ua_problem *p, const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_table, const int32_t *cu_seqlens_q,
                          const int32_t *seqused_k, int32_t num_seqs, int64_t total_q,
                          int32_t max_seqlen_q, int32_t max_seqlen_k, const uint32_t *tree_mask,
                          int32_t mask_stride, const int32_t *positions, uint32_t flags,
                          const float *sinks, const float *alibi_slopes, void *out, void *stream);

/*
 * ua_cache_accept -- keep one branch of every draft tree: the nodes from the root to
 * last[s].  With the branch r_0 < r_1 < ... the K and V rows of key ctx + r_t move to
 * key ctx + t, where ctx = S_k - S_q; other rows are left as they are.  (Keys stored by
 * ua_rope_store with a node's position are rotated for where they arrive.)
 *   parents        the trees, parents_stride >= max_seqlen_q
 *   last           int32 [num_seqs]: the deepest accepted node, -1: none; not read for
 *                  sequences without query rows
 *   path           int32 [num_seqs, path_stride] out: r_0, r_1, ..., then -1
 *   accepted       int32 [num_seqs] out: length of the branch
 *   seqused_out    int32 [num_seqs] out: ctx + accepted; may be seqused_k
 * A bad parent or last node accepts nothing (UA_DEVERR_TREE), nor does a branch longer
 * than path_stride (UA_DEVERR_BOUNDS); malformed lengths get seqused_out 0.  Rows whose
 * block id is out of range are not moved (UA_DEVERR_BLOCK_ID).  Needs max_seqlen_q <=
 * 1024 (else UA_ERR_UNSUPPORTED).
 */
ua_status ua_cache_accept(ua_problem *p, void *k_cache, void *v_cache, const int32_t *block_table,
                          const int32_t *cu_seqlens_q, const int32_t *seqused_k,
                          const int32_t *parents, int64_t parents_stride, const int32_t *last,
                          int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q,
                          int32_t max_seqlen_k, int32_t *path, int32_t path_stride,
                          int32_t *accepted, int32_t *seqused_out, void *stream);

/* Free the workspace and the problem.  NULL is a no-op. */
void ua_destroy(ua_problem *p);

/* Static string for a status code. */
const char *ua_status_string(ua_status s);

/* Text of the last CUDA error seen by this thread inside the library. */
const char *ua_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* UA_H_ */
