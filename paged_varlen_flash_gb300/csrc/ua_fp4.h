// ua_fp4.h -- launchers of the attention kernels over 4-bit (e2m1) caches (internal).
#pragma once

#include "ua_common.cuh"

namespace ua {

struct Fp4Plan {
    int rows = 16;   // packed rows per tile (8 or 16)
    int ctas = 1;    // CTAs; each warp has an equal share of the batch's keys
    int splits = 2;  // partial slots per row: the most pieces a job may be cut into
    int chunk = 1;   // smallest share, in steps of 32 keys
};

// Bytes of one partial slot for `rows` output rows; a problem's workspace
// holds at least two.
size_t fp4_workspace_bytes(int64_t rows, int d);

// False when the call does not fit.
bool plan_fp4(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4Plan* plan);

// Enqueue the kernel and the merge of cut jobs (p.splits / p.chunk from the plan;
// p.part_o, p.piece_ml and p.row_pieces the problem's workspace).  With p.scores set every
// row's scores and its final (m, l), the latter in p.part_ml, are stored as well.
cudaError_t launch_fp4(const Fp4Plan& plan, const FwdParams& p, cudaStream_t stream);

// Calls with at least this many packed rows per KV head go to the tcgen05
// kernel (tiles of 128 rows), the others to the register-operand one.  Measured
// (us, register / tcgen05): 16 sequences of 4096 keys, 8 KV heads, d = 128, 16
// rows 43 / 49, 32 rows 59 / 49, 64 rows 100 / 49; 4 of 30000, 2 heads, d = 256,
// 16 rows 58 / 78, 32 rows 86 / 80; 32 of 2000, 2 heads, d = 64, 32 rows 24 / 27,
// 64 rows 31 / 27.  One limit for every d: at d = 64 the crossing lies between 32
// and 64 rows, and calls between pay up to 12 % for it.  The choice is the call's,
// by its longest chunk: a batch of single tokens with one chunk in it takes
// 128-row tiles for all.
constexpr int kFp4RowsMin = 25;

struct Fp4RowsPlan {
    int tiles = 1;   // row tiles per (sequence, kv head)
    int splits = 1;  // KV segments of each
    int chunk = 0;   // keys per segment (a multiple of 128)
};

// False when the call does not suit the tcgen05 kernel.
bool plan_fp4_rows(const FwdParams& p, int num_sms, size_t workspace_bytes, Fp4RowsPlan* plan);

// Enqueue it (p.splits / p.chunk / partial pointers set from the plan).  With
// p.scores set partials are written even for one segment (scores are not).
cudaError_t launch_fp4_rows(const Fp4RowsPlan& plan, const FwdParams& p, cudaStream_t stream);

}  // namespace ua
