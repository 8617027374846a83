// norm.h -- kernel arguments and launchers of the fused norms, shared by their
// plan and kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "internal.h"

namespace mm {

// Forward pass of inference, in 100 bytes (see FfnSlim); NULL: absent.
struct NormFwd {
    const void *X, *B, *gate, *w1, *b1, *w2, *b2;
    void *R, *Y;
    int32_t M, N, gate_rows;
    float alpha, eps1, eps2;
    uint8_t post, pre, pad[2];  // MM_NORM_* of B and R
};
// A training plan's: statistics and checkpoints too.
struct NormFwdTrain : NormFwd {
    float *stats, *r32;
    void *rq, *rs, *bq, *bs, *yq, *ys;
};

// Rows of the backward pass are dealt to workers, `per` consecutive ones each;
// a worker keeps its columns' sums over them in registers.  part: [workers][jobs]
// [ldp] floats, the sums of dpost_weight, dpre_weight, dpost_bias, dpre_bias as far
// as they are wanted; gpart: [workers][2][ldp], of dgate for the worker's first and
// second group of gate rows (NULL: per is a multiple of gate_rows, and every
// group is finished by one worker).
struct NormBwd {
    const float *stats;
    const void *R, *rs, *B, *bs, *gate, *w1, *b1, *w2, *dY, *dS;
    void *dX, *dB, *dgate;
    float *part, *gpart;
    int64_t ldp;
    int32_t M, N, gate_rows, per, workers, jobs;
    float alpha;
    int8_t slot[4];  // of each sum, -1: not wanted
    uint8_t post, pre;
};
struct NormJoin {
    const float *part, *gpart;
    int64_t ldp;
    int32_t M, N, gate_rows, per, workers, jobs, groups;
    void *out[4];  // by slot
    void *dgate;
};

// Threads that share a row of N columns in the backward pass, and rows that a
// workgroup takes at once.
inline int norm_bwd_threads(int64_t N) {
    return N <= 64 * 8 ? 64 : N <= 128 * 8 ? 128 : N <= 256 * 8 ? 256 : N <= 512 * 8 ? 512 : 1024;
}
// A wave that has a row to itself shares a workgroup with three others.
constexpr int norm_bwd_block(int threads) { return threads == 64 ? 256 : threads; }
inline int norm_bwd_rows(int64_t N) { return norm_bwd_block(norm_bwd_threads(N)) / norm_bwd_threads(N); }

hipError_t launch_norm_fwd(int dtype, bool train, const NormFwdTrain &a, hipStream_t s);
// kept: what R and B are given in (dtype; MM_FLOAT: R in FP32; MM_INT8: checkpoints).
hipError_t launch_norm_bwd(int dtype, int kept, const NormBwd &a, hipStream_t s);
hipError_t launch_norm_join(int dtype, const NormJoin &a, hipStream_t s);

}  // namespace mm
