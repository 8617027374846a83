// ffn.h -- kernel arguments and launchers of the feed-forward operators (the
// gated block, its backward pass, the scaled INT8 product, row quantization),
// shared by their plans and kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "internal.h"

namespace mm {

// One call's operands, as the plans give them to the launchers.  A and B hold
// two matrices where the mode has two.
struct FfnArgs {
    const void *A[2];
    const void *B[2];
    void *Y[2];
    void *G, *U;           // gated block: where to keep A B0 and A B1 (NULL: nowhere)
    int64_t M, N, K;       // below 2^31, like the pitches
    int64_t lda, ldb, ldy;  // row pitches of the stored operands and of Y, G, U
    int64_t batch;         // products (scaled), or 2 for a pair
    int32_t act;
    int32_t y_vec;         // output rows are whole, aligned 16-byte chunks
    int32_t kept_vec;      // gated block: so are those of G and U,
    int32_t kept32;        // which are FP32 in a 16-bit plan
    // scaled INT8 product
    const float *sa, *sb;
    const void *bias;      // of the output type, or NULL (the linear layer's too)
    void *W;               // partial sums [split][batch][M][N], INT32 (INT8 operands) or FP32
    int32_t split;
    int32_t kstages;       // K stages of a partition
    BatchDesc bd;
    // linear layer: Z goes to G (kept32: FP32; q8: a checkpoint with its scale
    // bytes in zs), the residual is read from R
    const void *R;
    void *zs;
    int32_t q8;
    int32_t r_vec;         // rows of R are whole, aligned 16-byte chunks
};

// The same as the kernels take it: in 88 bytes, because a launch with more
// than about 100 bytes of arguments takes 0.8-1.1 us longer (2.8 us with 96,
// 3.5 with 128, 3.8 with 384), which a decoded token's call feels.  Slots that
// a mode leaves free hold what others need; the names below say which.
struct FfnSlim {
    const void *A[2];
    const void *B[2];
    void *Y[3];
    int32_t M, N, K, lda, ldb, ldy;
    int32_t kstages;
    uint16_t split;
    uint8_t act, flags;
    __host__ __device__ bool y_vec() const { return flags & 1; }
    __host__ __device__ bool kept_vec() const { return flags & 2; }
    __host__ __device__ bool kept32() const { return flags & 4; }
    __host__ __device__ void *G() const { return Y[1]; }  // gated block
    __host__ __device__ void *U() const { return Y[2]; }
    __host__ __device__ bool q8() const { return flags & 8; }  // linear layer: Z in G()
    __host__ __device__ bool r_vec() const { return flags & 16; }
    __host__ __device__ const void *R() const { return Y[2]; }
    __host__ __device__ void *zs() const { return (void *)A[1]; }
    __host__ __device__ const void *lin_bias() const { return B[1]; }
    __host__ __device__ const float *sa() const { return (const float *)A[1]; }  // scaled product
    __host__ __device__ const float *sb() const { return (const float *)B[1]; }
    __host__ __device__ const void *bias() const { return Y[1]; }
    __host__ __device__ void *part() const { return Y[0]; }     // split products write their partial sums instead of Y
    __host__ __device__ const void *W() const { return A[0]; }  // reductions read them
};
static_assert(sizeof(FfnSlim) == 88, "FfnSlim");
struct FfnSlimBatch : FfnSlim {  // scaled products over several batches
    int64_t batch;
    BatchDesc bd;
};

// Tile table of the tiled products: block rows and columns (the gated
// block's columns count gate and up) and the bytes of K in a stage, see
// k_ffn.h.  A smaller tile gives few-row and narrow products more workgroups
// and costs more LDS and cache reads for each MFMA: 32 bytes of K take 0.41 us
// on 256 x 256 (8 waves of 128 x 64), 0.24 on 256 x 128, 0.17 on 128 x 128 (0.285
// for two of them on a CU), 0.147 on 64 x 128 (two K groups) and 0.095 on 32 x 128
// (four), so plans choose by the time model in plan_ffn.cpp.  Four waves of 128 x
// 64 on 256 x 128 need fewer LDS reads than the eight of 64 x 64 but leave a
// SIMD one wave: 265 against 201 us at 4096 x 2048 x 5504, gated.
struct FfnTile {
    int bm, bn, bkb;
};
constexpr FfnTile kFfnTiles[] = {{256, 256, 64}, {128, 128, 64}, {64, 128, 128}, {32, 128, 256}, {256, 128, 128}};
constexpr int kNumFfnTiles = sizeof(kFfnTiles) / sizeof(kFfnTiles[0]);

// Kernel arguments of a product (glu, scaled, linear: which slots it needs), of a
// split one (its partial sums) and of its reduction.
enum FfnUse { kUsePlain, kUseGlu, kUseScaled, kUseLinear };
template <class T>
inline T slim_args(const FfnArgs &a, FfnUse use, bool split, bool reduce) {
    T s = {};
    for (int i = 0; i < 2; ++i) {
        s.A[i] = a.A[i];
        s.B[i] = a.B[i];
        s.Y[i] = a.Y[i];
    }
    s.M = (int32_t)a.M;
    s.N = (int32_t)a.N;
    s.K = (int32_t)a.K;
    s.lda = (int32_t)a.lda;
    s.ldb = (int32_t)a.ldb;
    s.ldy = (int32_t)a.ldy;
    s.kstages = a.kstages;
    s.split = (uint16_t)a.split;
    s.act = (uint8_t)a.act;
    s.flags = (uint8_t)((a.y_vec ? 1 : 0) | (a.kept_vec ? 2 : 0) | (a.kept32 ? 4 : 0) | (a.q8 ? 8 : 0) |
                        (a.r_vec ? 16 : 0));
    if (use == kUseGlu) {
        s.Y[1] = a.G;
        s.Y[2] = a.U;
    } else if (use == kUseScaled) {
        s.A[1] = a.sa;
        s.B[1] = a.sb;
        s.Y[1] = (void *)a.bias;
    } else if (use == kUseLinear) {
        s.A[1] = a.zs;
        s.B[1] = a.bias;
        s.Y[1] = a.G;
        s.Y[2] = (void *)a.R;
    }
    if (split) s.Y[0] = a.W;
    if (reduce) s.A[0] = a.W;
    return s;
}
inline FfnSlimBatch slim_batch(const FfnArgs &a, bool split, bool reduce) {
    FfnSlimBatch s = slim_args<FfnSlimBatch>(a, kUseScaled, split, reduce);
    s.batch = a.batch;
    s.bd = a.bd;
    return s;
}

// Element-wise part of the gated block's backward pass: dG = dH * U * f'(G),
// dU = dH * f(G).  G, U (of type `kept`: dtype or MM_FLOAT) and dH are dense
// [M, N]; dG, dU have rows of ldw elements (whole 16-byte chunks, 16-byte
// aligned), zero past N.
hipError_t launch_glu_dact(int dtype, int kept, int act, const void *G, const void *U, const void *dH, void *dG, void *dU,
                           int64_t M, int64_t N, int64_t ldw, hipStream_t s);
// Tiled products (vec: every operand row and base is 16-byte aligned; split:
// partial sums to W, to be joined by the matching reduction; the gated
// block's are [split][G, U][M][N]).
hipError_t launch_glu_fwd(int dtype, bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);
hipError_t launch_glu_reduce(int dtype, const FfnArgs &a, hipStream_t s);
hipError_t launch_glu_dx(int dtype, bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);
hipError_t launch_glu_dw(int dtype, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);
hipError_t launch_sum_reduce(int dtype, const FfnArgs &a, hipStream_t s);
hipError_t launch_scaled(int out_dtype, bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s);
hipError_t launch_scaled_split(bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s);
hipError_t launch_scaled_reduce(int out_dtype, const FfnArgs &a, hipStream_t s);
// Few-row kernels (any alignment, at most kFfnRows rows, one product).
// rows_quantize: whether the scaled one takes A in its own type and quantizes
// it itself (`quant`); its INT8 rows then fit kFfnQuantLds bytes of LDS.
constexpr int kFfnRows = 32;
constexpr int kFfnQuantLds = 48 * 1024;
// Workgroups of [K, N] weights take 64 columns (the gated block: 32 of each
// matrix), and half as many as long as all still start at once: a workgroup
// reads its columns at what one CU gets from memory, which more CUs multiply,
// but row pieces below 64 bytes cost more than they bring once every CU has
// one (M = 1, K = 4096, INT8: N = 4096 with 64, 32 and 16 columns 10.9, 9.4 and
// 7.8 us, N = 1024 9.5, 7.9 and 6.1, N = 11008 10.8, 14.7 and 18.3; BF16 gated,
// forced, N = 4096 with 32 and 16: 31.3 and 27.4, N = 11008: 53.5 and 62.3, where
// plans take split tiles, 22.6 us, and tiles, 50.3).  A lane's pieces shrink with
// the columns (8, 4, 2 in flight): the narrow forms are bound by latency, 24 x
// 4096 x 4096 INT8 9.6 us at 1.85 TB/s.
inline bool rows_halve(int64_t wgs) { return 2 * wgs <= kNumCUs; }
hipError_t launch_glu_rows(int dtype, bool tb, const FfnArgs &a, hipStream_t s);
bool rows_quantize(int a_type, int out_dtype, bool tb, int64_t M, int64_t K, int64_t N);
hipError_t launch_scaled_rows(int out_dtype, bool tb, bool quant, const FfnArgs &a, hipStream_t s);
// Linear layer: the forward products (also dX's, which has no epilogue), the
// joining of a split one with the epilogue, the few-row kernel; dW (batch 1).
hipError_t launch_linear(int dtype, bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);
hipError_t launch_linear_dw(int dtype, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);
hipError_t launch_linear_reduce(int dtype, const FfnArgs &a, hipStream_t s);
hipError_t launch_linear_rows(int dtype, bool tb, const FfnArgs &a, hipStream_t s);

// What a linear layer's backward products need first: dZ = dY f'(Z) (act; rows
// of ldz elements, zeros past N), the column sums of dZ over each block of
// `rows` rows (part, rows of ldp floats), and a checkpoint's values f(q s) as
// rows of ldx elements (zeros past K).  NULL dZ, part, X: not wanted.
struct LinearPrep {
    const void *dY, *Z, *zs;
    void *dZ;
    float *part;
    const void *xq, *xs;
    void *X;
    int64_t M, N, ldz, ldp, K, ldx;
    int32_t act, z_type, x_act, rows;
};
// Rows of a block: 64, or fewer (whole eights) while the GPU has two blocks for
// each CU (300 x 1364 FP32 gelu: 14.7 us with 64, 5 with 8).
inline int linear_prep_rows(int64_t M, int64_t N, int dtype) {
    const int64_t cols = 32 * (dtype == MM_FLOAT ? 4 : 8), blocks = (N + cols - 1) / cols;
    int rows = 64;
    while (rows > 8 && (M + rows - 1) / rows * blocks < 2 * kNumCUs) rows /= 2;
    return rows;
}
hipError_t launch_linear_prep(int dtype, const LinearPrep &a, hipStream_t s);
int64_t linear_prep_blocks(const LinearPrep &a, int dtype);

// out[n] = sum over p < P of part[p * ldp + n], n < N; ldp is a multiple of four.
struct JoinArgs {
    const float *part;
    int64_t P, ldp, N;
    void *out;
};
hipError_t launch_join(int dtype, const JoinArgs &a, hipStream_t s);

// Checkpoints (the format stands in checkpoint.h).
hipError_t launch_checkpoint_pack(int dtype, const void *X, int64_t rows, int64_t cols, void *q, void *scale, hipStream_t s);
hipError_t launch_checkpoint_unpack(int dtype, const void *q, const void *scale, int64_t rows, int64_t cols, void *X,
                                    hipStream_t s);

// Row quantization of a dense [rows, cols] matrix into rows of ldq bytes; the
// bytes past cols are set to zero.
hipError_t launch_quantize_rows(int dtype, const void *X, int64_t rows, int64_t cols, void *Q, int64_t ldq, float *scale,
                                hipStream_t s);

}  // namespace mm
