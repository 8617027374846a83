// ffn.h -- kernel arguments and launchers of the feed-forward operators (the
// gated block, its backward pass, the scaled INT8 product, row quantization),
// shared by their plans and kernels.
#pragma once

#include "internal.h"

namespace mm {

// Operands of the tiled products (k_ffn.h) and the few-row kernels
// (k_ffn_rows.hip).  A and B hold two matrices where the mode has two.
struct FfnArgs {
    const void *A[2];
    const void *B[2];
    void *Y[2];
    void *G, *U;           // gated block: where to keep A B0 and A B1 (NULL: nowhere)
    int64_t M, N, K;
    int64_t lda, ldb, ldy;  // row pitches of the stored operands and of Y, G, U
    int64_t batch;         // products (kScaled), or 2 for a pair
    int32_t act;
    int32_t y_vec;         // output rows are whole, aligned 16-byte chunks
    // scaled INT8 product
    const float *sa, *sb;
    const void *bias;      // of the output type, or NULL
    void *W;               // partial sums [split][batch][M][N], INT32 (INT8 operands) or FP32
    int32_t split;
    int32_t kstages;       // K stages of a partition
    BatchDesc bd;
};

// Tile table of the tiled products: block rows and columns (the gated
// block's columns count gate and up) and the bytes of K in a stage, see
// k_ffn.h.
struct FfnTile {
    int bm, bn, bkb;
};
constexpr FfnTile kFfnTiles[] = {{256, 256, 64}, {128, 128, 64}, {64, 128, 128}, {32, 128, 256}, {256, 128, 128}};
constexpr int kNumFfnTiles = sizeof(kFfnTiles) / sizeof(kFfnTiles[0]);

// Element-wise part of the gated block's backward pass: dG = dH * U * f'(G),
// dU = dH * f(G).  G, U, dH are dense [M, N]; dG, dU have rows of ldw elements
// (whole 16-byte chunks, 16-byte aligned), zero past N.
hipError_t launch_glu_dact(int dtype, int act, const void *G, const void *U, const void *dH, void *dG, void *dU,
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
hipError_t launch_glu_rows(int dtype, bool tb, const FfnArgs &a, hipStream_t s);
bool rows_quantize(int a_type, int out_dtype, bool tb, int64_t M, int64_t K, int64_t N);
hipError_t launch_scaled_rows(int out_dtype, bool tb, bool quant, const FfnArgs &a, hipStream_t s);
// Row quantization of a dense [rows, cols] matrix into rows of ldq bytes; the
// bytes past cols are set to zero.
hipError_t launch_quantize_rows(int dtype, const void *X, int64_t rows, int64_t cols, void *Q, int64_t ldq, float *scale,
                                hipStream_t s);

}  // namespace mm
