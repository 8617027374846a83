// plan.h -- the plan object behind mm_plan_t.
#pragma once

#include <stdarg.h>
#include <stdint.h>

#include <mutex>

#include "internal.h"

namespace mm {
// Tile entry and split of one tiled product of the feed-forward operators.
struct FfnChoice {
    int tile = 0;
    int32_t split = 1;
    int32_t kstages = 0;  // K stages of a partition
    double us = 0.0;      // estimated time
};
}  // namespace mm

struct mm_plan_s {
    int dtype = 0;
    int a_rank = 0, b_rank = 0;
    int64_t a_shape[MM_MAX_RANK] = {};
    int64_t b_shape[MM_MAX_RANK] = {};
    int out_rank = 0;
    int64_t out_shape[MM_MAX_RANK] = {};
    int64_t out_numel = 0;
    int64_t M = 0, N = 0, K = 0;  // promoted sizes of one product
    int64_t total_batch = 0;      // broadcast batch count before folding
    int64_t batch = 0;            // products launched (1 when folded)
    int64_t kernel_m = 0;         // rows per launched product
    int folded = 0;
    mm::BatchDesc bd = {};
    int algo = MM_ALGO_EMPTY;
    int tile = -1;  // tile table index (tiled algorithms)
    // GENERAL only: when tail_col > 0, the tile `tile` covers output columns
    // [0, tail_col) in whole rounds of workgroups and a second launch with
    // tile `tail_tile` covers [tail_col, N).
    int64_t tail_col = 0;
    int tail_tile = -1;
    int32_t split = 1;
    int64_t kchunk = 0;
    int64_t workspace_bytes = 0;

    // Device workspace for split-K and a split skinny-M, allocated by plan
    // creation on the current device (by the first execution when creation
    // found no GPU).
    std::mutex ws_mutex;
    void *ws = nullptr;
    int ws_device = -1;

    // Gemm (mm_gemm_plan_create): transposed operands, epilogue, C layout.
    bool is_gemm = false;
    int ta = 0, tb = 0;
    float alpha = 1.0f, beta = 0.0f;
    int c_mode = 0;  // mm::GemmBias
    int64_t ldc = 0;

    // MatMulInteger (mm_int_plan_create): operand types, zero-point kinds and
    // the row / column sums the zero points need (formed by the tiled kernel).
    bool is_int = false;
    int a_type = 0, b_type = 0;
    int zpa_kind = 0, zpb_kind = 0;
    bool need_ra = false, need_cb = false;

    // Scaled INT8 product (mm_scaled_int_plan_create): dtype is the output
    // type, a_type the type of A as given; tb says how B is stored.  An A to
    // be quantized goes to the workspace: its rows (q_pitch bytes each, at
    // q_off), then its scales (at qs_off); split partials lie before it.
    bool is_scaled = false;
    bool has_bias = false;
    bool fused_quant = false;  // the few-row kernel quantizes A itself
    int64_t a_rows = 0;  // rows of the whole A tensor
    int64_t q_pitch = 0, q_off = 0, qs_off = 0;

    // Gated feed-forward block (mm_glu_plan_create): tb is trans_w, M, N, K
    // are rows, hidden, in_features.  The workspace holds a split forward
    // pass's partials, then (training, at d_off) dG and dU with rows of
    // d_pitch elements, d_bytes each, and a split backward product's partials.
    bool is_glu = false;
    int act = 0;
    bool training = false;
    int kept = 0;          // type of G and U
    int64_t w_pitch = 0, d_off = 0, d_pitch = 0, d_bytes = 0;
    mm::FfnChoice dx, dw;  // the backward products
    int32_t kstages = 0;   // K stages of a partition (scaled product, forward pass)

    // Plan-owned constant B (mm_plan_set_constant_b).
    std::mutex cb_mutex;
    bool cb_set = false;
    void *cb = nullptr;
    int cb_device = -1;
    int64_t b_numel = 0;  // elements of the planned B tensor
    // The same B prepacked for the tiled 16-bit kernel (see KArgs::Bp): the
    // columns of `tile` (all of N, or [0, tail_col)) then those of
    // `tail_tile`, cbp_main and cbp_tail bytes per B matrix.
    void *cbp = nullptr;
    size_t cbp_bytes = 0;
    bool cbp_ok = false;
    int64_t cbp_main = 0, cbp_tail = 0;
};

namespace mm {
// Allocate the plan's split workspace on the current device (execute.cpp).
// At creation a host without a GPU is not an error: the first execution
// allocates instead.
mm_status alloc_workspace(mm_plan_s *p, bool at_create);
// Enqueue a MatMul or Gemm plan (C: the Gemm bias or NULL); split partial
// sums go to `ws` when it is not NULL, else to the plan's workspace.
// packed_b: read B's prepacked copy (the plan's constant B) where the tiled
// 16-bit kernel runs; B must then be the plan's row-major constant B.
mm_status execute_plan(mm_plan_s *p, const void *A, const void *B, const void *C, void *Y, void *stream, void *ws,
                       bool packed_b = false);
// Resolve MatMul shapes, strides, collapse and fold into `p`, and check the
// sizes the kernels index (plan.cpp).
mm_status resolve(const int64_t *a_shape, int a_rank, const int64_t *b_shape, int b_rank, mm_plan_s *p);
mm_status check_limits(const mm_plan_s *p);
// MM_OK for a plan of MatMul; MM_ERR_BAD_OPTION naming the call that runs it
// for any other (execute.cpp).
mm_status require_matmul(const mm_plan_s *p);
mm_status fail(mm_status st, const char *fmt, ...);
void clear_error();
int elem_size(int dtype);
}  // namespace mm
