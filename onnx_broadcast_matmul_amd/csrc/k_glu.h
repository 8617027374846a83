// k_glu.h -- the gated feed-forward block's tiled products for one element
// type (instantiated by k_glu_f32.hip, k_glu_f16.hip and k_glu_bf16.hip):
//
//   forward    H = f(G) * U, G = X Wg, U = X Wu: one pass over X; every wave
//              holds the gate and the up accumulators of the same outputs, so
//              the activation and the product happen in registers.
//   dX         = dG Wg^T + dU Wu^T: both terms in one K loop.
//   dWg, dWu   = X^T dG, X^T dU (or their transposes): one launch.
#pragma once

#include "k_ffn.h"

namespace mm {

template <int DT, bool TB>
static hipError_t glu_fwd(int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    switch (tile) {
    case 0:
        if constexpr (DT != MM_FLOAT) return launch_ffn<DT, DT, kGlu, false, TB, 256, 256, 2, 4, 64, 4, 8>(vec, a, s);
        else return hipErrorInvalidValue;
    case 1: return launch_ffn<DT, DT, kGlu, false, TB, 128, 128, 2, 2, 64, 4, 4>(vec, a, s);
    case 2: return launch_ffn<DT, DT, kGlu, false, TB, 64, 128, 2, 2, 64, 4, 4>(vec, a, s);
    case 3: return launch_ffn<DT, DT, kGlu, false, TB, 32, 128, 1, 2, 64, 4, 2>(vec, a, s);
    }
    return hipErrorInvalidValue;
}

template <int DT, int MODE, bool TA, bool TB>
static hipError_t glu_bwd(int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    switch (tile) {
    case 0:
        if constexpr (DT != MM_FLOAT) return launch_ffn<DT, DT, MODE, TA, TB, 256, 256, 2, 4, 64, 4, 8>(vec, a, s);
        else return hipErrorInvalidValue;
    case 1: return launch_ffn<DT, DT, MODE, TA, TB, 128, 128, 2, 2, 64, 4, 4>(vec, a, s);
    }
    return hipErrorInvalidValue;
}

#define MM_GLU_INSTANCE(DT, NAME)                                                                           \
    hipError_t glu_fwd_##NAME(bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s) {                \
        return tb ? glu_fwd<DT, true>(tile, vec, a, s) : glu_fwd<DT, false>(tile, vec, a, s);                \
    }                                                                                                       \
    hipError_t glu_dx_##NAME(bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s) {                 \
        return tb ? glu_bwd<DT, kSum2, false, true>(tile, vec, a, s)                                        \
                  : glu_bwd<DT, kSum2, false, false>(tile, vec, a, s);                                      \
    }                                                                                                       \
    hipError_t glu_dw_##NAME(int tile, bool vec, const FfnArgs &a, hipStream_t s) {                          \
        return glu_bwd<DT, kPair, true, false>(tile, vec, a, s);                                            \
    }

}  // namespace mm
