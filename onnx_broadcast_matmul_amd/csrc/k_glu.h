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

#define MM_GLU_INSTANCE(DT, NAME)                                                                           \
    hipError_t glu_fwd_##NAME(bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {    \
        if (split)                                                                                          \
            return tb ? launch_entry<DT, DT, kGlu, true, false, true>(tile, vec, a, s)                      \
                      : launch_entry<DT, DT, kGlu, true, false, false>(tile, vec, a, s);                    \
        return tb ? launch_entry<DT, DT, kGlu, false, false, true>(tile, vec, a, s)                         \
                  : launch_entry<DT, DT, kGlu, false, false, false>(tile, vec, a, s);                       \
    }                                                                                                       \
    hipError_t glu_dx_##NAME(bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {     \
        if (split)                                                                                          \
            return tb ? launch_entry<DT, DT, kSum2, true, false, true>(tile, vec, a, s)                     \
                      : launch_entry<DT, DT, kSum2, true, false, false>(tile, vec, a, s);                   \
        return tb ? launch_entry<DT, DT, kSum2, false, false, true>(tile, vec, a, s)                        \
                  : launch_entry<DT, DT, kSum2, false, false, false>(tile, vec, a, s);                      \
    }                                                                                                       \
    hipError_t glu_dw_##NAME(int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {              \
        return split ? launch_entry<DT, DT, kPair, true, true, false>(tile, vec, a, s)                      \
                     : launch_entry<DT, DT, kPair, false, true, false>(tile, vec, a, s);                    \
    }

}  // namespace mm
