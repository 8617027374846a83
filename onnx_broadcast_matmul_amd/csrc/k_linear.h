// k_linear.h -- the linear layer's tiled products for one element type
// (instantiated by k_linear_f32.hip, k_linear_f16.hip and k_linear_bf16.hip): the
// forward pass with bias, activation and residual in its epilogue, and dX = dZ W^T,
// the same product without one.
#pragma once

#include "k_ffn.h"

namespace mm {

#define MM_LINEAR_INSTANCE(DT, NAME)                                                                      \
    hipError_t linear_##NAME(bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {   \
        if (split)                                                                                        \
            return tb ? launch_entry<DT, DT, kLinear, true, false, true>(tile, vec, a, s)                 \
                      : launch_entry<DT, DT, kLinear, true, false, false>(tile, vec, a, s);               \
        return tb ? launch_entry<DT, DT, kLinear, false, false, true>(tile, vec, a, s)                    \
                  : launch_entry<DT, DT, kLinear, false, false, false>(tile, vec, a, s);                  \
    }

}  // namespace mm
