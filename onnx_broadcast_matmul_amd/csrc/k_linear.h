// k_linear.h -- the linear layer's products for one element type
// (instantiated by k_linear_f32.hip, k_linear_f16.hip and k_linear_bf16.hip): the
// forward pass with bias, activation and residual in its epilogue, dX = dZ W^T,
// the same product without one, and dW.  Large 16-bit ones run on k_big.h, all
// others on k_ffn.h.
#pragma once

#include "k_big.h"
#include "k_ffn.h"

namespace mm {

// dW of one product, the pair's kernel where the large one does not take it.
hipError_t launch_glu_dw(int dtype, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);

#define MM_LINEAR_INSTANCE(DT, NAME)                                                                      \
    hipError_t linear_##NAME(bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {   \
        if constexpr (DT != MM_FLOAT) {                                                                   \
            if (big_fits(false, tb, tile, split, vec, a)) {                                               \
                if (tile == 0)                                                                            \
                    return tb ? launch_big<DT, false, true, true, 256>(a, s)                              \
                              : launch_big<DT, false, false, true, 256>(a, s);                            \
                return tb ? launch_big<DT, false, true, true, 128>(a, s)                                  \
                          : launch_big<DT, false, false, true, 128>(a, s);                                \
            }                                                                                             \
        }                                                                                                 \
        if (tile == 0) tile = 1; /* rows off alignment, or too far apart */                               \
        if (split)                                                                                        \
            return tb ? launch_entry<DT, DT, kLinear, true, false, true>(tile, vec, a, s)                 \
                      : launch_entry<DT, DT, kLinear, true, false, false>(tile, vec, a, s);               \
        return tb ? launch_entry<DT, DT, kLinear, false, false, true>(tile, vec, a, s)                    \
                  : launch_entry<DT, DT, kLinear, false, false, false>(tile, vec, a, s);                  \
    }                                                                                                     \
    hipError_t linear_dw_##NAME(int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {         \
        if constexpr (DT != MM_FLOAT) {                                                                   \
            if (big_fits(true, false, tile, split, vec, a))                                               \
                return tile == 0 ? launch_big<DT, true, false, false, 256>(a, s)                          \
                                 : launch_big<DT, true, false, false, 128>(a, s);                         \
        }                                                                                                 \
        return launch_glu_dw(DT, tile, split, vec, a, s);                                                 \
    }

}  // namespace mm
