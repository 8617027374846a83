// k_scaled.h -- the scaled INT8 product's tiled kernels for one output type, or
// for the INT32 partial sums (instantiated by k_scaled_f32.hip, k_scaled_f16.hip,
// k_scaled_bf16.hip and k_scaled_split.hip).
#pragma once

#include "k_ffn.h"

#define MM_SCALED_INSTANCE(OD, SPLIT, NAME)                                                        \
    hipError_t scaled_##NAME(bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s) {        \
        return tb ? launch_entry<MM_INT8, OD, kScaled, SPLIT, false, true>(tile, vec, a, s)        \
                  : launch_entry<MM_INT8, OD, kScaled, SPLIT, false, false>(tile, vec, a, s);      \
    }
