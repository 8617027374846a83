// k_scaled_bf16.hip -- the scaled INT8 product's tiled kernels for BFLOAT16 outputs (see
// k_scaled.h).
#include "k_scaled.h"

namespace mm {
MM_SCALED_INSTANCE(MM_BFLOAT16, false, bf16)
}  // namespace mm
