// k_scaled_f16.hip -- the scaled INT8 product's tiled kernels for FLOAT16 outputs (see
// k_scaled.h).
#include "k_scaled.h"

namespace mm {
MM_SCALED_INSTANCE(MM_FLOAT16, false, f16)
}  // namespace mm
