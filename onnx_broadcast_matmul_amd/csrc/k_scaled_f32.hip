// k_scaled_f32.hip -- the scaled INT8 product's tiled kernels for FLOAT outputs (see
// k_scaled.h).
#include "k_scaled.h"

namespace mm {
MM_SCALED_INSTANCE(MM_FLOAT, false, f32)
}  // namespace mm
