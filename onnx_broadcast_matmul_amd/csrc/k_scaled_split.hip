// k_scaled_split.hip -- the scaled INT8 product's tiled kernels for INT32 partial sums (see
// k_scaled.h).
#include "k_scaled.h"

namespace mm {
MM_SCALED_INSTANCE(MM_FLOAT, true, split)
}  // namespace mm
