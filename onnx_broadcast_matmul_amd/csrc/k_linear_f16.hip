// k_linear_f16.hip -- the linear layer's tiled products for FLOAT16 (see k_linear.h).
#include "k_linear.h"

namespace mm {
MM_LINEAR_INSTANCE(MM_FLOAT16, f16)
}  // namespace mm
