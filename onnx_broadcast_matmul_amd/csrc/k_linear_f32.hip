// k_linear_f32.hip -- the linear layer's tiled products for FLOAT (see k_linear.h).
#include "k_linear.h"

namespace mm {
MM_LINEAR_INSTANCE(MM_FLOAT, f32)
}  // namespace mm
