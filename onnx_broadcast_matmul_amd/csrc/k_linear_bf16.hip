// k_linear_bf16.hip -- the linear layer's tiled products for BFLOAT16 (see k_linear.h).
#include "k_linear.h"

namespace mm {
MM_LINEAR_INSTANCE(MM_BFLOAT16, bf16)
}  // namespace mm
