// k_norm_bf16.hip -- the fused norms for BFLOAT16 (see k_norm.h).
#include "k_norm.h"

namespace mm {
MM_NORM_INSTANCE(MM_BFLOAT16, bf16)
}  // namespace mm
