// k_norm_f16.hip -- the fused norms for FLOAT16 (see k_norm.h).
#include "k_norm.h"

namespace mm {
MM_NORM_INSTANCE(MM_FLOAT16, f16)
}  // namespace mm
