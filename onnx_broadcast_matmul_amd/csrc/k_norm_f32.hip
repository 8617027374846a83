// k_norm_f32.hip -- the fused norms for FLOAT (see k_norm.h).
#include "k_norm.h"

namespace mm {
MM_NORM_INSTANCE(MM_FLOAT, f32)
}  // namespace mm
