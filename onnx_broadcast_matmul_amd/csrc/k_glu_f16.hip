// k_glu_f16.hip -- the gated block's tiled products for FLOAT16 (see k_glu.h).
#include "k_glu.h"

namespace mm {
MM_GLU_INSTANCE(MM_FLOAT16, f16)
}  // namespace mm
