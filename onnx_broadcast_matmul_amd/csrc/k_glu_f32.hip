// k_glu_f32.hip -- the gated block's tiled products for FLOAT (see k_glu.h).
#include "k_glu.h"

namespace mm {
MM_GLU_INSTANCE(MM_FLOAT, f32)
}  // namespace mm
