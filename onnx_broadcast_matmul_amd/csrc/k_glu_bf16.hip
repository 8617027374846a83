// k_glu_bf16.hip -- the gated block's tiled products for BFLOAT16 (see k_glu.h).
#include "k_glu.h"

namespace mm {
MM_GLU_INSTANCE(MM_BFLOAT16, bf16)
}  // namespace mm
