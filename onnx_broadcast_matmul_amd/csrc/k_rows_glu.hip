// k_rows_glu.hip -- the gated block over few rows (see k_ffn_rows.h).
#include "k_ffn_rows.h"

namespace mm {

template <int DT>
static hipError_t glu(bool tb, const FfnArgs &a, hipStream_t s) {
    if (tb)
        return a.M <= 16 ? launch_rows<DT, DT, true, false, 2, 1, 8, 0>(a, s) : launch_rows<DT, DT, true, false, 2, 2, 8, 0>(a, s);
    return a.M <= 16 ? launch_rows<DT, DT, true, true, 4, 1, 8, 0>(a, s) : launch_rows<DT, DT, true, true, 4, 2, 8, 0>(a, s);
}

hipError_t launch_glu_rows(int dtype, bool tb, const FfnArgs &a, hipStream_t s) {
    switch (dtype) {
    case MM_FLOAT: return glu<MM_FLOAT>(tb, a, s);
    case MM_FLOAT16: return glu<MM_FLOAT16>(tb, a, s);
    case MM_BFLOAT16: return glu<MM_BFLOAT16>(tb, a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
