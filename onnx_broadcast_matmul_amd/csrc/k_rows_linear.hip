// k_rows_linear.hip -- the linear layer over few rows (see k_ffn_rows.h).
#include "k_ffn_rows.h"

namespace mm {

template <int DT>
static hipError_t linear(bool tb, const FfnArgs &a, hipStream_t s) {
    if (tb)
        return a.M <= 16 ? launch_rows<DT, DT, false, false, 1, 1, 8, 0>(a, s) : launch_rows<DT, DT, false, false, 1, 2, 8, 0>(a, s);
    return a.M <= 16 ? launch_rows<DT, DT, false, true, 4, 1, 8, 0>(a, s) : launch_rows<DT, DT, false, true, 4, 2, 8, 0>(a, s);
}

hipError_t launch_linear_rows(int dtype, bool tb, const FfnArgs &a, hipStream_t s) {
    switch (dtype) {
    case MM_FLOAT: return linear<MM_FLOAT>(tb, a, s);
    case MM_FLOAT16: return linear<MM_FLOAT16>(tb, a, s);
    case MM_BFLOAT16: return linear<MM_BFLOAT16>(tb, a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
