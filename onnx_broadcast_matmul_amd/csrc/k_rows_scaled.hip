// k_rows_scaled.hip -- the scaled INT8 product over few rows (see
// k_ffn_rows.h).  With `quant` A[0] holds rows of the output's type that the
// kernel quantizes itself.
#include "k_ffn_rows.h"

namespace mm {

template <int OD>
static hipError_t scaled(bool tb, bool quant, const FfnArgs &a, hipStream_t s) {
    if (tb) {
        if (quant) return launch_rows<MM_INT8, OD, false, false, 1, 1, 8, OD>(a, s);
        return a.M <= 16 ? launch_rows<MM_INT8, OD, false, false, 1, 1, 8, 0>(a, s)
                         : launch_rows<MM_INT8, OD, false, false, 1, 2, 8, 0>(a, s);
    }
    if (quant) return launch_rows<MM_INT8, OD, false, true, 4, 1, 8, OD>(a, s);
    return a.M <= 16 ? launch_rows<MM_INT8, OD, false, true, 4, 1, 8, 0>(a, s)
                     : launch_rows<MM_INT8, OD, false, true, 4, 2, 8, 0>(a, s);
}

// Each workgroup quantizes the rows for itself: up to 4 rows that costs less
// than the launch it saves (BF16, N = 4096: one row of 11008 15.4 us against
// 12.8 + 5.8; eight rows of 4096 11.8 against 6.3 + 5).
bool rows_quantize(int a_type, int out_dtype, int64_t M, int64_t K) {
    return a_type == out_dtype && M <= kFfnQuantRows && M * ((K + 63) / 64 * 64 + 16) <= kFfnQuantLds;
}

hipError_t launch_scaled_rows(int od, bool tb, bool quant, const FfnArgs &a, hipStream_t s) {
    if (quant && !rows_quantize(od, od, a.M, a.K)) return hipErrorInvalidValue;
    switch (od) {
    case MM_FLOAT: return scaled<MM_FLOAT>(tb, quant, a, s);
    case MM_FLOAT16: return scaled<MM_FLOAT16>(tb, quant, a, s);
    case MM_BFLOAT16: return scaled<MM_BFLOAT16>(tb, quant, a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
