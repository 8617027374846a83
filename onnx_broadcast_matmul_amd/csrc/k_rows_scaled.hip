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

// Each workgroup quantizes the rows for itself.  Up to 2 rows, or 8 short ones,
// that costs less than the launch it saves (BF16, [N, K] weights from memory,
// N = 4096: 1 x 11008 15.1 against 19.3 us, 2 x 11008 17.3 against 19.5, 8 x 2048
// 6.8 against 8.6; but 4 x 4096 9.3 against 9.1, 4 x 11008 21.8 against 19.9 and,
// with N = 11008, 45.9 against 36.5).
bool rows_quantize(int a_type, int out_dtype, bool tb, int64_t M, int64_t K, int64_t N) {
    const int64_t waves = tb && (N + 15) / 16 > kRowsFit ? 4 : 8;  // see launch_rows
    return a_type == out_dtype && M <= waves && (M <= 2 || K <= 2048) && M * ((K + 63) / 64 * 64 + 16) <= kFfnQuantLds;
}

hipError_t launch_scaled_rows(int od, bool tb, bool quant, const FfnArgs &a, hipStream_t s) {
    if (quant && !rows_quantize(od, od, tb, a.M, a.K, a.N)) return hipErrorInvalidValue;
    switch (od) {
    case MM_FLOAT: return scaled<MM_FLOAT>(tb, quant, a, s);
    case MM_FLOAT16: return scaled<MM_FLOAT16>(tb, quant, a, s);
    case MM_BFLOAT16: return scaled<MM_BFLOAT16>(tb, quant, a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
