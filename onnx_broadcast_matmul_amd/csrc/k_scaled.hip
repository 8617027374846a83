// k_scaled.hip -- INT8 product with one FP32 scale for each row of A (token)
// and each column of B (channel):
//
//   Y[m][n] = sa[m] sb[n] sum_k A[m][k] B[k][n] + bias[n]
//
// The sum is exact: |A B| <= 2^14 and K < 2^17 keep it inside INT32, so every
// order and every split of K gives the same bits.  It is rounded once to FP32
// for the scales and once to the output type.
#include "k_ffn.h"

namespace mm {

template <int OD, int MODE, bool TB>
static hipError_t tiled(int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    switch (tile) {
    case 0: return launch_ffn<MM_INT8, OD, MODE, false, TB, 256, 256, 2, 4, 64, 4, 8>(vec, a, s);
    case 1: return launch_ffn<MM_INT8, OD, MODE, false, TB, 128, 128, 2, 2, 64, 4, 4>(vec, a, s);
    case 2: return launch_ffn<MM_INT8, OD, MODE, false, TB, 64, 128, 2, 2, 64, 4, 4>(vec, a, s);
    case 3: return launch_ffn<MM_INT8, OD, MODE, false, TB, 32, 128, 1, 2, 64, 4, 2>(vec, a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_scaled(int od, bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    switch (od) {
    case MM_FLOAT: return tb ? tiled<MM_FLOAT, kScaled, true>(tile, vec, a, s) : tiled<MM_FLOAT, kScaled, false>(tile, vec, a, s);
    case MM_FLOAT16:
        return tb ? tiled<MM_FLOAT16, kScaled, true>(tile, vec, a, s) : tiled<MM_FLOAT16, kScaled, false>(tile, vec, a, s);
    case MM_BFLOAT16:
        return tb ? tiled<MM_BFLOAT16, kScaled, true>(tile, vec, a, s) : tiled<MM_BFLOAT16, kScaled, false>(tile, vec, a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_scaled_split(bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    return tb ? tiled<MM_FLOAT, kScaledSplit, true>(tile, vec, a, s) : tiled<MM_FLOAT, kScaledSplit, false>(tile, vec, a, s);
}

// Sum of the K partitions' INT32 partials, then the epilogue of the tiled
// kernel; a thread owns four consecutive outputs.
template <int OD>
__global__ __launch_bounds__(256) void k_scaled_reduce(FfnArgs a) {
    using E = Elem<OD>;
    using S = typename E::S;
    const int64_t M = a.M, N = a.N, total = a.batch * M * N;
    const int64_t o0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (o0 >= total) return;
    int acc[4] = {0, 0, 0, 0};
    const bool whole = o0 + 4 <= total;
    if (whole && total % 4 == 0) {  // every partition's quadruple is aligned
        for (int p = 0; p < a.split; ++p) {
            const int4 v = *(const int4 *)(a.W + (int64_t)p * total + o0);
            acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
        }
    } else {
        for (int p = 0; p < a.split; ++p)
            for (int e = 0; e < 4; ++e)
                if (o0 + e < total) acc[e] += a.W[(int64_t)p * total + o0 + e];
    }
    S out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t o = o0 + e < total ? o0 + e : total - 1;
        const int64_t n = o % N, m = (o / N) % M, b = o / (M * N);
        int64_t oa, ob;
        batch_offsets(a.bd, b, oa, ob);
        const float bias = a.bias ? E::to_f32(((const S *)a.bias)[n]) : 0.0f;
        out[e] = E::from_f32(scaled_value(acc[e], a.sa[oa / a.lda + m], a.sb[ob / a.K + n], bias));
    }
    S *Y = (S *)a.Y[0] + o0;
    if (whole) __builtin_memcpy(Y, out, sizeof(out));
    else
        for (int e = 0; e < 4; ++e)
            if (o0 + e < total) Y[e] = out[e];
}

hipError_t launch_scaled_reduce(int od, const FfnArgs &a, hipStream_t s) {
    const int64_t g = ((a.batch * a.M * a.N + 3) / 4 + 255) / 256;
    if (g <= 0) return hipSuccess;
    if (g > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 gr((unsigned)g), bl(256);
    switch (od) {
    case MM_FLOAT: hipLaunchKernelGGL(k_scaled_reduce<MM_FLOAT>, gr, bl, 0, s, a); break;
    case MM_FLOAT16: hipLaunchKernelGGL(k_scaled_reduce<MM_FLOAT16>, gr, bl, 0, s, a); break;
    case MM_BFLOAT16: hipLaunchKernelGGL(k_scaled_reduce<MM_BFLOAT16>, gr, bl, 0, s, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace mm
