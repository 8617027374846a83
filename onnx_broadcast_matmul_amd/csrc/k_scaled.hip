// k_scaled.hip -- INT8 product with one FP32 scale for each row of A (token)
// and each column of B (channel):
//
//   Y[m][n] = sa[m] sb[n] sum_k A[m][k] B[k][n] + bias[n]
//
// The sum is exact: |A B| <= 2^14 and K < 2^17 keep it inside INT32, so every
// order and every split of K gives the same bits.  It is rounded once to FP32
// for the scales and once to the output type.
#include <type_traits>

#include "activation.h"
#include "device.h"
#include "ffn.h"

namespace mm {

#define MM_SCALED_DECLARE(NAME) hipError_t scaled_##NAME(bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s);
MM_SCALED_DECLARE(f32)
MM_SCALED_DECLARE(f16)
MM_SCALED_DECLARE(bf16)
MM_SCALED_DECLARE(split)

hipError_t launch_scaled(int od, bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    switch (od) {
    case MM_FLOAT: return scaled_f32(tb, tile, vec, a, s);
    case MM_FLOAT16: return scaled_f16(tb, tile, vec, a, s);
    case MM_BFLOAT16: return scaled_bf16(tb, tile, vec, a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_scaled_split(bool tb, int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    return scaled_split(tb, tile, vec, a, s);
}

// Sum of the K partitions' INT32 partials, then the epilogue of the tiled
// kernel; a thread owns four consecutive columns of one row of product
// blockIdx.y.
template <int OD, bool BATCH>
__global__ __launch_bounds__(256) void k_scaled_reduce(typename std::conditional<BATCH, FfnSlimBatch, FfnSlim>::type a) {
    using E = Elem<OD>;
    using S = typename E::S;
    const uint32_t N = (uint32_t)a.N, cpr = (N + 3) / 4;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= (int64_t)a.M * cpr) return;
    const int64_t row = x < 0x7fffffff ? (int64_t)((uint32_t)x / cpr) : x / cpr;
    const uint32_t col = (uint32_t)(x - row * cpr) * 4;
    const int64_t b = blockIdx.y, stride = (int64_t)gridDim.y * a.M * N;
    int64_t oa = 0, ob = 0;
    if constexpr (BATCH) batch_offsets(a.bd, b, oa, ob);
    const int *w = (const int *)a.W() + b * a.M * N + row * N + col;
    const float sa = a.sa()[oa / a.lda + row];
    const float *sb = a.sb() + ob / a.K + col;
    int acc[4] = {0, 0, 0, 0};
    if (N % 4 == 0) {
#pragma unroll 4
        for (int p = 0; p < a.split; ++p) {
            const int4 v = *(const int4 *)(w + p * stride);
            acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
        }
    } else {
        for (int p = 0; p < a.split; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < N) acc[e] += w[p * stride + e];
    }
    S out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t n = col + e < N ? e : 0;
        const float bias = a.bias() ? E::to_f32(((const S *)a.bias())[col + n]) : 0.0f;
        out[e] = E::from_f32(scaled_value(acc[e], sa, sb[n], bias));
    }
    S *y = (S *)a.Y[0] + b * a.M * a.ldy + row * a.ldy + col;
    if (col + 4 <= N) __builtin_memcpy(y, out, sizeof(out));
    else
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < N) y[e] = out[e];
}

template <int OD>
static hipError_t reduce(const FfnArgs &a, const dim3 &gr, hipStream_t s) {
    if (a.batch != 1) hipLaunchKernelGGL((k_scaled_reduce<OD, true>), gr, dim3(256), 0, s, slim_batch(a, false, true));
    else hipLaunchKernelGGL((k_scaled_reduce<OD, false>), gr, dim3(256), 0, s, slim_args<FfnSlim>(a, kUseScaled, false, true));
    return hipGetLastError();
}

hipError_t launch_scaled_reduce(int od, const FfnArgs &a, hipStream_t s) {
    const int64_t g = (a.M * ((a.N + 3) / 4) + 255) / 256;
    if (g <= 0 || a.batch <= 0) return hipSuccess;
    if (g > 0x7fffffff || a.batch > 65535) return hipErrorInvalidValue;
    const dim3 gr((unsigned)g, (unsigned)a.batch);
    switch (od) {
    case MM_FLOAT: return reduce<MM_FLOAT>(a, gr, s);
    case MM_FLOAT16: return reduce<MM_FLOAT16>(a, gr, s);
    case MM_BFLOAT16: return reduce<MM_BFLOAT16>(a, gr, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
