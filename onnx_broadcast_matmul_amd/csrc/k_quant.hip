// k_quant.hip -- row quantization of a dense [rows, cols] matrix to INT8 (the
// rule stands in quantize.h).  The row is read once and kept in registers
// while its maximum is formed; rows longer than a workgroup holds are read a
// second time.  Memory bounds it: 8192 x 4096 BF16 18-20 us (101 MB read and
// written, 5.0-5.5 TB/s); below about 1 MB the launch does (24 x 4096: 3.5 us).
#include "ffn.h"
#include "quantize.h"

namespace mm {

// TPR threads per row (64 or 256), CH 16-byte chunks per thread kept.
template <int DT, int TPR, int CH>
__global__ __launch_bounds__(256) void k_quantize_rows(const void *X, int64_t rows, int64_t cols, int8_t *Q,
                                                       int64_t ldq, float *scale) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int VE = E::kVE;
    constexpr int RPW = 256 / TPR;
    const int t = threadIdx.x % TPR;
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPW + threadIdx.x / TPR;
    const bool live = row < rows;  // all threads reach the barrier
    const S *x = (const S *)X + (live ? row : 0) * cols;
    uint4 keep[CH];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) keep[i] = quant_load<DT>(x, ((int64_t)i * TPR + t) * VE, cols);
#pragma unroll
    for (int i = 0; i < CH; ++i) m = quant_top<DT>(keep[i], m);
    for (int64_t c0 = ((int64_t)CH * TPR + t) * VE; c0 < cols; c0 += (int64_t)TPR * VE)
        m = quant_top<DT>(quant_load<DT>(x, c0, cols), m);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
        m = o > m ? o : m;
    }
    if constexpr (TPR == 256) {
        __shared__ uint32_t part[4];
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
        __syncthreads();
        m = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    if (!live) return;
    const float r = quant_factor(m);
    if (t == 0) scale[row] = quant_scale(m);
    int8_t *q = Q + row * ldq;  // bytes cols .. ldq - 1 hold zeros
    auto emit = [&](int64_t c0, const uint4 &v) {
        int8_t o[VE];
        quant_bytes<DT>(v, r, o);
        if (c0 + VE <= ldq) __builtin_memcpy(q + c0, o, VE);
        else
            for (int i = 0; i < VE; ++i)
                if (c0 + i < ldq) q[c0 + i] = o[i];
    };
#pragma unroll
    for (int i = 0; i < CH; ++i) emit(((int64_t)i * TPR + t) * VE, keep[i]);
    for (int64_t c0 = ((int64_t)CH * TPR + t) * VE; c0 < ldq; c0 += (int64_t)TPR * VE)
        emit(c0, quant_load<DT>(x, c0, cols));
}

template <int DT>
static hipError_t quantize(const void *X, int64_t rows, int64_t cols, void *Q, int64_t ldq, float *scale, hipStream_t s) {
    // A wave per row up to four chunks a lane, else a workgroup per row.
    constexpr int VE = Elem<DT>::kVE;
    const bool narrow = ldq <= 64 * 4 * VE;
    const int64_t g = narrow ? (rows + 3) / 4 : rows;
    if (g <= 0) return hipSuccess;
    // One dimension of a grid holds less than 2^32 threads.
    const int64_t gx = g < (1 << 23) ? g : (1 << 23), gy = (g + gx - 1) / gx;
    if (gy > 65535) return hipErrorInvalidValue;
    const dim3 gr((unsigned)gx, (unsigned)gy), bl(256);
    if (narrow) hipLaunchKernelGGL((k_quantize_rows<DT, 64, 4>), gr, bl, 0, s, X, rows, cols, (int8_t *)Q, ldq, scale);
    else if (ldq <= 256 * 2 * VE) hipLaunchKernelGGL((k_quantize_rows<DT, 256, 2>), gr, bl, 0, s, X, rows, cols, (int8_t *)Q, ldq, scale);
    else hipLaunchKernelGGL((k_quantize_rows<DT, 256, 8>), gr, bl, 0, s, X, rows, cols, (int8_t *)Q, ldq, scale);
    return hipGetLastError();
}

hipError_t launch_quantize_rows(int dtype, const void *X, int64_t rows, int64_t cols, void *Q, int64_t ldq, float *scale,
                                hipStream_t s) {
    switch (dtype) {
    case MM_FLOAT: return quantize<MM_FLOAT>(X, rows, cols, Q, ldq, scale, s);
    case MM_FLOAT16: return quantize<MM_FLOAT16>(X, rows, cols, Q, ldq, scale, s);
    case MM_BFLOAT16: return quantize<MM_BFLOAT16>(X, rows, cols, Q, ldq, scale, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
