// k_quant.hip -- row quantization of a dense [rows, cols] matrix to INT8:
//
//   amax = max(max_k |x_k|, 2^-100),  s = amax / 127,  q_k = rint(x_k r),
//   r = 127 / amax (rounded to FP32)
//
// so |x_k - s q_k| <= s / 2 up to FP32 rounding, and the largest element maps
// to +-127.  A row that holds an infinity or a NaN has no scale: its s is NaN
// and its q zero, so that whatever is computed from it is NaN.
//
// The row is read once and kept in registers while its maximum is formed;
// rows longer than a workgroup holds are read a second time.
#include "device.h"
#include "ffn.h"

namespace mm {

constexpr float kQuantFloor = 7.888609052210118e-31f;  // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// TPR threads per row (64 or 256), CH 16-byte chunks per thread kept.
template <int DT, int TPR, int CH>
__global__ __launch_bounds__(256) void k_quantize_rows(const void *X, int64_t rows, int64_t cols, int8_t *Q,
                                                       int64_t ldq, float *scale) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int VE = E::kVE;
    constexpr int RPW = 256 / TPR;
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
    const bool live = row < rows;  // all threads reach the barrier
    const S *x = (const S *)X + (live ? row : 0) * cols;
    auto load = [&](int64_t c0, uint4 &v) {
        v = make_uint4(0, 0, 0, 0);
        if (c0 + VE <= cols) {
            __builtin_memcpy(&v, x + c0, 16);
        } else if (c0 < cols) {
            S tmp[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) tmp[e] = c0 + e < cols ? x[c0 + e] : (S)0;
            __builtin_memcpy(&v, tmp, 16);
        }
    };
    // Magnitudes order as their bits, with infinity and NaN above all.
    auto top = [&](const uint4 &v, uint32_t m) {
        S e[VE];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const uint32_t b = __float_as_uint(E::to_f32(e[i])) & 0x7fffffffu;
            m = b > m ? b : m;
        }
        return m;
    };
    uint4 keep[CH];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) load(((int64_t)i * TPR + t) * VE, keep[i]);
#pragma unroll
    for (int i = 0; i < CH; ++i) m = top(keep[i], m);
    for (int64_t c0 = ((int64_t)CH * TPR + t) * VE; c0 < cols; c0 += (int64_t)TPR * VE) {
        uint4 v;
        load(c0, v);
        m = top(v, m);
    }
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
    const bool bad = m >= kInfBits;
    const float amax = fmaxf(__uint_as_float(m), kQuantFloor);
    const float r = bad ? 0.0f : 127.0f / amax;
    if (t == 0) scale[row] = bad ? __uint_as_float(0x7fc00000u) : amax / 127.0f;
    int8_t *q = Q + row * ldq;  // bytes cols .. ldq - 1 hold zeros
    auto emit = [&](int64_t c0, const uint4 &v) {
        S e[VE];
        __builtin_memcpy(e, &v, 16);
        int8_t o[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) o[i] = bad ? (int8_t)0 : (int8_t)(int)rintf(E::to_f32(e[i]) * r);
        if (c0 + VE <= ldq) __builtin_memcpy(q + c0, o, VE);
        else
            for (int i = 0; i < VE; ++i)
                if (c0 + i < ldq) q[c0 + i] = o[i];
    };
#pragma unroll
    for (int i = 0; i < CH; ++i) emit(((int64_t)i * TPR + t) * VE, keep[i]);
    for (int64_t c0 = ((int64_t)CH * TPR + t) * VE; c0 < ldq; c0 += (int64_t)TPR * VE) {
        uint4 v;
        load(c0, v);
        emit(c0, v);
    }
}

template <int DT>
static hipError_t quantize(const void *X, int64_t rows, int64_t cols, void *Q, int64_t ldq, float *scale, hipStream_t s) {
    // A wave per row up to four chunks a lane, else a workgroup per row.
    constexpr int VE = Elem<DT>::kVE;
    const bool narrow = ldq <= 64 * 4 * VE;
    const int64_t g = narrow ? (rows + 3) / 4 : rows;
    if (g <= 0) return hipSuccess;
    if (g > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 gr((unsigned)g), bl(256);
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
