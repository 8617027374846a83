// k_checkpoint.hip -- a dense [rows, cols] tensor to its 8-bit checkpoint and
// back (the format stands in checkpoint.h).  Memory bounds both.
#include "checkpoint.h"
#include "device.h"
#include "ffn.h"
#include "pieces.h"

namespace mm {

// A thread takes 16 bytes of a row, 32 / VE threads a block.
template <int DT>
__global__ __launch_bounds__(256) void k_checkpoint_pack(const void *X, int64_t rows, int64_t cols, int8_t *q, uint8_t *scale) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int VE = E::kVE, TPB = kCkBlock / VE, U = 4;
    const int64_t nb = (cols + kCkBlock - 1) / kCkBlock, cpr = nb * TPB, total = rows * cpr;
    const int64_t x0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 * U + threadIdx.x;
    uint4 v[U];
    int64_t row[U], col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t x = x0 + u * 256;
        row[u] = x < 0x7fffffff ? (int64_t)((uint32_t)x / (uint32_t)cpr) : x / cpr;
        col[u] = (x - row[u] * cpr) * VE;
        v[u] = x < total ? row_piece<S>((GlobalPtr<S>)((const S *)X + row[u] * cols + col[u]), cols - col[u], cols >= VE)
                         : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        S e[VE];
        __builtin_memcpy(e, &v[u], 16);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VE; ++i) top = max(top, ck_magnitude(E::to_f32(e[i])));
#pragma unroll
        for (int d = 1; d < TPB; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        if (row[u] >= rows) break;  // whole blocks
        const uint32_t ex = ck_exponent(top);
        const float inv = ck_inverse(ex);
        uint32_t w[VE / 4];
#pragma unroll
        for (int i = 0; i < VE / 4; ++i)
            w[i] = pack_bytes(ck_number(E::to_f32(e[4 * i]), inv), ck_number(E::to_f32(e[4 * i + 1]), inv),
                              ck_number(E::to_f32(e[4 * i + 2]), inv), ck_number(E::to_f32(e[4 * i + 3]), inv));
        int8_t *o = q + row[u] * cols + col[u];
        const int64_t left = cols - col[u];
        if (left >= VE) __builtin_memcpy(o, w, VE);
        else
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (i < left) o[i] = (int8_t)(w[i / 4] >> (i % 4 * 8));
        if (col[u] % kCkBlock == 0) scale[row[u] * nb + col[u] / kCkBlock] = (uint8_t)ex;
    }
}

// A thread takes eight values.
template <int DT>
__global__ __launch_bounds__(256) void k_checkpoint_unpack(const int8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                                                           void *X) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int U = 4;
    const int64_t nb = (cols + kCkBlock - 1) / kCkBlock, cpr = (cols + 7) / 8, total = rows * cpr;
    const int64_t x0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 * U + threadIdx.x;
    uint32_t w[U][2];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t x = x0 + u * 256;
        w[u][0] = w[u][1] = 0;
        s[u] = 0.0f;
        if (x >= total) continue;
        const int64_t row = x < 0x7fffffff ? (int64_t)((uint32_t)x / (uint32_t)cpr) : x / cpr;
        const int64_t col = (x - row * cpr) * 8, left = cols - col;
        const int8_t *p = q + row * cols + col;
        if (left >= 8) __builtin_memcpy(w[u], p, 8);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) w[u][i / 4] |= (uint32_t)(uint8_t)p[i] << (i % 4 * 8);
        s[u] = ck_scale(scale[row * nb + col / kCkBlock]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t x = x0 + u * 256;
        if (x >= total) break;
        const int64_t row = x < 0x7fffffff ? (int64_t)((uint32_t)x / (uint32_t)cpr) : x / cpr;
        const int64_t col = (x - row * cpr) * 8, left = cols - col;
        float f[8];
        unpack_bytes(w[u][0], s[u], f);
        unpack_bytes(w[u][1], s[u], f + 4);
        S o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = E::from_f32(f[i]);
        S *y = (S *)X + row * cols + col;
        if (left >= 8) __builtin_memcpy(y, o, sizeof(o));
        else
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) y[i] = o[i];
    }
}

// Blocks of 1024 pieces; one dimension of a grid holds less than 2^32 threads.
static bool grid_of(int64_t pieces, dim3 *g) {
    const int64_t n = (pieces + 1023) / 1024, gx = n < (1 << 23) ? n : (1 << 23), gy = (n + gx - 1) / gx;
    if (gy > 65535) return false;
    *g = dim3((unsigned)gx, (unsigned)gy);
    return true;
}

template <int DT>
static hipError_t pack(const void *X, int64_t rows, int64_t cols, void *q, void *scale, hipStream_t s) {
    dim3 g;
    if (!grid_of(rows * ((cols + kCkBlock - 1) / kCkBlock) * (kCkBlock / Elem<DT>::kVE), &g)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_checkpoint_pack<DT>, g, dim3(256), 0, s, X, rows, cols, (int8_t *)q, (uint8_t *)scale);
    return hipGetLastError();
}

hipError_t launch_checkpoint_pack(int dtype, const void *X, int64_t rows, int64_t cols, void *q, void *scale, hipStream_t s) {
    if (rows <= 0 || cols <= 0) return hipSuccess;
    switch (dtype) {
    case MM_FLOAT: return pack<MM_FLOAT>(X, rows, cols, q, scale, s);
    case MM_FLOAT16: return pack<MM_FLOAT16>(X, rows, cols, q, scale, s);
    case MM_BFLOAT16: return pack<MM_BFLOAT16>(X, rows, cols, q, scale, s);
    }
    return hipErrorInvalidValue;
}

template <int DT>
static hipError_t unpack(const void *q, const void *scale, int64_t rows, int64_t cols, void *X, hipStream_t s) {
    dim3 g;
    if (!grid_of(rows * ((cols + 7) / 8), &g)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_checkpoint_unpack<DT>, g, dim3(256), 0, s, (const int8_t *)q, (const uint8_t *)scale, rows, cols, X);
    return hipGetLastError();
}

hipError_t launch_checkpoint_unpack(int dtype, const void *q, const void *scale, int64_t rows, int64_t cols, void *X,
                                    hipStream_t s) {
    if (rows <= 0 || cols <= 0) return hipSuccess;
    switch (dtype) {
    case MM_FLOAT: return unpack<MM_FLOAT>(q, scale, rows, cols, X, s);
    case MM_FLOAT16: return unpack<MM_FLOAT16>(q, scale, rows, cols, X, s);
    case MM_BFLOAT16: return unpack<MM_BFLOAT16>(q, scale, rows, cols, X, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
