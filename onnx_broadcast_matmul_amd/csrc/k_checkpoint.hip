// k_checkpoint.hip -- a dense [rows, cols] tensor to its 8-bit checkpoint and
// back (the format stands in checkpoint.h).  Memory bounds both.
#include "checkpoint.h"
#include "device.h"
#include "ffn.h"
#include "pieces.h"

namespace mm {

// Where piece x (of cpr a row, VE elements each) lies.  FLAT: rows are whole
// blocks, so they follow each other without a seam and no row is told from the
// next (the division costs a third of the arithmetic).
template <bool FLAT, int VE>
__device__ __forceinline__ void piece_place(int64_t x, int64_t cpr, int64_t cols, int64_t nb, int64_t &row, int &col, int64_t &at,
                                            int64_t &block) {
    if constexpr (FLAT) {
        at = x * VE;
        block = x / (kCkBlock / VE);
        row = 0;
        col = 0;
    } else {
        row = x < 0x7fffffff ? (int64_t)((uint32_t)x / (uint32_t)cpr) : x / cpr;
        col = (int)(x - row * cpr) * VE;
        at = row * cols + col;
        block = row * nb + col / kCkBlock;
    }
}

// A thread takes 16 bytes of a row at a time, 32 / VE threads a block.
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void k_checkpoint_pack(const void *X, int64_t rows, int64_t cols, int8_t *q, uint8_t *scale) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int VE = E::kVE, TPB = kCkBlock / VE, U = 4;
    const int n = (int)cols;
    const int64_t nb = (cols + kCkBlock - 1) / kCkBlock, cpr = nb * TPB, total = rows * cpr;
    const int64_t x0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 * U + threadIdx.x;
    uint4 v[U];
    int64_t at[U], block[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t x = x0 + u * 256 < total ? x0 + u * 256 : 0;
        int64_t row;
        piece_place<FLAT, VE>(x, cpr, cols, nb, row, col[u], at[u], block[u]);
        if constexpr (FLAT) v[u] = stream_piece<S>((GlobalPtr<S>)X + at[u]);
        else v[u] = edge_load<S, true>((GlobalPtr<S>)((const S *)X + row * cols), n, col[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (x0 + u * 256 >= total) break;  // whole blocks
        if constexpr (!FLAT) v[u] = edge_piece<S>(v[u], n, col[u]);
        const uint32_t ex = ck_exponent(block_top<VE>(piece_top<DT>(v[u])));
        const float inv = ck_inverse(ex);
        S e[VE];
        __builtin_memcpy(e, &v[u], 16);
        uint32_t w[VE / 4];
#pragma unroll
        for (int i = 0; i < VE / 4; ++i)
            w[i] = ck_word(E::to_f32(e[4 * i]), E::to_f32(e[4 * i + 1]), E::to_f32(e[4 * i + 2]), E::to_f32(e[4 * i + 3]), inv);
        ck_store<VE>(q + (at[u] - col[u]), FLAT ? VE : n, col[u], w);
        if (threadIdx.x % TPB == 0) __builtin_nontemporal_store((uint8_t)ex, scale + block[u]);
    }
}

// A thread takes 16 bytes of results at a time.
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void k_checkpoint_unpack(const int8_t *q, const uint8_t *scale, int64_t rows, int64_t cols,
                                                           void *X) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int U = 4, VE = E::kVE;
    const int n = (int)cols;
    const int64_t nb = (cols + kCkBlock - 1) / kCkBlock, cpr = (cols + VE - 1) / VE, total = rows * cpr;
    const int64_t x0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 * U + threadIdx.x;
    uint32_t w[U][VE / 4];
    float s[U];
    int64_t at[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t x = x0 + u * 256 < total ? x0 + u * 256 : 0;
        int64_t row, block;
        piece_place<FLAT, VE>(x, cpr, cols, nb, row, col[u], at[u], block);
        ck_load<VE>(q + (at[u] - col[u]), FLAT ? VE : n, col[u], w[u]);
        s[u] = ck_scale(scale[block]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (x0 + u * 256 >= total) break;
        float f[VE];
#pragma unroll
        for (int i = 0; i < VE / 4; ++i) unpack_bytes(w[u][i], s[u], f + 4 * i);
        S o[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) o[i] = E::from_f32(f[i]);
        S *y = (S *)X + at[u];
        uint4 v;
        __builtin_memcpy(&v, o, 16);
        if (FLAT || col[u] <= n - VE) stream_store(y, v);
        else
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (col[u] + i < n) y[i] = o[i];
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
    if (cols % kCkBlock == 0) hipLaunchKernelGGL((k_checkpoint_pack<DT, true>), g, dim3(256), 0, s, X, rows, cols, (int8_t *)q, (uint8_t *)scale);
    else hipLaunchKernelGGL((k_checkpoint_pack<DT, false>), g, dim3(256), 0, s, X, rows, cols, (int8_t *)q, (uint8_t *)scale);
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
    constexpr int VE = Elem<DT>::kVE;
    if (!grid_of(rows * ((cols + VE - 1) / VE), &g)) return hipErrorInvalidValue;
    if (cols % kCkBlock == 0) hipLaunchKernelGGL((k_checkpoint_unpack<DT, true>), g, dim3(256), 0, s, (const int8_t *)q, (const uint8_t *)scale, rows, cols, X);
    else hipLaunchKernelGGL((k_checkpoint_unpack<DT, false>), g, dim3(256), 0, s, (const int8_t *)q, (const uint8_t *)scale, rows, cols, X);
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
