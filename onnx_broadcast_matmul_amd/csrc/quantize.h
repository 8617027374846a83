// quantize.h -- the row quantization rule's pieces, shared by its own kernel
// and by the few-row product that quantizes its input itself:
//
//   amax = max(max_k |x_k|, 2^-100),  s = amax / 127,  q_k = rint(x_k r),
//   r = 127 / amax (rounded to FP32)
//
// so |x_k - s q_k| <= s / 2 up to FP32 rounding, and the largest element maps
// to +-127.  A row that holds an infinity or a NaN has no scale: its s is NaN
// and its q zero, so that whatever is computed from it is NaN.
//
// A row's maximum is kept as the bits of |x| in FP32: magnitudes order as
// their bits do, with infinity and NaN above all.
#pragma once

#include "device.h"
#include "pieces.h"

namespace mm {

constexpr float kQuantFloor = 7.888609052210118e-31f;  // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// The 16-byte chunk of row x that starts at column c0, zeros past cols.
template <int DT>
__device__ __forceinline__ uint4 quant_load(const typename Elem<DT>::S *x, int64_t c0, int64_t cols) {
    using S = typename Elem<DT>::S;
    return row_piece<S>((GlobalPtr<S>)(x + c0), cols - c0, cols >= Elem<DT>::kVE);
}

template <int DT>
__device__ __forceinline__ uint32_t quant_top(const uint4 &v, uint32_t m) {
    constexpr int VE = Elem<DT>::kVE;
    typename Elem<DT>::S e[VE];
    __builtin_memcpy(e, &v, 16);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        const uint32_t b = __float_as_uint(Elem<DT>::to_f32(e[i])) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}

__device__ __forceinline__ float quant_scale(uint32_t top) {
    return top >= kInfBits ? __uint_as_float(0x7fc00000u) : fmaxf(__uint_as_float(top), kQuantFloor) / 127.0f;
}

// r, or 0 for a row without a scale.
__device__ __forceinline__ float quant_factor(uint32_t top) {
    return top >= kInfBits ? 0.0f : 127.0f / fmaxf(__uint_as_float(top), kQuantFloor);
}

// A chunk's INT8 values (kVE bytes) to q, which may have any alignment.
template <int DT>
__device__ __forceinline__ void quant_bytes(const uint4 &v, float r, int8_t *o) {
    constexpr int VE = Elem<DT>::kVE;
    typename Elem<DT>::S e[VE];
    __builtin_memcpy(e, &v, 16);
#pragma unroll
    for (int i = 0; i < VE; ++i) o[i] = r == 0.0f ? (int8_t)0 : (int8_t)(int)rintf(Elem<DT>::to_f32(e[i]) * r);
}

template <int DT>
__device__ __forceinline__ void quant_store(const uint4 &v, float r, char *q) {
    int8_t o[Elem<DT>::kVE];
    quant_bytes<DT>(v, r, o);
    __builtin_memcpy(q, o, Elem<DT>::kVE);
}

}  // namespace mm
