// checkpoint.h -- 8-bit activation checkpoints: the format's pieces, shared by
// everything that writes or reads one.
//
// A block of 32 elements of a row holds q s with s = 2^(E - 6), E = floor(log2
// (max |x|)) (of at least 2^-100), q = rint(x / s) limited to +-127; its scale
// byte is E + 127, or 255 where the block held an infinity or a NaN.  x / s and q s
// are exact in FP32 and |q| < 2^7, so q s is a BF16 number too and, of an FP16
// tensor, an FP16 one: what reads a checkpoint rounds nothing.
//
// Magnitudes are kept as the bits of |x| in FP32, which order as the
// magnitudes do, with infinity and NaN above all; E + 127 is their upper part.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mm {

constexpr int kCkBlock = 32;
constexpr uint32_t kCkFloor = (127u - 100u) << 23;  // 2^-100

__device__ __forceinline__ uint32_t ck_magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale byte of a block whose largest magnitude is `top`.
__device__ __forceinline__ uint32_t ck_exponent(uint32_t top) { return (top > kCkFloor ? top : kCkFloor) >> 23; }

// 1 / s, or 0 for the byte 255.
__device__ __forceinline__ float ck_inverse(uint32_t ex) { return ex == 255u ? 0.0f : __uint_as_float((260u - ex) << 23); }

// s, or NaN.  (No byte below 27 is written; those that a caller brings are
// taken as 2^-126 at least.)
__device__ __forceinline__ float ck_scale(uint32_t ex) {
    return __uint_as_float(ex == 255u ? 0x7fc00000u : (ex > 7u ? ex - 6u : 1u) << 23);
}

// q as a float.  A block without a scale has 1 / s = 0: its NaNs and infinities
// must not reach the conversion.
__device__ __forceinline__ float ck_number(float x, float inv) {
    return inv == 0.0f ? 0.0f : __builtin_amdgcn_fmed3f(rintf(x * inv), -127.0f, 127.0f);
}

// Four whole numbers of -128 .. 127 as bytes, the first lowest.
__device__ __forceinline__ uint32_t pack_bytes(float a, float b, float c, float d) {
    return ((uint32_t)(int)a & 255u) | ((uint32_t)(int)b & 255u) << 8 | ((uint32_t)(int)c & 255u) << 16 |
           (uint32_t)(int)d << 24;
}

// The four numbers of a word of bytes, times s.
__device__ __forceinline__ void unpack_bytes(uint32_t w, float s, float *x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)(int)(int8_t)(w >> (8 * e)) * s;
}

}  // namespace mm
