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

#include <type_traits>

#include "device.h"
#include "pieces.h"

namespace mm {

constexpr int kCkBlock = 32;
constexpr uint32_t kCkFloor = (127u - 100u) << 23;  // 2^-100

__device__ __forceinline__ uint32_t ck_magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The largest magnitude of 16 bytes of a row.  16-bit types order as their bits do.
template <int DT>
__device__ __forceinline__ uint32_t piece_top(const uint4 &v) {
    if constexpr (DT == MM_FLOAT) {
        return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
    } else {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2, w & 0x7fff7fffu); };
        const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag(v.x), mag(v.y)),
                                                  __builtin_elementwise_max(mag(v.z), mag(v.w)));
        return __float_as_uint(Elem<DT>::to_f32(m.x > m.y ? m.x : m.y));
    }
}

// The largest of a block, of which 32 / VE neighbouring lanes hold VE elements
// each: within quads, then (four elements a lane) across the two quads.
template <int VE>
__device__ __forceinline__ uint32_t block_top(uint32_t top) {
    auto other = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, true);
    };
    top = max(top, other(top, std::integral_constant<int, 0xb1>()));  // quad_perm 1 0 3 2
    top = max(top, other(top, std::integral_constant<int, 0x4e>()));  // quad_perm 2 3 0 1
    if constexpr (VE == 4) top = max(top, other(top, std::integral_constant<int, 0x141>()));  // row_half_mirror
    return top;
}

// The scale byte of a block whose largest magnitude is `top`.
__device__ __forceinline__ uint32_t ck_exponent(uint32_t top) { return (top > kCkFloor ? top : kCkFloor) >> 23; }

// 1 / s, or 0 for the byte 255.
__device__ __forceinline__ float ck_inverse(uint32_t ex) { return ex == 255u ? 0.0f : __uint_as_float((260u - ex) << 23); }

// s, or NaN.  (No byte below 27 is written; those that a caller brings are
// taken as 2^-126 at least.)
__device__ __forceinline__ float ck_scale(uint32_t ex) {
    return __uint_as_float(ex == 255u ? 0x7fc00000u : (ex > 7u ? ex - 6u : 1u) << 23);
}

// q as a whole number n in FP32, or (ck_word) four of them as bytes, the first
// lowest.  x / s + 1.5 2^23 is rounded to a whole number, ties to even, whose low
// byte is n's; the limits apply to that sum.  A block without a scale has
// 1 / s = 0 and its numbers are 0, whatever it holds.
constexpr float kCkMagic = 12582912.0f;  // 1.5 2^23

__device__ __forceinline__ float ck_sum(float x, float inv) {
    return __builtin_amdgcn_fmed3f(fmaf(x, inv, kCkMagic), kCkMagic - 127.0f, kCkMagic + 127.0f);
}

__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
    const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x0c0c0400u);
    const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x04000c0cu);
    return ab | cd;
}

__device__ __forceinline__ uint32_t ck_word(float a, float b, float c, float d, float inv) {
    const uint32_t w = low_bytes(ck_sum(a, inv), ck_sum(b, inv), ck_sum(c, inv), ck_sum(d, inv));
    return inv == 0.0f ? 0u : w;
}

// The four numbers of a word of bytes, times s (less m, rounded once).
__device__ __forceinline__ void unpack_bytes(uint32_t w, float s, float *x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)(int)(int8_t)(w >> (8 * e)) * s;
}
__device__ __forceinline__ void unpack_bytes(uint32_t w, float s, float m, float *x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = fmaf((float)(int)(int8_t)(w >> (8 * e)), s, -m);
}

// VE bytes (4 or 8) of a row of n at c; past the end zeros.  Checkpoints are
// streamed through (see pieces.h).
template <int VE>
__device__ __forceinline__ void ck_load(const int8_t *row, int n, int c, uint32_t *w) {
    if (c <= n - VE) {
        if constexpr (VE == 4) {
            w[0] = __builtin_nontemporal_load((const u32u *)(row + (uint32_t)c));
        } else {
            const u32x2u v = __builtin_nontemporal_load((const u32x2u *)(row + (uint32_t)c));
            w[0] = v.x;
            w[1] = v.y;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) w[i] = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e)
        if (c + e < n) w[e / 4] |= (uint32_t)(uint8_t)row[c + e] << (e % 4 * 8);
}

// Words of numbers to a row of n at c, as far as it goes.
template <int VE>
__device__ __forceinline__ void ck_store(int8_t *row, int n, int c, const uint32_t *w) {
    if (c <= n - VE) {
        if constexpr (VE == 4) {
            __builtin_nontemporal_store(w[0], (u32u *)(row + (uint32_t)c));
        } else {
            const u32x2u v = {w[0], w[1]};
            __builtin_nontemporal_store(v, (u32x2u *)(row + (uint32_t)c));
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < VE; ++e)
        if (c + e < n) row[c + e] = (int8_t)(w[e / 4] >> (e % 4 * 8));
}

}  // namespace mm
