// pieces.h -- 16-byte pieces of matrix rows of any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mm {

template <typename S>
using GlobalPtr = const __attribute__((address_space(1))) S *;

// 16 bytes at any address: one load.
template <typename S>
__device__ __forceinline__ uint4 whole_piece(GlobalPtr<S> p) {
    typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
    return __builtin_bit_cast(uint4, *(const __attribute__((address_space(1))) u32x4u *)p);
}

// The piece at p of a row that ends `left` elements after p: those elements
// and zeros behind them (left <= 0: zeros, nothing is read).  `back`: the row
// is at least a piece long, so a piece at its end is read ending there and
// shifted down; shorter rows are read element by element.
template <typename S>
__device__ __forceinline__ uint4 row_piece(GlobalPtr<S> p, int64_t left, bool back) {
    constexpr int ES = (int)sizeof(S), VE = 16 / ES;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (left <= 0) return v;
    if (back) {
        const int miss = left < VE ? VE - (int)left : 0;
        v = whole_piece<S>(p - miss);
        uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
        const int sh = miss * ES * 8;
        if (sh >= 64) {
            lo = hi >> (sh - 64);
            hi = 0;
        } else if (sh > 0) {
            lo = lo >> sh | hi << (64 - sh);
            hi >>= sh;
        }
        v = make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
        asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
        return v;
    }
    S tmp[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) tmp[e] = e < left ? p[e] : (S)0;
    __builtin_memcpy(&v, tmp, 16);
    // Packed here (and shifted above): otherwise whole pieces are waited for,
    // taken apart and packed again where the paths meet.
    if constexpr (ES == 1) asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
    return v;
}

}  // namespace mm
