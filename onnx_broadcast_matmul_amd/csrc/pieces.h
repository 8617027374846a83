// pieces.h -- 16-byte pieces of matrix rows of any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mm {

template <typename S>
using GlobalPtr = const __attribute__((address_space(1))) S *;

// Vectors at any address.
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2u __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32u __attribute__((aligned(1)));

// 16 bytes at any address: one load.
template <typename S>
__device__ __forceinline__ uint4 whole_piece(GlobalPtr<S> p) {
    return __builtin_bit_cast(uint4, *(const __attribute__((address_space(1))) u32x4u *)p);
}

// The same of a tensor that is read once, and stored to one that is written
// once: past the caches, which then do not turn over for them (8192 x 11008
// BF16 to a checkpoint and back 111 -> 87 us, a copy of it 5.5 -> 6.2 TB/s).
template <typename S>
__device__ __forceinline__ uint4 stream_piece(GlobalPtr<S> p) {
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const __attribute__((address_space(1))) u32x4u *)p));
}

__device__ __forceinline__ void stream_store(void *p, const uint4 &v) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4u, v), (u32x4u *)p);
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

// row_piece in two steps, for rows that are read several pieces at a time: the
// loads of all of them first, without a test (rows of at least a piece: a
// piece that would pass the row's end ends there), and what the end needs where
// they are used.  row_piece waits for its piece before the next one is asked for
// (8192 x 4096 BF16 norms forward: 75 us so, 61 in two steps).
// ONCE: a tensor that is streamed through (see stream_piece).  Offset: holds the
// row's bytes.  A row may be longer than 2^32 bytes; where it cannot be, 32 bits are
// one register for a row whose address is uniform.
template <typename S, bool ONCE = false, typename Offset = uint64_t>
__device__ __forceinline__ uint4 edge_load(GlobalPtr<S> row, int n, int c) {
    constexpr int ES = (int)sizeof(S), VE = 16 / ES;
    using Bytes = const __attribute__((address_space(1))) char *;
    if (n >= VE) {
        const GlobalPtr<S> p = (GlobalPtr<S>)((Bytes)row + (Offset)(uint32_t)(c < n - VE ? c : n - VE) * ES);
        return ONCE ? stream_piece<S>(p) : whole_piece<S>(p);
    }
    S tmp[VE];  // the whole row
#pragma unroll
    for (int e = 0; e < VE; ++e) tmp[e] = e < n ? row[e] : (S)0;
    uint4 v;
    __builtin_memcpy(&v, tmp, 16);
    return v;
}

// What edge_load read at c of a row of n: the piece, zeros past the end.  (c + VE
// may pass 2^31 in a row of nearly as many.)
template <typename S>
__device__ __forceinline__ uint4 edge_piece(uint4 v, int n, int c) {
    constexpr int ES = (int)sizeof(S), VE = 16 / ES;
    if (c <= n - VE || (n < VE && c == 0)) return v;
    const int miss = VE - (n - c);
    uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
    const int sh = miss * ES * 8;
    if (miss >= VE) {
        lo = hi = 0;
    } else if (sh >= 64) {
        lo = hi >> (sh - 64);
        hi = 0;
    } else {
        lo = lo >> sh | hi << (64 - sh);
        hi >>= sh;
    }
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}

}  // namespace mm
