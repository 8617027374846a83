// ffn_choice.h -- what the plans of the feed-forward operators share: limits on
// sizes, and the choice of kernel, tile entry and split by estimated time
// (plan_ffn.cpp).
#pragma once

#include <math.h>

#include "ffn.h"
#include "plan.h"

namespace mm {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

inline mm_status launched(hipError_t e) {
    return e == hipSuccess ? MM_OK : fail(MM_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

// Matrices of at most 2^40 elements: their byte counts and the kernels' grids
// then stay in range (and the memory of any device is smaller).
inline bool too_large(int64_t rows, int64_t cols) { return (double)rows * (double)cols > 1099511627776.0; }

// Sizes and pitches, rounded up to whole chunks, are 32-bit in the kernels.
constexpr int64_t kMaxSize = (int64_t)INT32_MAX - 64;

// A launch has at most 2^32 - 1 threads.
inline bool launchable(double wgs, int threads) { return wgs * threads < 4294967296.0; }

// Whether an entry's grid for `batch` products of M x cols can be launched.
// Operands that are not 16-byte aligned run entry 1 in entry 0's place: four
// times its workgroups, of half its size.
inline bool tile_launchable(const FfnChoice &c, int64_t batch, int64_t M, int64_t cols) {
    const FfnTile &t = kFfnTiles[c.tile];
    const double wgs = (double)batch * (double)cdiv(M, t.bm) * (double)cdiv(cols, t.bn) * c.split;
    return launchable(c.tile == 0 ? 4.0 * wgs : wgs, c.tile <= 1 ? 256 : 512);
}

// The same for kernels of 256 threads that take `pieces` of each of M rows: the
// joining of partial sums (four columns a thread) and the backward pass's
// element-wise part.
inline bool pieces_launchable(int64_t M, int64_t pieces) {
    return launchable(ceil((double)M * (double)pieces / 256.0), 256);
}

inline bool float_type(int t) { return t == MM_FLOAT || t == MM_FLOAT16 || t == MM_BFLOAT16; }

// Classes of operand types that the time model tells apart; the linear layer's
// 16-bit products run another kernel on entries 0 and 4 (k_big.h).
enum { kClass16 = 0, kClass8 = 1, kClass32 = 2, kClassLinear16 = 3 };
int type_class(int dtype);

double rows_us(int cls, bool nk, int64_t M, int64_t N, int64_t kbytes, int64_t row, double wbytes);
// The same for the linear layer.
double linear_rows_us(int cls, bool nk, int64_t M, int64_t N, int64_t kbytes, int64_t row, double wbytes);
double tiles_us(int cls, const FfnChoice &c, bool nk, bool aligned, int64_t row, double wbytes);
FfnChoice choose(int cls, bool aligned, int64_t batch, int64_t M, int64_t cols, int64_t kbytes, int terms,
                 unsigned tiles, bool may_split);
// Whether a product of an entry's tiles runs faster as whole rounds of workgroups
// over its first columns and another entry (of `tiles`) over the rest: the first
// column of the rest and its entry, c then is the first's; or 0.
int64_t balance(int cls, FfnChoice *c, int64_t M, int64_t N, int64_t kbytes, unsigned tiles, int *rest);
void set_split(FfnChoice *c, int64_t kbytes, int terms, int64_t split);
mm_status tile_option(const mm_plan_options *opt, int *tile);
mm_status choose_backward(const char *name, int cls, bool aligned, int64_t batch, int64_t M, int64_t cols,
                          int64_t kbytes, int terms, unsigned tiles, int treq, int sreq, FfnChoice *c);
mm_status forced_alone(const mm_plan_options *opt);

}  // namespace mm
