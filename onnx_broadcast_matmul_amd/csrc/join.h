// join.h -- joining partial column sums: what a workgroup of 256 threads does
// for 32 columns.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mm {

// The sum over i < P of row(i)[c], c = 0 .. 31: eight threads of four columns,
// 32 slices of the rows, the slices' sums added in order.  Threads 0 .. 31 get
// column threadIdx.x.  row(i) gives the address of 32 columns (of `left`, a
// multiple of four).
template <class Row>
__device__ __forceinline__ float join_columns(int64_t P, int64_t left, Row row) {
    __shared__ float part[32][33];
    const int t = threadIdx.x & 7, slice = threadIdx.x >> 3;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t * 4 < left) {
#pragma unroll 4
        for (int64_t i = slice; i < P; i += 32) {
            const float4 v = *(const float4 *)(row(i) + t * 4);
            sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
        }
    }
    part[slice][t * 4] = sum.x;
    part[slice][t * 4 + 1] = sum.y;
    part[slice][t * 4 + 2] = sum.z;
    part[slice][t * 4 + 3] = sum.w;
    __syncthreads();
    float v = 0.0f;
    if (threadIdx.x < 32) {
#pragma unroll 8
        for (int i = 0; i < 32; ++i) v += part[i][threadIdx.x];
    }
    return v;
}

}  // namespace mm
