// k_norm.hip -- fused norms: dispatch by element type (the kernels stand in
// k_norm.h) and the joining of the backward pass's column sums.
#include "device.h"
#include "join.h"
#include "norm.h"

namespace mm {

#define MM_NORM_DECLARE(NAME)                                                      \
    hipError_t norm_fwd_##NAME(bool train, const NormFwdTrain &a, hipStream_t s);  \
    hipError_t norm_bwd_##NAME(int kept, const NormBwd &a, hipStream_t s);
MM_NORM_DECLARE(f32)
MM_NORM_DECLARE(f16)
MM_NORM_DECLARE(bf16)

hipError_t launch_norm_fwd(int dtype, bool train, const NormFwdTrain &a, hipStream_t s) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    return dtype == MM_FLOAT ? norm_fwd_f32(train, a, s)
           : dtype == MM_FLOAT16 ? norm_fwd_f16(train, a, s) : norm_fwd_bf16(train, a, s);
}

hipError_t launch_norm_bwd(int dtype, int kept, const NormBwd &a, hipStream_t s) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    return dtype == MM_FLOAT ? norm_bwd_f32(kept, a, s)
           : dtype == MM_FLOAT16 ? norm_bwd_f16(kept, a, s) : norm_bwd_bf16(kept, a, s);
}

// The workers' sums, in worker order within each of 32 slices (see join.h):
// blockIdx.y < jobs, a weight's or a bias's; behind them, a group of gate rows.
template <int DT>
__global__ __launch_bounds__(256) void k_norm_join(NormJoin a) {
    using E = Elem<DT>;
    using S = typename E::S;
    const int64_t c0 = (int64_t)blockIdx.x * 32, left = a.ldp - c0;
    float v;
    S *out;
    if ((int)blockIdx.y < a.jobs) {
        v = join_columns(a.workers, left, [&](int64_t i) { return a.part + (i * a.jobs + blockIdx.y) * a.ldp + c0; });
        out = (S *)a.out[blockIdx.y];
    } else {
        const int64_t g = blockIdx.y - a.jobs, begin = g * a.gate_rows;
        const int64_t end = begin + a.gate_rows < a.M ? begin + a.gate_rows : a.M;
        const int64_t w0 = begin / a.per, w1 = (end - 1) / a.per;
        v = join_columns(w1 - w0 + 1, left, [&](int64_t i) {
            const int64_t w = w0 + i;
            return a.gpart + (w * 2 + (w * a.per / a.gate_rows == g ? 0 : 1)) * a.ldp + c0;
        });
        out = (S *)a.dgate + g * a.N;
    }
    if (threadIdx.x < 32 && c0 + threadIdx.x < a.N) out[c0 + threadIdx.x] = E::from_f32(v);
}

hipError_t launch_norm_join(int dtype, const NormJoin &a, hipStream_t s) {
    const int64_t gx = (a.N + 31) / 32, gy = (int64_t)a.jobs + (a.gpart ? a.groups : 0);
    if (gx <= 0 || gy <= 0) return hipSuccess;
    if (gy > 65535) return hipErrorInvalidValue;
    const dim3 g((unsigned)gx, (unsigned)gy), b(256);
    if (dtype == MM_FLOAT) hipLaunchKernelGGL(k_norm_join<MM_FLOAT>, g, b, 0, s, a);
    else if (dtype == MM_FLOAT16) hipLaunchKernelGGL(k_norm_join<MM_FLOAT16>, g, b, 0, s, a);
    else hipLaunchKernelGGL(k_norm_join<MM_BFLOAT16>, g, b, 0, s, a);
    return hipGetLastError();
}

}  // namespace mm
