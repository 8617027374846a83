// k_glu.hip -- gated feed-forward block: dispatch of the tiled products by
// element type, and the element-wise part of the backward pass.
#include <type_traits>

#include "activation.h"
#include "device.h"
#include "ffn.h"

namespace mm {

#define MM_GLU_DECLARE(NAME)                                                                               \
    hipError_t glu_fwd_##NAME(bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);    \
    hipError_t glu_dx_##NAME(bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);     \
    hipError_t glu_dw_##NAME(int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);
MM_GLU_DECLARE(f32)
MM_GLU_DECLARE(f16)
MM_GLU_DECLARE(bf16)

hipError_t launch_glu_fwd(int dtype, bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {
    return dtype == MM_FLOAT ? glu_fwd_f32(tb, tile, split, vec, a, s)
           : dtype == MM_FLOAT16 ? glu_fwd_f16(tb, tile, split, vec, a, s) : glu_fwd_bf16(tb, tile, split, vec, a, s);
}

hipError_t launch_glu_dx(int dtype, bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {
    return dtype == MM_FLOAT ? glu_dx_f32(tb, tile, split, vec, a, s)
           : dtype == MM_FLOAT16 ? glu_dx_f16(tb, tile, split, vec, a, s) : glu_dx_bf16(tb, tile, split, vec, a, s);
}

hipError_t launch_glu_dw(int dtype, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {
    return dtype == MM_FLOAT ? glu_dw_f32(tile, split, vec, a, s)
           : dtype == MM_FLOAT16 ? glu_dw_f16(tile, split, vec, a, s) : glu_dw_bf16(tile, split, vec, a, s);
}

// f(g) for an activation known at run time.
template <bool EXACT>
__device__ __forceinline__ float act_switch(int act, float g) {
    switch (act) {
    case MM_ACT_SILU: return act_value<MM_ACT_SILU, EXACT>(g);
    case MM_ACT_GELU: return act_value<MM_ACT_GELU, EXACT>(g);
    case MM_ACT_GELU_TANH: return act_value<MM_ACT_GELU_TANH, EXACT>(g);
    case MM_ACT_RELU: return act_value<MM_ACT_RELU, EXACT>(g);
    default: return act_value<MM_ACT_SIGMOID, EXACT>(g);
    }
}

// Forward pass over split K: the partitions' G and U added in partition order,
// then the tiled kernel's epilogue.  A thread owns four consecutive elements
// of the dense [M, N] outputs.
template <int DT>
__global__ __launch_bounds__(256) void k_glu_reduce(FfnSlim a) {
    using E = Elem<DT>;
    using S = typename E::S;
    const int64_t total = (int64_t)a.M * a.N;
    const int64_t i0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i0 >= total) return;
    const int n = total - i0 < 4 ? (int)(total - i0) : 4;
    const float *w = (const float *)a.W() + i0;
    float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (total % 4 == 0) {
#pragma unroll 4
        for (int p = 0; p < a.split; ++p) {
            const float4 x = *(const float4 *)(w + 2 * p * total), y = *(const float4 *)(w + (2 * p + 1) * total);
            g[0] += x.x; g[1] += x.y; g[2] += x.z; g[3] += x.w;
            u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
        }
    } else {
        for (int p = 0; p < a.split; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) {
                    g[e] += w[2 * p * total + e];
                    u[e] += w[(2 * p + 1) * total + e];
                }
    }
    S og[4], ou[4], oh[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        og[e] = E::from_f32(g[e]);
        ou[e] = E::from_f32(u[e]);
        oh[e] = E::from_f32(act_switch<DT == MM_FLOAT>(a.act, g[e]) * u[e]);
    }
    auto put = [&](void *p, const auto *v) {
        auto *y = (typename std::remove_const<typename std::remove_pointer<decltype(v)>::type>::type *)p + i0;
        if (n == 4) __builtin_memcpy(y, v, 4 * sizeof(*v));
        else
            for (int e = 0; e < n; ++e) y[e] = v[e];
    };
    if (a.G()) {
        if (DT != MM_FLOAT && a.kept32()) {
            put(a.G(), g);
            put(a.U(), u);
        } else {
            put(a.G(), og);
            put(a.U(), ou);
        }
    }
    put(a.Y[0], oh);
}

hipError_t launch_glu_reduce(int dtype, const FfnArgs &a, hipStream_t s) {
    const int64_t g = ((a.M * a.N + 3) / 4 + 255) / 256;
    if (g <= 0) return hipSuccess;
    if (g > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 gr((unsigned)g), bl(256);
    const FfnSlim r = slim_args<FfnSlim>(a, kUseGlu, false, true);
    if (dtype == MM_FLOAT) hipLaunchKernelGGL(k_glu_reduce<MM_FLOAT>, gr, bl, 0, s, r);
    else if (dtype == MM_FLOAT16) hipLaunchKernelGGL(k_glu_reduce<MM_FLOAT16>, gr, bl, 0, s, r);
    else hipLaunchKernelGGL(k_glu_reduce<MM_BFLOAT16>, gr, bl, 0, s, r);
    return hipGetLastError();
}

// Sum of the K partitions' FP32 partials in partition order, narrowed once;
// product b (blockIdx.y of gridDim.y) goes to Y[b], rows ldy elements apart.  A
// thread owns four consecutive columns of one row.  The launch bounds it
// (300 x 512, 6 partitions: 4.0 us, of which 3 are an empty kernel's).
template <int DT>
__global__ __launch_bounds__(256) void k_sum_reduce(FfnSlim a) {
    using E = Elem<DT>;
    using S = typename E::S;
    const uint32_t N = (uint32_t)a.N, cpr = (N + 3) / 4;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= (int64_t)a.M * cpr) return;
    const int64_t row = x < 0x7fffffff ? (int64_t)((uint32_t)x / cpr) : x / cpr;
    const uint32_t col = (uint32_t)(x - row * cpr) * 4;
    const int64_t stride = (int64_t)gridDim.y * a.M * N;
    const float *w = (const float *)a.W() + (int64_t)blockIdx.y * a.M * N + row * N + col;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    S *y = (S *)a.Y[blockIdx.y] + row * a.ldy + col;
    if (N % 4 == 0) {
#pragma unroll 4
        for (int p = 0; p < a.split; ++p) {
            const float4 v = *(const float4 *)(w + p * stride);
            acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
        }
    } else {
        for (int p = 0; p < a.split; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < N) acc[e] += w[p * stride + e];
    }
    S out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = E::from_f32(acc[e]);
    if (col + 4 <= N) __builtin_memcpy(y, out, sizeof(out));
    else
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < N) y[e] = out[e];
}

hipError_t launch_sum_reduce(int dtype, const FfnArgs &a, hipStream_t s) {
    const int64_t g = (a.M * ((a.N + 3) / 4) + 255) / 256;
    if (g <= 0 || a.batch <= 0) return hipSuccess;
    if (g > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 gr((unsigned)g, (unsigned)a.batch), bl(256);
    const FfnSlim r = slim_args<FfnSlim>(a, kUsePlain, false, true);
    if (dtype == MM_FLOAT) hipLaunchKernelGGL(k_sum_reduce<MM_FLOAT>, gr, bl, 0, s, r);
    else if (dtype == MM_FLOAT16) hipLaunchKernelGGL(k_sum_reduce<MM_FLOAT16>, gr, bl, 0, s, r);
    else hipLaunchKernelGGL(k_sum_reduce<MM_BFLOAT16>, gr, bl, 0, s, r);
    return hipGetLastError();
}

// dG = dH U f'(G) and dU = dH f(G), a thread per 16 bytes of each tensor's
// row.  Three tensors are read and two written once, which bounds it (8192 x
// 11008 BF16: 0.90 GB in 151 us, 6.0 TB/s, and 1.26 GB in 210 us with FP32 G and
// U; 4096 x 5504 41 and 48 us).  A kernel of its
// own because dX reduces over N and dW over M: formed inside those products it
// would be formed once for every tile column.  G and U come as the forward
// pass kept them (KT): FP32 sums, or rounded to the element type, which halves
// their bytes and makes BF16 gradients off by 0.0031 of their norm, not 0.0024.
// dG and dU are rounded to the element type because the matrix cores take them
// in it.  They have rows of ldw elements, whole 16-byte chunks; the columns past
// N hold zeros, so the products may read them.
template <int DT, int KT, int ACT>
__global__ __launch_bounds__(256) void k_glu_dact(const void *G, const void *U, const void *dH, void *dG, void *dU,
                                                  int64_t M, int64_t N, int64_t ldw) {
    using E = Elem<DT>;
    using S = typename E::S;
    using KE = Elem<KT>;
    using KS = typename KE::S;
    constexpr int VE = E::kVE;
    const int64_t cpr = ldw / VE;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= M * cpr) return;
    // cpr < 2^31: one 32-bit division where the index allows it.
    const int64_t row = x < 0x7fffffff ? (int64_t)((uint32_t)x / (uint32_t)cpr) : x / cpr;
    const int64_t col = (x - row * cpr) * VE, i0 = row * N + col;
    KS g[VE], u[VE];
    S h[VE], og[VE], ou[VE];
    if (col + VE <= N) {
        __builtin_memcpy(g, (const KS *)G + i0, sizeof(g));
        __builtin_memcpy(u, (const KS *)U + i0, sizeof(u));
        __builtin_memcpy(h, (const S *)dH + i0, 16);
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const bool in = col + e < N;
            g[e] = in ? ((const KS *)G)[i0 + e] : (KS)0;
            u[e] = in ? ((const KS *)U)[i0 + e] : (KS)0;
            h[e] = in ? ((const S *)dH)[i0 + e] : (S)0;
        }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        float f, d;
        act_grad<ACT, DT == MM_FLOAT>(KE::to_f32(g[e]), f, d);
        const float dh = E::to_f32(h[e]);
        og[e] = E::from_f32(dh * KE::to_f32(u[e]) * d);
        ou[e] = E::from_f32(dh * f);
    }
    uint4 vg, vu;
    __builtin_memcpy(&vg, og, 16);
    __builtin_memcpy(&vu, ou, 16);
    *(uint4 *)((S *)dG + row * ldw + col) = vg;
    *(uint4 *)((S *)dU + row * ldw + col) = vu;
}

template <int DT, int KT, int ACT>
static hipError_t dact(const void *G, const void *U, const void *dH, void *dG, void *dU, int64_t M, int64_t N,
                       int64_t ldw, hipStream_t s) {
    const int64_t g = (M * (ldw / Elem<DT>::kVE) + 255) / 256;
    if (g <= 0) return hipSuccess;
    if (g > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_glu_dact<DT, KT, ACT>), dim3((unsigned)g), dim3(256), 0, s, G, U, dH, dG, dU, M, N, ldw);
    return hipGetLastError();
}

template <int DT, int KT>
static hipError_t dact(int act, const void *G, const void *U, const void *dH, void *dG, void *dU, int64_t M, int64_t N,
                       int64_t ldw, hipStream_t s) {
    switch (act) {
    case MM_ACT_SILU: return dact<DT, KT, MM_ACT_SILU>(G, U, dH, dG, dU, M, N, ldw, s);
    case MM_ACT_GELU: return dact<DT, KT, MM_ACT_GELU>(G, U, dH, dG, dU, M, N, ldw, s);
    case MM_ACT_GELU_TANH: return dact<DT, KT, MM_ACT_GELU_TANH>(G, U, dH, dG, dU, M, N, ldw, s);
    case MM_ACT_RELU: return dact<DT, KT, MM_ACT_RELU>(G, U, dH, dG, dU, M, N, ldw, s);
    case MM_ACT_SIGMOID: return dact<DT, KT, MM_ACT_SIGMOID>(G, U, dH, dG, dU, M, N, ldw, s);
    }
    return hipErrorInvalidValue;
}

template <int DT>
static hipError_t dact(int kept, int act, const void *G, const void *U, const void *dH, void *dG, void *dU, int64_t M,
                       int64_t N, int64_t ldw, hipStream_t s) {
    return kept == DT ? dact<DT, DT>(act, G, U, dH, dG, dU, M, N, ldw, s)
                      : dact<DT, MM_FLOAT>(act, G, U, dH, dG, dU, M, N, ldw, s);
}

hipError_t launch_glu_dact(int dtype, int kept, int act, const void *G, const void *U, const void *dH, void *dG, void *dU,
                           int64_t M, int64_t N, int64_t ldw, hipStream_t s) {
    return dtype == MM_FLOAT ? dact<MM_FLOAT>(kept, act, G, U, dH, dG, dU, M, N, ldw, s)
           : dtype == MM_FLOAT16 ? dact<MM_FLOAT16>(kept, act, G, U, dH, dG, dU, M, N, ldw, s)
                                 : dact<MM_BFLOAT16>(kept, act, G, U, dH, dG, dU, M, N, ldw, s);
}

}  // namespace mm
