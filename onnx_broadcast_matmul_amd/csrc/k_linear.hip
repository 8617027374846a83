// k_linear.hip -- linear layer: dispatch of the tiled products by element type,
// the joining of a split product with the epilogue, what the backward products
// need first, and the joining of column sums.
#include <type_traits>

#include "activation.h"
#include "checkpoint.h"
#include "device.h"
#include "ffn.h"
#include "join.h"
#include "pieces.h"

namespace mm {

#define MM_LINEAR_DECLARE(NAME)                                                                         \
    hipError_t linear_##NAME(bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);  \
    hipError_t linear_dw_##NAME(int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s);
MM_LINEAR_DECLARE(f32)
MM_LINEAR_DECLARE(f16)
MM_LINEAR_DECLARE(bf16)

hipError_t launch_linear(int dtype, bool tb, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {
    return dtype == MM_FLOAT ? linear_f32(tb, tile, split, vec, a, s)
           : dtype == MM_FLOAT16 ? linear_f16(tb, tile, split, vec, a, s) : linear_bf16(tb, tile, split, vec, a, s);
}

hipError_t launch_linear_dw(int dtype, int tile, bool split, bool vec, const FfnArgs &a, hipStream_t s) {
    return dtype == MM_FLOAT ? linear_dw_f32(tile, split, vec, a, s)
           : dtype == MM_FLOAT16 ? linear_dw_f16(tile, split, vec, a, s) : linear_dw_bf16(tile, split, vec, a, s);
}

// Forward pass over split K: the partitions' sums added in partition order,
// then the tiled kernel's epilogue.  A thread owns four consecutive columns of
// one row, eight threads a checkpoint block of Z.
template <int DT>
__global__ __launch_bounds__(256) void k_linear_reduce(FfnSlim a) {
    using E = Elem<DT>;
    using S = typename E::S;
    const uint32_t N = (uint32_t)a.N, nb = (N + 31) / 32, cpr = nb * 8;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (x >= (int64_t)a.M * cpr) return;  // whole groups of eight
    const int64_t row = x < 0x7fffffff ? (int64_t)((uint32_t)x / cpr) : x / cpr;
    const uint32_t col = (uint32_t)(x - row * cpr) * 4;
    const int n = col >= N ? 0 : N - col < 4 ? (int)(N - col) : 4;
    const int64_t stride = (int64_t)a.M * N, at = row * N + col;
    const float *w = (const float *)a.W() + at;
    float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (N % 4 == 0 && n > 0) {
#pragma unroll 4
        for (int p = 0; p < a.split; ++p) {
            const float4 v = *(const float4 *)(w + p * stride);
            z[0] += v.x; z[1] += v.y; z[2] += v.z; z[3] += v.w;
        }
    } else {
        for (int p = 0; p < a.split; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) z[e] += w[p * stride + e];
    }
    if (a.lin_bias()) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) z[e] += E::to_f32(((const S *)a.lin_bias())[col + e]);
    }
    auto put = [&](void *p, const auto *v) {
        auto *y = (typename std::remove_const<typename std::remove_pointer<decltype(v)>::type>::type *)p + at;
        if (n == 4) __builtin_memcpy(y, v, 4 * sizeof(*v));
        else
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) y[e] = v[e];
    };
    if (a.G()) {
        if (a.q8()) {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, ck_magnitude(z[e]));
#pragma unroll
            for (int d = 1; d < 8; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
            const uint32_t ex = ck_exponent(top);
            const float inv = ck_inverse(ex);
            const uint32_t w = ck_word(z[0], z[1], z[2], z[3], inv);
            int8_t q[4];
            __builtin_memcpy(q, &w, 4);
            put(a.G(), q);
            if (col % 32 == 0) ((uint8_t *)a.zs())[row * nb + col / 32] = (uint8_t)ex;
        } else if (DT != MM_FLOAT && a.kept32()) {
            put(a.G(), z);
        } else {
            S o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = E::from_f32(z[e]);
            put(a.G(), o);
        }
    }
    S y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float v = act_run<DT == MM_FLOAT>(a.act, z[e]);
        if (a.R() && e < n) v += E::to_f32(((const S *)a.R())[at + e]);
        y[e] = E::from_f32(v);
    }
    put(a.Y[0], y);
}

hipError_t launch_linear_reduce(int dtype, const FfnArgs &a, hipStream_t s) {
    const int64_t g = (a.M * ((a.N + 31) / 32 * 8) + 255) / 256;
    if (g <= 0) return hipSuccess;
    if (g > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 gr((unsigned)g), bl(256);
    const FfnSlim r = slim_args<FfnSlim>(a, kUseLinear, false, true);
    if (dtype == MM_FLOAT) hipLaunchKernelGGL(k_linear_reduce<MM_FLOAT>, gr, bl, 0, s, r);
    else if (dtype == MM_FLOAT16) hipLaunchKernelGGL(k_linear_reduce<MM_FLOAT16>, gr, bl, 0, s, r);
    else hipLaunchKernelGGL(k_linear_reduce<MM_BFLOAT16>, gr, bl, 0, s, r);
    return hipGetLastError();
}

// ---- before the backward products

// Blocks [0, prep_z) form dZ and its column sums: 32 threads along a row, 16
// bytes each, eight rows side by side, `rows` rows.  The blocks behind them turn
// the checkpoint of X into rows of the products' type.  Memory bounds both.
template <int DT, int ZT>
__global__ __launch_bounds__(256) void k_linear_prep(LinearPrep a, uint32_t prep_z) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int VE = E::kVE;
    constexpr bool EXACT = DT == MM_FLOAT;
    if (blockIdx.x < prep_z) {
        using ZE = Elem<ZT == 0 || ZT == MM_INT8 ? DT : ZT>;
        using ZS = typename ZE::S;
        constexpr int ZV = ZE::kVE, ZP = ZT == 0 || ZT == MM_INT8 ? 1 : VE / ZV, U = 2;
        const int t = threadIdx.x & 31, r = threadIdx.x >> 5;
        const uint32_t ncb = (uint32_t)((a.ldz + 32 * VE - 1) / (32 * VE));
        const int64_t rb = blockIdx.x / ncb;
        const int N = (int)a.N, col = ((int)(blockIdx.x % ncb) * 32 + t) * VE, nb = (N + 31) / 32;
        const int64_t end = (rb + 1) * a.rows < a.M ? (rb + 1) * a.rows : a.M;
        float sum[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) sum[e] = 0.0f;
        if (col < N) {
            for (int64_t row0 = rb * a.rows + r; row0 < end; row0 += 8 * U) {
                uint4 hv[U], zv[U][ZP];
                uint32_t w[U][VE / 4];
                float sc[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t row = row0 + 8 * u < end ? row0 + 8 * u : row0;
                    hv[u] = edge_load<S, true>((GlobalPtr<S>)((const S *)a.dY + row * N), N, col);
                    if constexpr (ZT == MM_INT8) {
                        ck_load<VE>((const int8_t *)a.Z + row * N, N, col, w[u]);
                        sc[u] = ck_scale(((const uint8_t *)a.zs)[row * nb + col / kCkBlock]);
                    } else if constexpr (ZT != 0) {
#pragma unroll
                        for (int i = 0; i < ZP; ++i)
                            zv[u][i] = edge_load<ZS, true>((GlobalPtr<ZS>)((const ZS *)a.Z + row * N), N, col + i * ZV);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t row = row0 + 8 * u;
                    if (row >= end) break;
                    S h[VE];
                    hv[u] = edge_piece<S>(hv[u], N, col);
                    __builtin_memcpy(h, &hv[u], 16);
                    float d[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) d[e] = E::to_f32(h[e]);
                    if constexpr (ZT != 0) {
                        float z[VE];
                        if constexpr (ZT == MM_INT8) {
#pragma unroll
                            for (int i = 0; i < VE / 4; ++i) unpack_bytes(w[u][i], sc[u], z + 4 * i);
                        } else {
#pragma unroll
                            for (int i = 0; i < ZP; ++i) {
                                ZS v[ZV];
                                const uint4 p = edge_piece<ZS>(zv[u][i], N, col + i * ZV);
                                __builtin_memcpy(v, &p, 16);
#pragma unroll
                                for (int e = 0; e < ZV; ++e) z[i * ZV + e] = ZE::to_f32(v[e]);
                            }
                        }
                        auto slope = [&](auto kind) {
#pragma unroll
                            for (int e = 0; e < VE; ++e) {
                                float f, g;
                                act_grad<decltype(kind)::value, EXACT>(z[e], f, g);
                                d[e] *= g;
                            }
                        };
                        switch (a.act) {
                        case MM_ACT_SILU: slope(std::integral_constant<int, MM_ACT_SILU>()); break;
                        case MM_ACT_GELU: slope(std::integral_constant<int, MM_ACT_GELU>()); break;
                        case MM_ACT_GELU_TANH: slope(std::integral_constant<int, MM_ACT_GELU_TANH>()); break;
                        case MM_ACT_RELU: slope(std::integral_constant<int, MM_ACT_RELU>()); break;
                        default: slope(std::integral_constant<int, MM_ACT_SIGMOID>()); break;
                        }
                        S o[VE];
#pragma unroll
                        for (int e = 0; e < VE; ++e) o[e] = E::from_f32(col + e < N ? d[e] : 0.0f);
                        uint4 ov;
                        __builtin_memcpy(&ov, o, 16);
                        *(uint4 *)((S *)a.dZ + row * a.ldz + col) = ov;
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e) sum[e] += d[e];
                }
            }
        }
        if (!a.part) return;
        __shared__ float part[8][32][VE + 1];
#pragma unroll
        for (int e = 0; e < VE; ++e) part[r][t][e] = sum[e];
        __syncthreads();
        const int64_t c0 = (int64_t)(blockIdx.x % ncb) * 32 * VE;
        for (int x = threadIdx.x; x < 32 * VE; x += 256) {
            if (c0 + x >= N) break;
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v += part[i][x / VE][x % VE];
            a.part[rb * a.ldp + c0 + x] = v;
        }
        return;
    }
    constexpr int U = 4;
    const int K = (int)a.K, nb = (K + 31) / 32;
    const int64_t cpr = a.ldx / VE, total = a.M * cpr;
    uint32_t w[U][VE / 4];
    float sc[U];
    int64_t to[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int64_t x = ((int64_t)(blockIdx.x - prep_z) * U + u) * 256 + threadIdx.x;
        to[u] = x < total ? x * VE : -1;
        x = x < total ? x : 0;
        const int64_t row = x < 0x7fffffff ? (int64_t)((uint32_t)x / (uint32_t)cpr) : x / cpr;
        col[u] = (int)(x - row * cpr) * VE;
        ck_load<VE>((const int8_t *)a.xq + row * K, K, col[u], w[u]);
        sc[u] = ck_scale(((const uint8_t *)a.xs)[row * nb + col[u] / kCkBlock]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (to[u] < 0) break;
        float v[VE];
#pragma unroll
        for (int i = 0; i < VE / 4; ++i) unpack_bytes(w[u][i], sc[u], v + 4 * i);
        S o[VE];
        if (a.x_act != MM_ACT_NONE) {
#pragma unroll
            for (int e = 0; e < VE; ++e) v[e] = act_run<EXACT>(a.x_act, v[e]);
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) o[e] = E::from_f32(col[u] + e < K ? v[e] : 0.0f);
        uint4 ov;
        __builtin_memcpy(&ov, o, 16);
        *(uint4 *)((S *)a.X + to[u]) = ov;
    }
}

static int64_t prep_z_blocks(const LinearPrep &a, int ve) {
    if (!a.dZ && !a.part) return 0;
    return (a.M + a.rows - 1) / a.rows * ((a.ldz + 32 * ve - 1) / (32 * ve));
}

int64_t linear_prep_blocks(const LinearPrep &a, int dtype) {
    const int ve = dtype == MM_FLOAT ? 4 : 8;
    return prep_z_blocks(a, ve) + (a.X ? (a.M * (a.ldx / ve) + 1023) / 1024 : 0);
}

template <int DT>
static hipError_t prep(const LinearPrep &a, hipStream_t s) {
    const int64_t g = linear_prep_blocks(a, DT);
    if (g <= 0) return hipSuccess;
    if (g > 0xffffff) return hipErrorInvalidValue;
    const dim3 gr((unsigned)g), bl(256);
    const uint32_t pz = (uint32_t)prep_z_blocks(a, Elem<DT>::kVE);
    if (!a.dZ) hipLaunchKernelGGL((k_linear_prep<DT, 0>), gr, bl, 0, s, a, pz);
    else if (a.z_type == DT) hipLaunchKernelGGL((k_linear_prep<DT, DT>), gr, bl, 0, s, a, pz);
    else if (a.z_type == MM_INT8) hipLaunchKernelGGL((k_linear_prep<DT, MM_INT8>), gr, bl, 0, s, a, pz);
    else hipLaunchKernelGGL((k_linear_prep<DT, MM_FLOAT>), gr, bl, 0, s, a, pz);
    return hipGetLastError();
}

hipError_t launch_linear_prep(int dtype, const LinearPrep &a, hipStream_t s) {
    return dtype == MM_FLOAT ? prep<MM_FLOAT>(a, s) : dtype == MM_FLOAT16 ? prep<MM_FLOAT16>(a, s) : prep<MM_BFLOAT16>(a, s);
}

// ---- column sums

// A workgroup joins 32 columns (see join.h).
template <int DT>
__global__ __launch_bounds__(256) void k_join(JoinArgs a) {
    using E = Elem<DT>;
    const int64_t c0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 32;
    if (c0 >= a.N) return;
    const float v = join_columns(a.P, a.ldp - c0, [&](int64_t i) { return a.part + i * a.ldp + c0; });
    if (threadIdx.x < 32 && c0 + threadIdx.x < a.N) ((typename E::S *)a.out)[c0 + threadIdx.x] = E::from_f32(v);
}

hipError_t launch_join(int dtype, const JoinArgs &a, hipStream_t s) {
    // One dimension of a grid holds less than 2^32 threads: 2^29 columns.
    const int64_t g = (a.N + 31) / 32, gx = g < (1 << 23) ? g : (1 << 23);
    if (g <= 0) return hipSuccess;
    if (g > 0x7ffffff) return hipErrorInvalidValue;
    const dim3 gr((unsigned)gx, (unsigned)((g + gx - 1) / gx)), bl(256);
    if (dtype == MM_FLOAT) hipLaunchKernelGGL(k_join<MM_FLOAT>, gr, bl, 0, s, a);
    else if (dtype == MM_FLOAT16) hipLaunchKernelGGL(k_join<MM_FLOAT16>, gr, bl, 0, s, a);
    else hipLaunchKernelGGL(k_join<MM_BFLOAT16>, gr, bl, 0, s, a);
    return hipGetLastError();
}

}  // namespace mm
