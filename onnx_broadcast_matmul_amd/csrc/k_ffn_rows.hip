// k_ffn_rows.hip -- the gated block and the scaled INT8 product over few rows
// (one decoded token to kFfnRows of them), weights stored [N, K].
//
// The weights are the traffic: each is read once, straight into MFMA
// operands.  A workgroup owns 16 hidden features (the gate and the up rows)
// or 32 outputs of the INT8 product as two 16-row operands; its waves take
// every NWV-th 256-byte block of K and their sums meet in LDS in wave order,
// so the result does not depend on timing.  X (a few rows) is re-read by every
// workgroup from cache.  Rows of any alignment are read in 16-byte pieces;
// only the end of K, less than one block, goes element by element.
#include "activation.h"
#include "device.h"
#include "ffn.h"

namespace mm {

typedef int i32x4v __attribute__((ext_vector_type(4)));

template <int DT, int OD, bool GLU, int MB, int NWV>
__global__ __launch_bounds__(64 * NWV) void k_ffn_rows(FfnArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
    using E = Elem<DT>;
    using S = typename E::S;
    using OE = Elem<OD>;
    constexpr bool INT = DT == MM_INT8;
    constexpr int ES = (int)sizeof(S);
    constexpr int VE = 16 / ES;
    constexpr int U = 4;               // 16-byte pieces per lane, row and block
    constexpr int BK = 256 / ES;       // K elements of a block
    using AccT = typename std::conditional<INT, i32x4v, f32x4>::type;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t M = a.M, N = a.N, K = a.K;
    const int64_t n0 = (int64_t)blockIdx.x * (GLU ? 16 : 32);
    const int64_t lasta = a.lda, lastb = a.ldb;
    // Rows past the end read the last row; their results are not stored.
    const S *w[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int64_t n = n0 + (GLU ? 0 : 16 * p) + r;
        w[p] = (const S *)a.B[GLU ? p : 0] + (n < N ? n : N - 1) * lastb + g * VE;
    }
    const S *x[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int64_t m = 16 * i + r;
        x[i] = (const S *)a.A[0] + (m < M ? m : M - 1) * lasta + g * VE;
    }

    AccT acc[2][MB];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[p][i][e] = 0;

    struct Block {
        uint4 w[2][U], x[MB][U];
    };
    auto load = [&](int64_t kb, Block &t) {
        const int64_t k0 = kb * BK;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int p = 0; p < 2; ++p) __builtin_memcpy(&t.w[p][u], w[p] + k0 + u * 4 * VE, 16);
#pragma unroll
            for (int i = 0; i < MB; ++i) __builtin_memcpy(&t.x[i][u], x[i] + k0 + u * 4 * VE, 16);
        }
    };
    auto load_tail = [&](int64_t kb, Block &t) {
        auto piece = [&](const S *src, int64_t left) {
            S tmp[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) tmp[e] = e < left ? src[e] : (S)0;
            uint4 v;
            __builtin_memcpy(&v, tmp, 16);
            return v;
        };
        const int64_t k0 = kb * BK;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t left = K - (k0 + (u * 4 + g) * VE);
#pragma unroll
            for (int p = 0; p < 2; ++p) t.w[p][u] = piece(w[p] + k0 + u * 4 * VE, left);
#pragma unroll
            for (int i = 0; i < MB; ++i) t.x[i][u] = piece(x[i] + k0 + u * 4 * VE, left);
        }
    };
    auto mul = [&](const Block &t) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    const uint4 &y = t.w[p][u], &z = t.x[i][u];
                    if constexpr (INT) {
                        acc[p][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4v, y),
                                                                         __builtin_bit_cast(i32x4v, z), acc[p][i], 0, 0, 0);
                    } else if constexpr (DT == MM_BFLOAT16) {
                        acc[p][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, y), __builtin_bit_cast(bf16x8, z), acc[p][i], 0, 0, 0);
                    } else if constexpr (DT == MM_FLOAT16) {
                        acc[p][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            __builtin_bit_cast(f16x8, y), __builtin_bit_cast(f16x8, z), acc[p][i], 0, 0, 0);
                    } else {
                        acc[p][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.x), __uint_as_float(z.x), acc[p][i], 0, 0, 0);
                        acc[p][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.y), __uint_as_float(z.y), acc[p][i], 0, 0, 0);
                        acc[p][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.z), __uint_as_float(z.z), acc[p][i], 0, 0, 0);
                        acc[p][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.w), __uint_as_float(z.w), acc[p][i], 0, 0, 0);
                    }
                }
    };
    // Whole blocks with the next one's loads in flight, then the end of K.
    const int64_t nb = K / BK;
    Block cur, nxt;
    if (wave < nb) load(wave, cur);
    for (int64_t kb = wave; kb < nb; kb += NWV) {
        const bool more = kb + NWV < nb;
        if (more) load(kb + NWV, nxt);
        mul(cur);
        if (more) cur = nxt;
    }
    if (nb * BK < K && wave == (int)(nb % NWV)) {
        load_tail(nb, cur);
        mul(cur);
    }

    // Element e of lane is weight row 4 (lane / 16) + e and X row lane % 16.
    using P = typename std::conditional<INT, int, float>::type;
    __shared__ __attribute__((aligned(16))) P red[NWV][2][MB][256];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < MB; ++i) *(AccT *)&red[wave][p][i][r * 16 + 4 * g] = acc[p][i];
    __syncthreads();
    using OS = typename OE::S;
    if constexpr (GLU) {
        for (int idx = tid; idx < MB * 256; idx += 64 * NWV) {
            const int i = idx >> 8, at = idx & 255;
            const int64_t m = 16 * i + (at >> 4), n = n0 + (at & 15);
            if (m >= M || n >= N) continue;
            float sg = 0.0f, su = 0.0f;
#pragma unroll
            for (int v = 0; v < NWV; ++v) {
                sg += red[v][0][i][at];
                su += red[v][1][i][at];
            }
            const int64_t o = m * a.ldy + n;
            if (a.G) {
                ((OS *)a.G)[o] = OE::from_f32(sg);
                ((OS *)a.U)[o] = OE::from_f32(su);
            }
            constexpr bool X = DT == MM_FLOAT;
            float f;
            switch (a.act) {
            case MM_ACT_SILU: f = act_value<MM_ACT_SILU, X>(sg); break;
            case MM_ACT_GELU: f = act_value<MM_ACT_GELU, X>(sg); break;
            case MM_ACT_GELU_TANH: f = act_value<MM_ACT_GELU_TANH, X>(sg); break;
            case MM_ACT_RELU: f = act_value<MM_ACT_RELU, X>(sg); break;
            default: f = act_value<MM_ACT_SIGMOID, X>(sg); break;
            }
            ((OS *)a.Y[0])[o] = OE::from_f32(f * su);
        }
    } else {
        for (int idx = tid; idx < MB * 512; idx += 64 * NWV) {
            const int i = idx >> 9, m16 = (idx >> 5) & 15, c = idx & 31;
            const int64_t m = 16 * i + m16, n = n0 + c;
            if (m >= M || n >= N) continue;
            int sum = 0;
#pragma unroll
            for (int v = 0; v < NWV; ++v) sum += (int)red[v][c >> 4][i][m16 * 16 + (c & 15)];
            const float bias = a.bias ? OE::to_f32(((const OS *)a.bias)[n]) : 0.0f;
            ((OS *)a.Y[0])[m * a.ldy + n] = OE::from_f32(scaled_value(sum, a.sa[m], a.sb[n], bias));
        }
    }
#endif
}

template <int DT, int OD, bool GLU>
static hipError_t rows(const FfnArgs &a, hipStream_t s) {
    const int64_t wgs = (a.N + (GLU ? 15 : 31)) / (GLU ? 16 : 32);
    if (wgs <= 0 || a.M <= 0) return hipSuccess;
    if (wgs > 0x7fffffff || a.M > kFfnRows) return hipErrorInvalidValue;
    constexpr int NWV = 8;
    const dim3 gr((unsigned)wgs), bl(64 * NWV);
    if (a.M <= 16) hipLaunchKernelGGL((k_ffn_rows<DT, OD, GLU, 1, NWV>), gr, bl, 0, s, a);
    else hipLaunchKernelGGL((k_ffn_rows<DT, OD, GLU, 2, NWV>), gr, bl, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_glu_rows(int dtype, const FfnArgs &a, hipStream_t s) {
    switch (dtype) {
    case MM_FLOAT: return rows<MM_FLOAT, MM_FLOAT, true>(a, s);
    case MM_FLOAT16: return rows<MM_FLOAT16, MM_FLOAT16, true>(a, s);
    case MM_BFLOAT16: return rows<MM_BFLOAT16, MM_BFLOAT16, true>(a, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_scaled_rows(int od, const FfnArgs &a, hipStream_t s) {
    switch (od) {
    case MM_FLOAT: return rows<MM_INT8, MM_FLOAT, false>(a, s);
    case MM_FLOAT16: return rows<MM_INT8, MM_FLOAT16, false>(a, s);
    case MM_BFLOAT16: return rows<MM_INT8, MM_BFLOAT16, false>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
