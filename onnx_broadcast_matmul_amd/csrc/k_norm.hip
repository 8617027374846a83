// k_norm.hip -- norms before and after a block, fused with its gate and residual
// scale, and their backward pass:
//
//   n1 = norm1(B) w1 + b1 (or B)    R = X + alpha g n1    Y = norm2(R) w2 + b2
//
// The threads of a row hold it in registers from the first load to the last
// store, so every tensor is read or written once: memory bounds long runs of
// rows, the launch a few.  The variance of a layer norm is formed from the
// differences to the mean (a second sum over the registers), so that a large
// mean costs no digits.
#include "checkpoint.h"
#include "device.h"
#include "join.h"
#include "norm.h"
#include "pieces.h"

namespace mm {

// ---- sums over the threads of a row

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float x) {
    const int y = __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, true);
    return x + __int_as_float(y);
}

// The wave's sum, in every lane: within rows of 16 lanes, then across them.
__device__ __forceinline__ float wave_sum(float x) {
    x = dpp_add<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8
    x = dpp_add<0x112, 0xf>(x);
    x = dpp_add<0x114, 0xf>(x);
    x = dpp_add<0x118, 0xf>(x);
    x = dpp_add<0x142, 0xa>(x);  // row_bcast 15, 31
    x = dpp_add<0x143, 0xc>(x);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// Sums of two values over the TPR threads of a row.  Above a wave they meet in
// LDS; `turn` alternates between two buffers, so that one barrier serves: a
// buffer is written again only after the next sum's barrier, which every
// reader has passed.
template <int NT, int TPR>
struct RowSums {
    static constexpr int W = TPR / 64;
    float2 (*part)[NT / 64];
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
        float2 s = make_float2(wave_sum(a), wave_sum(b));
        if constexpr (TPR > 64) {
            const int wave = threadIdx.x >> 6, first = wave / W * W;
            if ((threadIdx.x & 63) == 0) part[turn][wave] = s;
            __syncthreads();
            s = part[turn][first];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                const float2 o = part[turn][first + i];
                s.x += o.x;
                s.y += o.y;
            }
            turn ^= 1;
        }
        return s;
    }
};

// ---- rows in pieces of 16 bytes (VE columns)

template <int DT>
__device__ __forceinline__ void piece_floats(const uint4 &v, float *x) {
    constexpr int VE = Elem<DT>::kVE;
    typename Elem<DT>::S e[VE];
    __builtin_memcpy(e, &v, 16);
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = Elem<DT>::to_f32(e[i]);
}

// The piece of row p (of N columns) at column c; NULL and past the end: zeros.
template <int DT>
__device__ __forceinline__ uint4 piece_at(const void *p, int64_t row, int N, int c) {
    using S = typename Elem<DT>::S;
    if (!p) return make_uint4(0, 0, 0, 0);
    return row_piece<S>((GlobalPtr<S>)((const S *)p + row * N + c), N - c, N >= Elem<DT>::kVE);
}

// x rounded to the type, in both forms.
template <int DT>
__device__ __forceinline__ void piece_store(void *p, int64_t row, int N, int c, const float *x, float *rounded) {
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int VE = E::kVE;
    S o[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        o[i] = E::from_f32(x[i]);
        if (rounded) rounded[i] = E::to_f32(o[i]);
    }
    if (!p) return;
    S *y = (S *)p + row * N + c;
    if (c + VE <= N) __builtin_memcpy(y, o, 16);
    else
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (c + i < N) y[i] = o[i];
}

// The checkpoint of a piece; 32 / VE neighbouring lanes hold a block.
template <int DT>
__device__ __forceinline__ void piece_checkpoint(void *q, void *scale, int64_t row, int N, int c, const float *x) {
    constexpr int VE = Elem<DT>::kVE;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i)
        if (c + i < N) top = max(top, ck_magnitude(x[i]));
#pragma unroll
    for (int d = 1; d < kCkBlock / VE; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const uint32_t ex = ck_exponent(top);
    const float inv = ck_inverse(ex);
    uint32_t w[VE / 4];
#pragma unroll
    for (int i = 0; i < VE / 4; ++i)
        w[i] = pack_bytes(ck_number(x[4 * i], inv), ck_number(x[4 * i + 1], inv), ck_number(x[4 * i + 2], inv),
                          ck_number(x[4 * i + 3], inv));
    int8_t *o = (int8_t *)q + row * N + c;
    if (c + VE <= N) __builtin_memcpy(o, w, VE);
    else
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (c + i < N) o[i] = (int8_t)(w[i / 4] >> (i % 4 * 8));
    if (c < N && c % kCkBlock == 0) ((uint8_t *)scale)[row * ((N + 31) / 32) + c / kCkBlock] = (uint8_t)ex;
}

// ---- forward

constexpr int kFwdCols = 16;  // columns of a thread

template <int DT, int TPR, bool TRAIN>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_fwd(typename std::conditional<TRAIN, NormFwdTrain, NormFwd>::type a) {
    constexpr int VE = Elem<DT>::kVE, CH = kFwdCols / VE, NT = TPR < 256 ? 256 : TPR;
    __shared__ float2 part[2][NT / 64];
    RowSums<NT, TPR> sums{part};
    const int t = threadIdx.x % TPR, N = a.N;
    const int64_t at = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (NT / TPR) + threadIdx.x / TPR;
    const bool live = at < a.M;  // every thread reaches the barriers
    const int64_t row = live ? at : a.M - 1;
    const float inv_n = 1.0f / (float)N;
    auto col = [&](int i) { return (i * TPR + t) * VE; };
    uint4 xr[CH], br[CH], gr[CH];
    const int64_t grow = a.gate ? row / a.gate_rows : 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) br[i] = piece_at<DT>(a.B, row, N, col(i));
#pragma unroll
    for (int i = 0; i < CH; ++i) xr[i] = piece_at<DT>(a.X, row, N, col(i));
#pragma unroll
    for (int i = 0; i < CH; ++i) gr[i] = piece_at<DT>(a.gate, grow, N, col(i));
    // Mean and reciprocal deviation of v.
    auto moments = [&](int kind, float eps, const float (*v)[VE]) {
        float mean = 0.0f, s = 0.0f;
        if (kind == MM_NORM_LAYER) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) s += v[i][e];
            mean = sums(s, 0.0f).x * inv_n;
            s = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = col(i) + e < N ? v[i][e] - mean : 0.0f;
                s = fmaf(d, d, s);
            }
        return make_float2(mean, 1.0f / sqrtf(sums(s, 0.0f).x * inv_n + eps));
    };
    float2 m1 = make_float2(0.0f, 1.0f), m2 = m1;
    float v[CH][VE];
    if (a.B) {
#pragma unroll
        for (int i = 0; i < CH; ++i) piece_floats<DT>(br[i], v[i]);
        if constexpr (TRAIN) {
            if (a.bq && live) {
#pragma unroll
                for (int i = 0; i < CH; ++i) piece_checkpoint<DT>(a.bq, a.bs, row, N, col(i), v[i]);
            }
        }
        if (a.post != MM_NORM_NONE) m1 = moments(a.post, a.eps1, v);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float w[VE], x[VE];
            if (a.post != MM_NORM_NONE) {
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] = (v[i][e] - m1.x) * m1.y;
                if (a.w1) {
                    piece_floats<DT>(piece_at<DT>(a.w1, 0, N, col(i)), w);
#pragma unroll
                    for (int e = 0; e < VE; ++e) v[i][e] *= w[e];
                }
                if (a.b1) {
                    piece_floats<DT>(piece_at<DT>(a.b1, 0, N, col(i)), w);
#pragma unroll
                    for (int e = 0; e < VE; ++e) v[i][e] += w[e];
                }
            }
            piece_floats<DT>(xr[i], x);
            if (a.gate) {
                piece_floats<DT>(gr[i], w);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] *= w[e];
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = col(i) + e < N ? fmaf(a.alpha, v[i][e], x[e]) : 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) piece_floats<DT>(xr[i], v[i]);
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if constexpr (TRAIN) {
                float r[VE];
                piece_store<DT>(a.R, row, N, col(i), v[i], r);
                if (a.r32) {
#pragma unroll
                    for (int k = 0; k < VE / 4; ++k) piece_store<MM_FLOAT>(a.r32, row, N, col(i) + 4 * k, v[i] + 4 * k, nullptr);
                }
                if (a.rq) piece_checkpoint<DT>(a.rq, a.rs, row, N, col(i), r);
            } else if (a.R) {
                piece_store<DT>(a.R, row, N, col(i), v[i], nullptr);
            }
        }
    }
    if (a.pre != MM_NORM_NONE) {
        m2 = moments(a.pre, a.eps2, v);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float w[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = (v[i][e] - m2.x) * m2.y;
            if (a.w2) {
                piece_floats<DT>(piece_at<DT>(a.w2, 0, N, col(i)), w);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] *= w[e];
            }
            if (a.b2) {
                piece_floats<DT>(piece_at<DT>(a.b2, 0, N, col(i)), w);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] += w[e];
            }
            if (!live) continue;
            if constexpr (TRAIN) {
                float r[VE];
                piece_store<DT>(a.Y, row, N, col(i), v[i], r);
                if (a.yq) piece_checkpoint<DT>(a.yq, a.ys, row, N, col(i), r);
            } else {
                piece_store<DT>(a.Y, row, N, col(i), v[i], nullptr);
            }
        }
    }
    if constexpr (TRAIN) {
        if (a.stats && live && t == 0) *(float4 *)(a.stats + row * 4) = make_float4(m1.x, m1.y, m2.x, m2.y);
    }
}

static int fwd_threads(int64_t N) { return N <= 64 * kFwdCols ? 64 : N <= 256 * kFwdCols ? 256 : N <= 512 * kFwdCols ? 512 : 1024; }

template <int DT, int TPR>
static hipError_t fwd(bool train, const NormFwdTrain &a, hipStream_t s) {
    constexpr int NT = TPR < 256 ? 256 : TPR;
    // One dimension of a grid holds less than 2^32 threads.
    const int64_t n = ((int64_t)a.M + NT / TPR - 1) / (NT / TPR), gx = n < (1 << 21) ? n : (1 << 21);
    const dim3 g((unsigned)gx, (unsigned)((n + gx - 1) / gx)), b(NT);
    if (train) hipLaunchKernelGGL((k_norm_fwd<DT, TPR, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_norm_fwd<DT, TPR, false>), g, b, 0, s, (const NormFwd &)a);
    return hipGetLastError();
}

template <int DT>
static hipError_t fwd(bool train, const NormFwdTrain &a, hipStream_t s) {
    if (a.N > 1024 * kFwdCols) return hipErrorInvalidValue;
    switch (fwd_threads(a.N)) {
    case 64: return fwd<DT, 64>(train, a, s);
    case 256: return fwd<DT, 256>(train, a, s);
    case 512: return fwd<DT, 512>(train, a, s);
    default: return fwd<DT, 1024>(train, a, s);
    }
}

hipError_t launch_norm_fwd(int dtype, bool train, const NormFwdTrain &a, hipStream_t s) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    return dtype == MM_FLOAT ? fwd<MM_FLOAT>(train, a, s)
           : dtype == MM_FLOAT16 ? fwd<MM_FLOAT16>(train, a, s) : fwd<MM_BFLOAT16>(train, a, s);
}

// ---- backward

// What a thread holds of one row before it is converted.
template <int DT, int KEPT, int CH>
struct NormRaw {
    static constexpr int VE = Elem<DT>::kVE;
    static constexpr bool KEPT8 = KEPT == MM_INT8;
    static constexpr int RP = KEPT8 ? 1 : VE / Elem<KEPT8 ? DT : KEPT>::kVE;  // pieces of R in place of one
    using Kept = typename std::conditional<KEPT8, uint32_t[VE / 4], uint4>::type;
    uint4 dy[CH], ds[CH];
    Kept r[CH * RP], b[CH];
    float rs[CH], bs[CH];  // checkpoints: the blocks' scales
    float4 st;
};

// VE bytes of a checkpoint row and their scale; NULL and past the end: zeros.
template <int VE>
__device__ __forceinline__ void kept_piece(const void *p, const void *scale, int64_t row, int N, int c, uint32_t *w, float &s) {
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) w[i] = 0;
    s = 0.0f;
    if (!p || c >= N) return;
    const int8_t *q = (const int8_t *)p + row * N + c;
    if (c + VE <= N) __builtin_memcpy(w, q, VE);
    else
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (c + i < N) w[i / 4] |= (uint32_t)(uint8_t)q[i] << (i % 4 * 8);
    s = ck_scale(((const uint8_t *)scale)[row * ((N + 31) / 32) + c / kCkBlock]);
}

template <int DT, int KEPT, int TPR, int COLS>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_bwd(NormBwd a) {
    constexpr int VE = Elem<DT>::kVE, CH = COLS / VE, NT = TPR < 256 ? 256 : TPR;
    __shared__ float2 part[2][NT / 64];
    RowSums<NT, TPR> sums{part};
    const int t = threadIdx.x % TPR, N = a.N;
    const int worker = (int)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
    const int64_t r0 = (int64_t)worker * a.per, r1 = r0 + a.per < a.M ? r0 + a.per : a.M;
    const float inv_n = 1.0f / (float)N;
    auto col = [&](int i) { return (i * TPR + t) * VE; };
    using Raw = NormRaw<DT, KEPT, CH>;
    constexpr bool KEPT8 = Raw::KEPT8;
    constexpr int RP = Raw::RP, RV = VE / RP;
    auto load = [&](int64_t row, Raw &x) {
        if (row >= r1) return;
        x.st = *(const float4 *)(a.stats + row * 4);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            x.dy[i] = piece_at<DT>(a.dY, row, N, col(i));
            x.ds[i] = piece_at<DT>(a.dS, row, N, col(i));
            if constexpr (KEPT8) {
                kept_piece<VE>(a.R, a.rs, row, N, col(i), x.r[i], x.rs[i]);
                kept_piece<VE>(a.B, a.bs, row, N, col(i), x.b[i], x.bs[i]);
            } else {
#pragma unroll
                for (int k = 0; k < RP; ++k) x.r[i * RP + k] = piece_at<KEPT>(a.R, row, N, col(i) + k * RV);
                x.b[i] = piece_at<DT>(a.B, row, N, col(i));
            }
        }
    };
    // Weights stay as they lie in memory; absent ones count as 1.
    uint4 w1[CH], w2[CH], gate[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        w1[i] = piece_at<DT>(a.w1, 0, N, col(i));
        w2[i] = piece_at<DT>(a.w2, 0, N, col(i));
    }
    float sum[4][CH][VE], gsum[CH][VE];  // dw1, db1, dw2, db2; dgate of the group
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            sum[0][i][e] = sum[1][i][e] = sum[2][i][e] = sum[3][i][e] = 0.0f;
            gsum[i][e] = 0.0f;
        }
    int64_t group = -1;
    const int64_t group0 = a.gate_rows ? r0 / a.gate_rows : 0;
    auto finish_group = [&]() {
        if (!a.dgate || group < 0) return;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (a.gpart) {
                float *p = a.gpart + ((int64_t)worker * 2 + (group == group0 ? 0 : 1)) * a.ldp + col(i);
#pragma unroll
                for (int e = 0; e < VE; e += 4)
                    if (col(i) + e < N)  // ldp is a multiple of four
                        *(float4 *)(p + e) = make_float4(gsum[i][e], gsum[i][e + 1], gsum[i][e + 2], gsum[i][e + 3]);
            } else {
                piece_store<DT>(a.dgate, group, N, col(i), gsum[i], nullptr);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) gsum[i][e] = 0.0f;
        }
    };
    Raw cur, nxt;
    load(r0, cur);
    for (int it = 0; it < a.per; ++it) {
        const int64_t row = r0 + it;
        const bool live = row < r1;  // every thread reaches the barriers
        load(row + 1, nxt);
        if (live && a.gate_rows && row / a.gate_rows != group) {
            finish_group();
            group = row / a.gate_rows;
#pragma unroll
            for (int i = 0; i < CH; ++i) gate[i] = piece_at<DT>(a.gate, group, N, col(i));
        }
        float d[CH][VE], x[CH][VE], w[VE], y[VE];
        // dR, from dY through the second norm and from dS.
        if (a.pre != MM_NORM_NONE) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                if constexpr (KEPT8) {
#pragma unroll
                    for (int k = 0; k < VE / 4; ++k) unpack_bytes(cur.r[i][k], cur.rs[i], x[i] + 4 * k);
                } else {
#pragma unroll
                    for (int k = 0; k < RP; ++k) piece_floats<KEPT>(cur.r[i * RP + k], x[i] + k * RV);
                }
                piece_floats<DT>(cur.dy[i], y);
                if (a.w2) piece_floats<DT>(w2[i], w);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    x[i][e] = (x[i][e] - cur.st.z) * cur.st.w;
                    d[i][e] = a.w2 ? y[e] * w[e] : y[e];
                    if (live) {
                        sum[2][i][e] = fmaf(y[e], x[i][e], sum[2][i][e]);
                        sum[3][i][e] += y[e];
                    }
                    s0 += d[i][e];
                    s1 = fmaf(d[i][e], x[i][e], s1);
                }
            }
            const float2 s = sums(s0, s1);
            const float mean = a.pre == MM_NORM_LAYER ? s.x * inv_n : 0.0f, proj = s.y * inv_n;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                piece_floats<DT>(cur.ds[i], y);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    d[i][e] = col(i) + e < N ? fmaf(cur.st.w, d[i][e] - mean - x[i][e] * proj, y[e]) : 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_floats<DT>(cur.ds[i], d[i]);
        }
        if (live && a.dX) {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_store<DT>(a.dX, row, N, col(i), d[i], nullptr);
        }
        if (a.dB || a.dgate || a.slot[0] >= 0 || a.slot[1] >= 0) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                // x: the normalised B (or B), y: n1, d: dn1
                if constexpr (KEPT8) {
#pragma unroll
                    for (int k = 0; k < VE / 4; ++k) unpack_bytes(cur.b[i][k], cur.bs[i], x[i] + 4 * k);
                } else {
                    piece_floats<DT>(cur.b[i], x[i]);
                }
                if (a.post != MM_NORM_NONE) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) x[i][e] = (x[i][e] - cur.st.x) * cur.st.y;
                }
                if (a.dgate && live) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) y[e] = x[i][e];
                    if (a.w1) {
                        piece_floats<DT>(w1[i], w);
#pragma unroll
                        for (int e = 0; e < VE; ++e) y[e] *= w[e];
                    }
                    if (a.b1) {
                        piece_floats<DT>(piece_at<DT>(a.b1, 0, N, col(i)), w);
#pragma unroll
                        for (int e = 0; e < VE; ++e) y[e] += w[e];
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e) gsum[i][e] = fmaf(a.alpha * d[i][e], y[e], gsum[i][e]);
                }
                if (a.gate_rows) piece_floats<DT>(gate[i], w);
#pragma unroll
                for (int e = 0; e < VE; ++e) d[i][e] *= a.gate_rows ? a.alpha * w[e] : a.alpha;
                if (a.post != MM_NORM_NONE) {
                    if (a.w1) piece_floats<DT>(w1[i], w);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        if (live) {
                            sum[0][i][e] = fmaf(d[i][e], x[i][e], sum[0][i][e]);
                            sum[1][i][e] += d[i][e];
                        }
                        if (a.w1) d[i][e] *= w[e];
                        s0 += d[i][e];
                        s1 = fmaf(d[i][e], x[i][e], s1);
                    }
                }
            }
            if (a.dB) {
                if (a.post != MM_NORM_NONE) {
                    const float2 s = sums(s0, s1);
                    const float mean = a.post == MM_NORM_LAYER ? s.x * inv_n : 0.0f, proj = s.y * inv_n;
#pragma unroll
                    for (int i = 0; i < CH; ++i)
#pragma unroll
                        for (int e = 0; e < VE; ++e) d[i][e] = cur.st.y * (d[i][e] - mean - x[i][e] * proj);
                }
                if (live) {
#pragma unroll
                    for (int i = 0; i < CH; ++i) piece_store<DT>(a.dB, row, N, col(i), d[i], nullptr);
                }
            }
        }
        cur = nxt;
    }
    finish_group();
    if (worker >= a.workers) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (a.slot[k] < 0) continue;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float *p = a.part + ((int64_t)worker * a.jobs + a.slot[k]) * a.ldp + col(i);
#pragma unroll
            for (int e = 0; e < VE; e += 4)
                if (col(i) + e < N)
                    *(float4 *)(p + e) = make_float4(sum[k][i][e], sum[k][i][e + 1], sum[k][i][e + 2], sum[k][i][e + 3]);
        }
    }
}

int norm_bwd_threads(int64_t N) {
    return N <= 64 * 8 ? 64 : N <= 128 * 8 ? 128 : N <= 256 * 8 ? 256 : N <= 512 * 8 ? 512 : 1024;
}

template <int DT, int KEPT, int TPR, int COLS>
static hipError_t bwd(const NormBwd &a, hipStream_t s) {
    constexpr int NT = TPR < 256 ? 256 : TPR, R = NT / TPR;
    hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS>), dim3((unsigned)((a.workers + R - 1) / R)), dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <int DT, int KEPT>
static hipError_t bwd(const NormBwd &a, hipStream_t s) {
    if (a.N > 1024 * 16) return hipErrorInvalidValue;
    switch (norm_bwd_threads(a.N)) {
    case 64: return bwd<DT, KEPT, 64, 8>(a, s);
    case 128: return bwd<DT, KEPT, 128, 8>(a, s);
    case 256: return bwd<DT, KEPT, 256, 8>(a, s);
    case 512: return bwd<DT, KEPT, 512, 8>(a, s);
    default: return a.N <= 1024 * 8 ? bwd<DT, KEPT, 1024, 8>(a, s) : bwd<DT, KEPT, 1024, 16>(a, s);
    }
}

template <int DT>
static hipError_t bwd(int kept, const NormBwd &a, hipStream_t s) {
    if (kept == MM_INT8) return bwd<DT, MM_INT8>(a, s);
    return kept == DT ? bwd<DT, DT>(a, s) : bwd<DT, MM_FLOAT>(a, s);
}

hipError_t launch_norm_bwd(int dtype, int kept, const NormBwd &a, hipStream_t s) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    return dtype == MM_FLOAT ? bwd<MM_FLOAT>(kept, a, s)
           : dtype == MM_FLOAT16 ? bwd<MM_FLOAT16>(kept, a, s) : bwd<MM_BFLOAT16>(kept, a, s);
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
