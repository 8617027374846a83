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

// The piece of row p (of N columns) at column c, as loaded and as used (see
// edge_load); NULL and past the end: zeros.  ONCE: see stream_piece.
template <int DT, bool ONCE = false>
__device__ __forceinline__ uint4 piece_load(const void *p, int64_t row, int N, int c) {
    using S = typename Elem<DT>::S;
    if (!p) return make_uint4(0, 0, 0, 0);
    return edge_load<S, ONCE>((GlobalPtr<S>)((const S *)p + row * N), N, c);
}
template <int DT>
__device__ __forceinline__ void piece_use(const uint4 &v, int N, int c, float *x) {
    piece_floats<DT>(edge_piece<typename Elem<DT>::S>(v, N, c), x);
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
    S *y = (S *)((char *)((S *)p + row * N) + (uint32_t)(c * (int)sizeof(S)));
    uint4 v;
    __builtin_memcpy(&v, o, 16);
    if (c + VE <= N) stream_store(y, v);
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
    for (int i = 0; i < VE; ++i) top = max(top, c + i < N ? ck_magnitude(x[i]) : 0u);
#pragma unroll
    for (int d = 1; d < kCkBlock / VE; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const uint32_t ex = ck_exponent(top);
    const float inv = ck_inverse(ex);
    uint32_t w[VE / 4];
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) w[i] = ck_word(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], inv);
    ck_store<VE>((int8_t *)q + row * N, N, c, w);
    if (c < N && c % kCkBlock == 0) ((uint8_t *)scale)[row * ((N + 31) / 32) + c / kCkBlock] = (uint8_t)ex;
}

// Keeps pieces as they lie in memory across a loop, and a thread's number: what
// is formed of them in it (elements as floats, twice the registers; offsets
// and tests of columns) is not formed before it and held.
template <int CH>
__device__ __forceinline__ void keep_packed(uint4 (&p)[CH]) {
#pragma unroll
    for (int i = 0; i < CH; ++i) asm("" : "+v"(p[i].x), "+v"(p[i].y), "+v"(p[i].z), "+v"(p[i].w));
}

__device__ __forceinline__ void keep_number(int &t) { asm("" : "+v"(t)); }

// ---- forward

constexpr int kFwdCols = 16;  // columns of a thread

// A workgroup takes every gridDim-th row (or four, a wave each) and asks for
// the next one before it works on the present one; 16-bit weights stay in
// registers as they lie in memory.  The row is the same for a whole wave and
// kept in scalar registers, its addresses with it.
template <int DT, int TPR, bool TRAIN>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, 4) void k_norm_fwd(typename std::conditional<TRAIN, NormFwdTrain, NormFwd>::type a) {
    constexpr int VE = Elem<DT>::kVE, CH = kFwdCols / VE, NT = TPR < 256 ? 256 : TPR, SLOTS = NT / TPR;
    __shared__ float2 part[2][NT / 64];
    RowSums<NT, TPR> sums{part};
    int t = threadIdx.x % TPR;
    const int N = a.N;
    const int slot = TPR == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
    const int64_t step = (int64_t)gridDim.x * SLOTS;
    const float inv_n = 1.0f / (float)N;
    auto col = [&](int i) { return (i * TPR + t) * VE; };
    constexpr bool HOLD = VE == 8;  // FP32 weights would take too many registers: read again for each row
    uint4 xr[CH], br[CH], gr[CH], w1[CH], w2[CH];
    int64_t group = -1;
    auto load = [&](int64_t row, uint4 *x, uint4 *b) {
#pragma unroll
        for (int i = 0; i < CH; ++i) b[i] = piece_load<DT, true>(a.B, row, N, col(i));
#pragma unroll
        for (int i = 0; i < CH; ++i) x[i] = piece_load<DT, true>(a.X, row, N, col(i));
    };
    // Rows of a workgroup run together: all of them pass the barriers.
    int64_t first = (int64_t)blockIdx.x * SLOTS;
    auto row_at = [&](int64_t f) { return f + slot < a.M ? f + slot : (int64_t)a.M - 1; };
    load(row_at(first), xr, br);
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            w1[i] = piece_load<DT>(a.w1, 0, N, col(i));
            w2[i] = piece_load<DT>(a.w2, 0, N, col(i));
        }
    }
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
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = col(i) + e < N ? v[i][e] - mean : 0.0f;
                    s = fmaf(d, d, s);
                }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) s = fmaf(v[i][e], v[i][e], s);
        }
        return make_float2(mean, 1.0f / sqrtf(sums(s, 0.0f).x * inv_n + eps));
    };
    // v = (v - mean) r w + b.
    auto normalise = [&](float (*v)[VE], const float2 &m, const void *w, const uint4 *held, const void *b) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float y[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = (v[i][e] - m.x) * m.y;
            if (w) {
                piece_use<DT>(HOLD ? held[i] : piece_load<DT>(w, 0, N, col(i)), N, col(i), y);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] *= y[e];
            }
            if (b) {
                piece_use<DT>(piece_load<DT>(b, 0, N, col(i)), N, col(i), y);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] += y[e];
            }
        }
    };
    for (; first < a.M; first += step) {
        const bool live = first + slot < a.M;
        const int64_t row = row_at(first);
        keep_number(t);
        if constexpr (HOLD) {
            keep_packed(w1);
            keep_packed(w2);
        }
        if (a.gate) keep_packed(gr);
        uint4 xn[CH], bn[CH];
        if (first + step < a.M) load(row_at(first + step), xn, bn);
        float2 m1 = make_float2(0.0f, 1.0f), m2 = m1;
        float v[CH][VE];
        if (a.B) {
            const int64_t g = a.gate ? row / a.gate_rows : 0;
            if (g != group) {
                group = g;
#pragma unroll
                for (int i = 0; i < CH; ++i) gr[i] = piece_load<DT>(a.gate, g, N, col(i));
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_use<DT>(br[i], N, col(i), v[i]);
            if constexpr (TRAIN) {
                if (a.bq && live) {
#pragma unroll
                    for (int i = 0; i < CH; ++i) piece_checkpoint<DT>(a.bq, a.bs, row, N, col(i), v[i]);
                }
            }
            if (a.post != MM_NORM_NONE) {
                m1 = moments(a.post, a.eps1, v);
                normalise(v, m1, a.w1, w1, a.b1);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float w[VE], x[VE];
                piece_use<DT>(xr[i], N, col(i), x);
                if (a.gate) {
                    piece_use<DT>(gr[i], N, col(i), w);
#pragma unroll
                    for (int e = 0; e < VE; ++e) v[i][e] *= w[e];
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] = col(i) + e < N ? fmaf(a.alpha, v[i][e], x[e]) : 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_use<DT>(xr[i], N, col(i), v[i]);
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                if constexpr (TRAIN) {
                    float r[VE];
                    piece_store<DT>(a.R, row, N, col(i), v[i], r);
                    if (a.r32) {
#pragma unroll
                        for (int k = 0; k < VE / 4; ++k)
                            piece_store<MM_FLOAT>(a.r32, row, N, col(i) + 4 * k, v[i] + 4 * k, nullptr);
                    }
                    if (a.rq) piece_checkpoint<DT>(a.rq, a.rs, row, N, col(i), r);
                } else if (a.R) {
                    piece_store<DT>(a.R, row, N, col(i), v[i], nullptr);
                }
            }
        }
        if (a.pre != MM_NORM_NONE) {
            m2 = moments(a.pre, a.eps2, v);
            normalise(v, m2, a.w2, w2, a.b2);
            if (live) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if constexpr (TRAIN) {
                        float r[VE];
                        piece_store<DT>(a.Y, row, N, col(i), v[i], r);
                        if (a.yq) piece_checkpoint<DT>(a.yq, a.ys, row, N, col(i), r);
                    } else {
                        piece_store<DT>(a.Y, row, N, col(i), v[i], nullptr);
                    }
                }
            }
        }
        if constexpr (TRAIN) {
            if (a.stats && live && t == 0) *(float4 *)(a.stats + row * 4) = make_float4(m1.x, m1.y, m2.x, m2.y);
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            xr[i] = xn[i];
            br[i] = bn[i];
        }
    }
}

template <int DT, int TPR>
static hipError_t fwd(bool train, const NormFwdTrain &a, hipStream_t s) {
    constexpr int NT = TPR < 256 ? 256 : TPR, SLOTS = NT / TPR;
    // As many workgroups as the GPU holds at once.
    const int64_t n = ((int64_t)a.M + SLOTS - 1) / SLOTS, most = (int64_t)kNumCUs * (1024 / NT);
    const dim3 g((unsigned)(n < most ? n : most)), b(NT);
    if (train) hipLaunchKernelGGL((k_norm_fwd<DT, TPR, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_norm_fwd<DT, TPR, false>), g, b, 0, s, (const NormFwd &)a);
    return hipGetLastError();
}

template <int DT>
static hipError_t fwd(bool train, const NormFwdTrain &a, hipStream_t s) {
    if (a.N > 1024 * kFwdCols) return hipErrorInvalidValue;
    if (a.N <= 64 * kFwdCols) return fwd<DT, 64>(train, a, s);
    if (a.N <= 256 * kFwdCols) return fwd<DT, 256>(train, a, s);
    if (a.N <= 512 * kFwdCols) return fwd<DT, 512>(train, a, s);
    return fwd<DT, 1024>(train, a, s);
}

hipError_t launch_norm_fwd(int dtype, bool train, const NormFwdTrain &a, hipStream_t s) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    return dtype == MM_FLOAT ? fwd<MM_FLOAT>(train, a, s)
           : dtype == MM_FLOAT16 ? fwd<MM_FLOAT16>(train, a, s) : fwd<MM_BFLOAT16>(train, a, s);
}

// ---- backward

// What a thread holds of one row as it lies in memory.
template <int DT, int KEPT, int CH>
struct NormRaw {
    static constexpr int VE = Elem<DT>::kVE;
    static constexpr bool KEPT8 = KEPT == MM_INT8;
    static constexpr int RP = KEPT8 ? 1 : VE / Elem<KEPT8 ? DT : KEPT>::kVE;  // pieces of R in place of one
    using Kept = typename std::conditional<KEPT8, uint32_t[VE / 4], uint4>::type;
    uint4 dy[CH], ds[CH];
    Kept r[CH * RP], b[CH];
    uint32_t rs[CH], bs[CH];  // checkpoints: the blocks' scale bytes
};

// VE bytes of a checkpoint row and their scale byte; NULL and past the end: zeros.
template <int VE>
__device__ __forceinline__ void kept_load(const void *p, const void *scale, int64_t row, int N, int c, uint32_t *w, uint32_t &ex) {
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) w[i] = 0;
    ex = 0;
    if (!p || c >= N) return;
    ck_load<VE>((const int8_t *)p + row * N, N, c, w);
    ex = ((const uint8_t *)scale)[row * ((N + 31) / 32) + c / kCkBlock];
}

// A row's threads hold their columns of it, and of all of a worker's rows the
// sums, in registers; between the two sums over the row only what memory gave and
// dR stay, the normalised values are formed again.  BIAS: the sums of the biases'
// gradients are wanted.  128 registers keep the GPU full (two workgroups of 512
// threads on a CU); in 16-bit types, up to 4096 columns, they also hold the next
// row, which is asked for before the present one is worked on, and the weights.
template <int DT, int KEPT, int TPR, int COLS, bool BIAS>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, 4) void k_norm_bwd(NormBwd a) {
    constexpr int VE = Elem<DT>::kVE, CH = COLS / VE, NT = TPR < 256 ? 256 : TPR, NS = BIAS ? 4 : 2;
    constexpr bool AHEAD = TPR <= 512 && VE == 8, HOLD = AHEAD && !BIAS;
    __shared__ float2 part[2][NT / 64];
    RowSums<NT, TPR> sums{part};
    int t = threadIdx.x % TPR;
    const int N = a.N;
    const int worker = (int)blockIdx.x * (NT / TPR) + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    const int64_t r0 = (int64_t)worker * a.per, r1 = r0 + a.per < a.M ? r0 + a.per : a.M;
    const float inv_n = 1.0f / (float)N;
    auto col = [&](int i) { return (i * TPR + t) * VE; };
    using Raw = NormRaw<DT, KEPT, CH>;
    constexpr bool KEPT8 = Raw::KEPT8;
    constexpr int RP = Raw::RP, RV = VE / RP;
    auto load = [&](int64_t row, Raw &x) {
        if (row >= r1) return;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            x.dy[i] = piece_load<DT, true>(a.dY, row, N, col(i));
            if constexpr (KEPT8) {
                kept_load<VE>(a.R, a.rs, row, N, col(i), x.r[i], x.rs[i]);
            } else {
#pragma unroll
                for (int k = 0; k < RP; ++k) x.r[i * RP + k] = piece_load<KEPT, true>(a.R, row, N, col(i) + k * RV);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            x.ds[i] = piece_load<DT, true>(a.dS, row, N, col(i));
            if constexpr (KEPT8) kept_load<VE>(a.B, a.bs, row, N, col(i), x.b[i], x.bs[i]);
            else x.b[i] = piece_load<DT, true>(a.B, row, N, col(i));
        }
    };
    // Weights as they lie in memory; absent ones count as 1.
    uint4 w1[CH], w2[CH], gate[CH];
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            w1[i] = piece_load<DT>(a.w1, 0, N, col(i));
            w2[i] = piece_load<DT>(a.w2, 0, N, col(i));
        }
    }
    auto weight = [&](const uint4 *held, const void *w, int i, float *y) {
        piece_use<DT>(HOLD ? held[i] : piece_load<DT>(w, 0, N, col(i)), N, col(i), y);
    };
    float sum[NS][CH][VE], gsum[CH][VE];  // dw1, dw2 (, db1, db2); dgate of the group
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
#pragma unroll
            for (int k = 0; k < NS; ++k) sum[k][i][e] = 0.0f;
            gsum[i][e] = 0.0f;
        }
    int64_t group = -1;
    const int64_t group0 = a.gate_rows ? r0 / a.gate_rows : 0;
    auto finish_group = [&]() {
        if (!a.dgate || group < 0) return;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (a.gpart) {
                float *p = a.gpart + ((int64_t)worker * 2 + (group == group0 ? 0 : 1)) * a.ldp;
#pragma unroll
                for (int e = 0; e < VE; e += 4)
                    if (col(i) + e < N)  // ldp is a multiple of four
                        *(float4 *)(p + col(i) + e) = make_float4(gsum[i][e], gsum[i][e + 1], gsum[i][e + 2], gsum[i][e + 3]);
            } else {
                piece_store<DT>(a.dgate, group, N, col(i), gsum[i], nullptr);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) gsum[i][e] = 0.0f;
        }
    };
    Raw cur, nxt;
    if (AHEAD) load(r0, cur);
    const bool to_block = a.dB || a.dgate || a.slot[0] >= 0 || a.slot[2] >= 0;
    for (int it = 0; it < a.per; ++it) {
        const int64_t row = r0 + it;
        const bool live = row < r1;  // every thread reaches the barriers
        keep_number(t);
        if constexpr (HOLD) {
            keep_packed(w1);
            keep_packed(w2);
            keep_packed(gate);
        }
        if (AHEAD) load(row + 1, nxt);
        else load(row, cur);
        float m1 = 0.0f, rr1 = 1.0f, m2 = 0.0f, rr2 = 1.0f;
        if (live) {
            const float *st = a.stats + row * 4;
            if (a.post != MM_NORM_NONE) {
                m1 = st[0];
                rr1 = st[1];
            }
            m2 = st[2];
            rr2 = st[3];
        }
        if (live && a.gate_rows && row / a.gate_rows != group) {
            finish_group();
            group = row / a.gate_rows;
            if constexpr (HOLD) {
#pragma unroll
                for (int i = 0; i < CH; ++i) gate[i] = piece_load<DT>(a.gate, group, N, col(i));
            }
        }
        // x2 and d2 of a piece.
        auto second = [&](int i, float *x, float *y, float *d) {
            if constexpr (KEPT8) {
                const float sc = ck_scale(cur.rs[i]);
#pragma unroll
                for (int k = 0; k < VE / 4; ++k) unpack_bytes(cur.r[i][k], sc, x + 4 * k);
            } else {
#pragma unroll
                for (int k = 0; k < RP; ++k) piece_use<KEPT>(cur.r[i * RP + k], N, col(i) + k * RV, x + k * RV);
            }
            piece_use<DT>(cur.dy[i], N, col(i), y);
            float w[VE];
            if (a.w2) weight(w2, a.w2, i, w);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                x[e] = (x[e] - m2) * rr2;
                d[e] = a.w2 ? y[e] * w[e] : y[e];
            }
        };
        // x1 (or B) of a piece.
        auto first = [&](int i, float *x) {
            if constexpr (KEPT8) {
                const float sc = ck_scale(cur.bs[i]);
#pragma unroll
                for (int k = 0; k < VE / 4; ++k) unpack_bytes(cur.b[i][k], sc, x + 4 * k);
            } else {
                piece_use<DT>(cur.b[i], N, col(i), x);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) x[e] = (x[e] - m1) * rr1;
        };
        float d[CH][VE];
        // dR, from dY through the second norm and from dS.
        if (a.pre != MM_NORM_NONE) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float x[VE], y[VE], d2[VE];
                second(i, x, y, d2);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (live) {
                        sum[1][i][e] = fmaf(y[e], x[e], sum[1][i][e]);
                        if constexpr (BIAS) sum[3][i][e] += y[e];
                    }
                    s0 += d2[e];
                    s1 = fmaf(d2[e], x[e], s1);
                }
            }
            const float2 s = sums(s0, s1);
            const float mean = a.pre == MM_NORM_LAYER ? s.x * inv_n : 0.0f, proj = s.y * inv_n;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float x[VE], y[VE], d2[VE];
                second(i, x, y, d2);
                piece_use<DT>(cur.ds[i], N, col(i), y);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    d[i][e] = col(i) + e < N ? fmaf(rr2, d2[e] - mean - x[e] * proj, y[e]) : 0.0f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_use<DT>(cur.ds[i], N, col(i), d[i]);
        }
        if (live && a.dX) {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_store<DT>(a.dX, row, N, col(i), d[i], nullptr);
        }
        if (to_block) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                // y: n1; d becomes dn1, then d1
                float x[VE], w[VE], y[VE];
                first(i, x);
                if (a.w1) weight(w1, a.w1, i, w);
                if (a.dgate && live) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) y[e] = a.w1 ? x[e] * w[e] : x[e];
                    if (a.b1) {
                        float b[VE];
                        piece_use<DT>(piece_load<DT>(a.b1, 0, N, col(i)), N, col(i), b);
#pragma unroll
                        for (int e = 0; e < VE; ++e) y[e] += b[e];
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e) gsum[i][e] = fmaf(a.alpha * d[i][e], y[e], gsum[i][e]);
                }
                if (a.gate_rows) {
                    piece_use<DT>(HOLD ? gate[i] : piece_load<DT>(a.gate, live ? group : 0, N, col(i)), N, col(i), y);
#pragma unroll
                    for (int e = 0; e < VE; ++e) d[i][e] *= a.alpha * y[e];
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) d[i][e] *= a.alpha;
                }
                if (a.post != MM_NORM_NONE) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        if (live) {
                            sum[0][i][e] = fmaf(d[i][e], x[e], sum[0][i][e]);
                            if constexpr (BIAS) sum[2][i][e] += d[i][e];
                        }
                        if (a.w1) d[i][e] *= w[e];
                        s0 += d[i][e];
                        s1 = fmaf(d[i][e], x[e], s1);
                    }
                }
            }
            if (a.dB) {
                float mean = 0.0f, proj = 0.0f;
                if (a.post != MM_NORM_NONE) {
                    const float2 s = sums(s0, s1);
                    mean = a.post == MM_NORM_LAYER ? s.x * inv_n : 0.0f;
                    proj = s.y * inv_n;
                }
                if (live) {
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        if (a.post != MM_NORM_NONE) {
                            float x[VE];
                            first(i, x);
#pragma unroll
                            for (int e = 0; e < VE; ++e) d[i][e] = rr1 * (d[i][e] - mean - x[e] * proj);
                        }
                        piece_store<DT>(a.dB, row, N, col(i), d[i], nullptr);
                    }
                }
            }
        }
        if (AHEAD) cur = nxt;
    }
    finish_group();
    if (worker >= a.workers) return;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        if (a.slot[k] < 0) continue;
        float *p = a.part + ((int64_t)worker * a.jobs + a.slot[k]) * a.ldp;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int e = 0; e < VE; e += 4)
                if (col(i) + e < N)
                    *(float4 *)(p + col(i) + e) = make_float4(sum[k][i][e], sum[k][i][e + 1], sum[k][i][e + 2], sum[k][i][e + 3]);
    }
}

int norm_bwd_threads(int64_t N) {
    return N <= 64 * 8 ? 64 : N <= 128 * 8 ? 128 : N <= 256 * 8 ? 256 : N <= 512 * 8 ? 512 : 1024;
}

template <int DT, int KEPT, int TPR, int COLS>
static hipError_t bwd(const NormBwd &a, hipStream_t s) {
    constexpr int NT = TPR < 256 ? 256 : TPR, R = NT / TPR;
    const dim3 g((unsigned)((a.workers + R - 1) / R)), b(NT);
    if (a.slot[2] >= 0 || a.slot[3] >= 0) hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS, false>), g, b, 0, s, a);
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
