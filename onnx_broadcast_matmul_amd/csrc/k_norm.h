// k_norm.h -- norms before and after a block, fused with its gate and residual
// scale, and their backward pass, for one element type (instantiated by
// k_norm_f32.hip, k_norm_f16.hip and k_norm_bf16.hip):
//
//   n1 = norm1(B) w1 + b1 (or B)    R = X + alpha g n1    Y = norm2(R) w2 + b2
//
// The threads of a row hold it in registers from the first load to the last
// store, so every tensor is read or written once: memory bounds long runs of
// rows, the launch a few.  The variance of a layer norm is formed from the
// differences to the mean (a second sum over the registers), and the mean
// corrected by their sum, so that a large mean costs its own rounding alone.
#pragma once

#include <type_traits>

#include "checkpoint.h"
#include "device.h"
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

// Sums of two values (`both`, else of the second) over the TPR threads of a row.
// Above a wave they meet in LDS; `turn` alternates between two buffers, so that
// one barrier serves: a buffer is written again only after the next sum's barrier,
// which every reader has passed.
template <int NT, int TPR>
struct RowSums {
    static constexpr int W = TPR / 64;
    float2 (*part)[NT / 64];
    int turn = 0;
    __device__ __forceinline__ float2 operator()(bool both, float a, float b) {
        float2 s = make_float2(both ? wave_sum(a) : 0.0f, wave_sum(b));
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

template <int DT>
__device__ __forceinline__ uint4 piece_ones() {
    constexpr uint32_t one = DT == MM_FLOAT ? 0x3f800000u : DT == MM_FLOAT16 ? 0x3c003c00u : 0x3f803f80u;
    return make_uint4(one, one, one, one);
}

// The piece of row p (of N columns) at column c, as loaded (see edge_load); NULL and past the end: zeros.  ONCE: see stream_piece.  !EDGE: rows
// are whole pieces and c is inside.
template <int DT, bool ONCE = false, bool EDGE = true>
__device__ __forceinline__ uint4 piece_load(const void *p, int64_t row, int N, int c) {
    using S = typename Elem<DT>::S;
    if constexpr (!EDGE) {
        const GlobalPtr<S> at = (GlobalPtr<S>)((const __attribute__((address_space(1))) char *)((const S *)p + row * N) +
                                               (uint32_t)(c * (int)sizeof(S)));
        return ONCE ? stream_piece<S>(at) : whole_piece<S>(at);
    }
    if (!p) return make_uint4(0, 0, 0, 0);
    return edge_load<S, ONCE, uint32_t>((GlobalPtr<S>)((const S *)p + row * N), N, c);  // (of at most MM_NORM_MAX_COLS)
}
// x rounded to the type.
template <int DT>
__device__ __forceinline__ uint4 piece_pack(const float *x) {
    using E = Elem<DT>;
    typename E::S o[E::kVE];
#pragma unroll
    for (int i = 0; i < E::kVE; ++i) o[i] = E::from_f32(x[i]);
    uint4 v;
    __builtin_memcpy(&v, o, 16);
    return v;
}

// A piece to row p at column c, as far as the row goes.
template <int DT, bool EDGE = true>
__device__ __forceinline__ void piece_store(void *p, int64_t row, int N, int c, const uint4 &v) {
    using S = typename Elem<DT>::S;
    constexpr int VE = Elem<DT>::kVE;
    S *y = (S *)((char *)((S *)p + row * N) + (uint32_t)(c * (int)sizeof(S)));
    if constexpr (!EDGE) {
        if (c < N) stream_store(y, v);
        return;
    }
    if (c + VE <= N) {
        stream_store(y, v);
        return;
    }
    S o[VE];
    __builtin_memcpy(o, &v, 16);
#pragma unroll
    for (int i = 0; i < VE; ++i)
        if (c + i < N) y[i] = o[i];
}

// The checkpoint of a piece (zeros past the end); 32 / VE neighbouring lanes
// hold a block.
template <int DT, bool EDGE>
__device__ __forceinline__ void piece_checkpoint(void *q, void *scale, int64_t row, int N, int c, const uint4 &v) {
    constexpr int VE = Elem<DT>::kVE;
    const uint32_t ex = ck_exponent(block_top<VE>(piece_top<DT>(v)));
    const float inv = ck_inverse(ex);
    float x[VE];
    piece_floats<DT>(v, x);
    uint32_t w[VE / 4];
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) w[i] = ck_word(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], inv);
    if (c >= N) return;
    ck_store<VE>((int8_t *)q + row * N, EDGE ? N : c + VE, c, w);
    if (c % kCkBlock == 0) ((uint8_t *)scale + row * ((N + 31) / 32))[(uint32_t)(c / kCkBlock)] = (uint8_t)ex;
}

// Keeps pieces as they lie in memory across a loop, and a thread's number: what
// is formed of them in it (elements as floats, twice the registers; offsets
// and tests of columns) is not formed before it and held.
template <int CH>
__device__ __forceinline__ void keep_packed(uint4 (&p)[CH]) {
#pragma unroll
    for (int i = 0; i < CH; ++i) asm("" : "+v"(p[i].x), "+v"(p[i].y), "+v"(p[i].z), "+v"(p[i].w));
}

// The same for one piece until `late` is known: FP16 ones otherwise are taken apart
// before the sums over the row, for which there are no registers (8192 x 4096, RMS
// norms on both sides: 67 us with what went to scratch, 52 so).
__device__ __forceinline__ uint4 packed_until(uint4 p, float late) {
    asm("" : "+v"(p.x), "+v"(p.y), "+v"(p.z), "+v"(p.w) : "v"(late));
    return p;
}

__device__ __forceinline__ void keep_number(int &t) { asm("" : "+v"(t)); }

// ---- forward

constexpr int kFwdCols = 16;  // columns of a thread

// A workgroup takes every gridDim-th row (or four of a wave, two of two); in
// 16-bit types it asks for the next one before it works on the present one and
// keeps weights and biases in registers as they lie in memory.  The row is the same for a whole
// wave and kept in scalar registers, its addresses with it.  ALL: layer norms,
// biases and rows that are no whole number of pieces (see k_norm_bwd).
template <int DT, int TPR, bool TRAIN, bool ALL>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, 4) void k_norm_fwd(typename std::conditional<TRAIN, NormFwdTrain, NormFwd>::type a) {
    constexpr int VE = Elem<DT>::kVE, CH = kFwdCols / VE, NT = TPR < 256 ? 256 : TPR, SLOTS = NT / TPR;
    constexpr bool HOLD = VE == 8;
    __shared__ float2 part[2][NT / 64];
    RowSums<NT, TPR> sums{part};
    int t = threadIdx.x % TPR;
    const int N = a.N;
    const int slot = TPR < 256 ? __builtin_amdgcn_readfirstlane(threadIdx.x / TPR) : 0;
    const int step = (int)gridDim.x * SLOTS;
    const bool edge = N % VE != 0, ragged = N < TPR * kFwdCols;
    const float inv_n = 1.0f / (float)N;
    auto col = [&](int i) { return (i * TPR + t) * VE; };
    auto load = [&](int row, uint4 *x, uint4 *b) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (col(i) >= N) continue;  // absent pieces keep the zeros that they begin with
            if (a.B) b[i] = piece_load<DT, true, ALL>(a.B, row, N, col(i));
            x[i] = piece_load<DT, true, ALL>(a.X, row, N, col(i));
        }
    };
    auto settle = [&](uint4 *x) {
        if (!ALL || !edge) return;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (col(i) < N) x[i] = edge_piece<typename Elem<DT>::S>(x[i], N, col(i));
    };
    // A weight's piece, `none` where the plan has no such weight.
    auto weight_or = [&](const uint4 &none, const void *w, int64_t row, int i) {
        if (!w) return none;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (col(i) < N) {
            v = piece_load<DT, false, ALL>(w, row, N, col(i));
            if constexpr (ALL) v = edge_piece<typename Elem<DT>::S>(v, N, col(i));
        }
        return v;
    };
    // Rows of a workgroup run together: all of them pass the barriers.
    int first = (int)blockIdx.x * SLOTS;
    auto row_at = [&](int f) { return f < a.M - slot ? f + slot : a.M - 1; };
    uint4 xr[CH] = {}, br[CH] = {}, xn[CH] = {}, bn[CH] = {}, gr[CH], w1[CH], w2[CH], b1[CH], b2[CH];
    int change = 0;  // the row at which the next group of gate rows begins
    auto gate_group = [&](int row) {
        const int group = (int)((uint32_t)row / (uint32_t)a.gate_rows);
        const int64_t next = (int64_t)(group + 1) * a.gate_rows;
        change = next < a.M ? (int)next : a.M;
        return group;
    };
    if constexpr (HOLD) {
        // Everything that the first row needs is asked for at once.
        load(row_at(first), xn, bn);
        const int group = a.gate ? gate_group(row_at(first)) : 0;
        auto ask = [&](const void *w, int row, int i) {
            return w && col(i) < N ? piece_load<DT, false, ALL>(w, row, N, col(i)) : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            gr[i] = ask(a.gate, group, i);
            w1[i] = ask(a.w1, 0, i);
            w2[i] = ask(a.w2, 0, i);
            if constexpr (ALL) {
                b1[i] = ask(a.b1, 0, i);
                b2[i] = ask(a.b2, 0, i);
            }
        }
        if constexpr (ALL) {
            if (edge) {
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (col(i) < N)
                        for (uint4 *v : {&gr[i], &w1[i], &w2[i], &b1[i], &b2[i]})
                            *v = edge_piece<typename Elem<DT>::S>(*v, N, col(i));
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (!a.gate) gr[i] = piece_ones<DT>();
            if (!a.w1) w1[i] = piece_ones<DT>();
            if (!a.w2) w2[i] = piece_ones<DT>();
        }
    }
    // Mean and reciprocal deviation of v.  A layer norm's first mean is off by its
    // sum's roundings, some units in the last place.  The differences to it, small
    // where a mean is large, are summed too and correct both, so that the mean is
    // off by its last rounding alone and a constant row is nothing but its mean.
    auto moments = [&](int kind, float eps, const float (*v)[VE]) {
        float mean = 0.0f, s = 0.0f, var;
        if (ALL && kind == MM_NORM_LAYER) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) s += v[i][e];
            mean = sums(false, 0.0f, s).y * inv_n;
            asm("" : "+v"(mean));  // rounded here, not within the differences' fma
            float rest = 0.0f;
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = col(i) + e < N ? v[i][e] - mean : 0.0f;
                    rest += d;
                    s = fmaf(d, d, s);
                }
            const float2 both = sums(true, rest, s);
            const float more = both.x * inv_n;
            mean += more;
            var = fmaf(-more, more, both.y * inv_n);
            var = var < 0.0f ? 0.0f : var;  // (NaN stays)
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int e = 0; e < VE; ++e) s = fmaf(v[i][e], v[i][e], s);
            var = sums(false, 0.0f, s).y * inv_n;
        }
        return make_float2(mean, 1.0f / sqrtf(var + eps));
    };
    // v = (v - mean) r w + b.
    auto normalise = [&](float (*v)[VE], int kind, const float2 &m, const void *w, const uint4 *held, const void *b,
                         const uint4 *held_b) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            float y[VE];
            if (ALL && kind == MM_NORM_LAYER) {
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] -= m.x;
            }
            if constexpr (HOLD) piece_floats<DT>(packed_until(held[i], m.y), y);
            else piece_floats<DT>(weight_or(piece_ones<DT>(), w, 0, i), y);
#pragma unroll
            for (int e = 0; e < VE; ++e) v[i][e] = v[i][e] * m.y * y[e];
            if (ALL && b) {
                if constexpr (HOLD) piece_floats<DT>(packed_until(held_b[i], m.y), y);
                else piece_floats<DT>(weight_or(make_uint4(0, 0, 0, 0), b, 0, i), y);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] += y[e];
            }
        }
    };
    // Zeros in a row's absent columns, which a mean or a bias has reached.
    auto cut = [&](float (*v)[VE]) {
        if (!ALL || !ragged) return;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (col(i) + e >= N) v[i][e] = 0.0f;
    };
    for (;;) {
        keep_number(t);
        if constexpr (HOLD) {
            keep_packed(w1);
            keep_packed(w2);
            keep_packed(gr);
            if constexpr (ALL) {
                keep_packed(b1);
                keep_packed(b2);
            }
        }
        const bool live = first < a.M - slot;
        const int row = row_at(first);
        if constexpr (HOLD) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                xr[i] = xn[i];
                br[i] = bn[i];
            }
            if (first < a.M - step) load(row_at(first + step), xn, bn);
        } else {
            load(row, xr, br);
        }
        settle(xr);
        float2 m1 = make_float2(0.0f, 1.0f), m2 = m1;
        float v[CH][VE];
        if (a.B) {
            settle(br);
            int group = 0;
            if constexpr (HOLD) {
                if (a.gate && row >= change) {
                    group = gate_group(row);
#pragma unroll
                    for (int i = 0; i < CH; ++i) gr[i] = weight_or(piece_ones<DT>(), a.gate, group, i);
                }
            } else if (a.gate) {
                group = (int)((uint32_t)row / (uint32_t)a.gate_rows);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_floats<DT>(br[i], v[i]);
            if constexpr (TRAIN) {
                if (a.bq && live) {
#pragma unroll
                    for (int i = 0; i < CH; ++i) piece_checkpoint<DT, ALL>(a.bq, a.bs, row, N, col(i), br[i]);
                }
            }
            if (a.post != MM_NORM_NONE) {
                m1 = moments(a.post, a.eps1, v);
                normalise(v, a.post, m1, a.w1, w1, a.b1, b1);
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float w[VE], x[VE];
                piece_floats<DT>(HOLD ? packed_until(xr[i], m1.y) : xr[i], x);
                if constexpr (HOLD) piece_floats<DT>(packed_until(gr[i], m1.y), w);
                else piece_floats<DT>(weight_or(piece_ones<DT>(), a.gate, group, i), w);
#pragma unroll
                for (int e = 0; e < VE; ++e) v[i][e] = fmaf(a.alpha * w[e], v[i][e], x[e]);
            }
            cut(v);
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_floats<DT>(xr[i], v[i]);
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const uint4 r = piece_pack<DT>(v[i]);
                if (a.R) piece_store<DT, ALL>(a.R, row, N, col(i), r);
                if constexpr (TRAIN) {
                    if (a.r32) {
#pragma unroll
                        for (int k = 0; k < VE / 4; ++k)
                            if (VE == 4 || col(i) + 4 * k < N)
                                piece_store<MM_FLOAT, ALL>(a.r32, row, N, col(i) + 4 * k, piece_pack<MM_FLOAT>(v[i] + 4 * k));
                    }
                    if (a.rq) piece_checkpoint<DT, ALL>(a.rq, a.rs, row, N, col(i), r);
                }
            }
        }
        if (a.pre != MM_NORM_NONE) {
            m2 = moments(a.pre, a.eps2, v);
            normalise(v, a.pre, m2, a.w2, w2, a.b2, b2);
            if (TRAIN) cut(v);
            if (live) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const uint4 y = piece_pack<DT>(v[i]);
                    piece_store<DT, ALL>(a.Y, row, N, col(i), y);
                    if constexpr (TRAIN) {
                        if (a.yq) piece_checkpoint<DT, ALL>(a.yq, a.ys, row, N, col(i), y);
                    }
                }
            }
        }
        if constexpr (TRAIN) {
            if (a.stats && live && t == 0) *(float4 *)(a.stats + (int64_t)row * 4) = make_float4(m1.x, m1.y, m2.x, m2.y);
        }
        if (first >= a.M - step) break;  // (first + step may pass 2^31)
        first += step;
    }
}

template <int DT, int TPR>
static hipError_t fwd(bool train, const NormFwdTrain &a, hipStream_t s) {
    constexpr int NT = TPR < 256 ? 256 : TPR, SLOTS = NT / TPR;
    // As many workgroups as the GPU holds at once.
    const int64_t n = ((int64_t)a.M + SLOTS - 1) / SLOTS, most = (int64_t)kNumCUs * (1024 / NT);
    const dim3 g((unsigned)(n < most ? n : most)), b(NT);
    const bool all = a.post == MM_NORM_LAYER || a.pre == MM_NORM_LAYER || a.b1 || a.b2 || a.N % Elem<DT>::kVE != 0;
    if (train && all) hipLaunchKernelGGL((k_norm_fwd<DT, TPR, true, true>), g, b, 0, s, a);
    else if (train) hipLaunchKernelGGL((k_norm_fwd<DT, TPR, true, false>), g, b, 0, s, a);
    else if (all) hipLaunchKernelGGL((k_norm_fwd<DT, TPR, false, true>), g, b, 0, s, (const NormFwd &)a);
    else hipLaunchKernelGGL((k_norm_fwd<DT, TPR, false, false>), g, b, 0, s, (const NormFwd &)a);
    return hipGetLastError();
}

template <int DT>
static hipError_t fwd(bool train, const NormFwdTrain &a, hipStream_t s) {
    if (a.N > 1024 * kFwdCols) return hipErrorInvalidValue;
    if (a.N <= 64 * kFwdCols) return fwd<DT, 64>(train, a, s);
    if (a.N <= 128 * kFwdCols) return fwd<DT, 128>(train, a, s);
    if (a.N <= 256 * kFwdCols) return fwd<DT, 256>(train, a, s);
    if (a.N <= 512 * kFwdCols) return fwd<DT, 512>(train, a, s);
    return fwd<DT, 1024>(train, a, s);
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
    float4 st;
};

// VE bytes of a checkpoint row and their scale byte.
template <int VE, bool EDGE>
__device__ __forceinline__ void kept_load(const void *p, const void *scale, int64_t row, int N, int c, uint32_t *w, uint32_t &ex) {
    ck_load<VE>((const int8_t *)p + row * N, EDGE ? N : c + VE, c, w);
    ex = ((const uint8_t *)scale + row * ((N + 31) / 32))[(uint32_t)(c / kCkBlock)];
}

// A row's threads hold their columns of it, and of all of a worker's rows the
// sums, in registers; between the two sums over the row only what memory gave and
// the gradient on its way stay, centred values are formed again.  128 registers
// keep the GPU full (two workgroups of 512 threads on a CU); in 16-bit types, up
// to 4096 columns and without ALL, they also hold the next row, which is asked for
// before the present one is worked on, and the weights.  They are too few for both
// norms with ALL (12 to 280 bytes a lane go to scratch, but for a wave a row from
// checkpoints and in FP16 and FP32) and for the 16 columns a lane of rows above 8192 (92
// to 684 in every form).
//
// What a plan has is told apart at compile time as far as the loop over a row's
// columns feels it: its arithmetic bounds the kernel, not memory alone (with
// every choice made at run time, 70 instructions a column, 94 us for 8192 x 4096
// from checkpoints).  ALL: layer norms, gradients of biases, a post bias where the
// gate's gradient is wanted, and rows that are no whole number of pieces; without them absent columns (zeros) stay zero by
// themselves.  Absent weights and gates are ones.
template <int DT, int KEPT, int TPR, int COLS, bool PRE, bool POST, bool ALL>
__global__ __launch_bounds__(norm_bwd_block(TPR), 4) void k_norm_bwd(NormBwd a) {
    constexpr int VE = Elem<DT>::kVE, CH = COLS / VE, NT = norm_bwd_block(TPR), NS = ALL ? 4 : 2;
    constexpr bool HOLD = TPR <= 512 && VE == 8 && !ALL;
    __shared__ float2 part[2][NT / 64];
    RowSums<NT, TPR> sums{part};
    int t = threadIdx.x % TPR;
    const int N = a.N;
    // A workgroup is one worker, or (a wave a row, no barrier) four.
    const int worker = TPR == 64 ? (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : (int)blockIdx.x;
    if (worker >= a.workers) return;
    const int r0 = worker * a.per, r1 = a.M - r0 < a.per ? a.M : r0 + a.per;
    const bool edge = N % VE != 0, ragged = N < TPR * COLS;
    const float inv_n = 1.0f / (float)N;
    auto col = [&](int i) { return (i * TPR + t) * VE; };
    using Raw = NormRaw<DT, KEPT, CH>;
    constexpr bool KEPT8 = Raw::KEPT8;
    constexpr int RP = Raw::RP, RV = VE / RP;
    constexpr int KE = KEPT8 ? DT : KEPT;  // (type of R's pieces)
    // Absent pieces are never loaded: they keep the zeros that they begin with.
    auto load = [&](int row, Raw &x) {
        x.st = *(const float4 *)(a.stats + (int64_t)row * 4);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (col(i) >= N) continue;
            if constexpr (PRE) {
                x.dy[i] = piece_load<DT, true, ALL>(a.dY, row, N, col(i));
                if constexpr (KEPT8) {
                    kept_load<VE, ALL>(a.R, a.rs, row, N, col(i), x.r[i], x.rs[i]);
                } else {
#pragma unroll
                    for (int k = 0; k < RP; ++k)
                        if (RP == 1 || col(i) + k * RV < N) x.r[i * RP + k] = piece_load<KE, true, ALL>(a.R, row, N, col(i) + k * RV);
                }
            }
            if (a.dS) x.ds[i] = piece_load<DT, true, ALL>(a.dS, row, N, col(i));
            if (a.B) {
                if constexpr (KEPT8) kept_load<VE, ALL>(a.B, a.bs, row, N, col(i), x.b[i], x.bs[i]);
                else x.b[i] = piece_load<DT, true, ALL>(a.B, row, N, col(i));
            }
        }
    };
    // The end of a row whose length is no whole number of pieces.
    auto settle = [&](Raw &x) {
        if (!ALL || !edge) return;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (col(i) >= N) continue;
            x.dy[i] = edge_piece<typename Elem<DT>::S>(x.dy[i], N, col(i));
            x.ds[i] = edge_piece<typename Elem<DT>::S>(x.ds[i], N, col(i));
            if constexpr (!KEPT8) {
                x.b[i] = edge_piece<typename Elem<DT>::S>(x.b[i], N, col(i));
#pragma unroll
                for (int k = 0; k < RP; ++k)
                    if (RP == 1 || col(i) + k * RV < N)
                        x.r[i * RP + k] = edge_piece<typename Elem<KE>::S>(x.r[i * RP + k], N, col(i) + k * RV);
            }
        }
    };
    // Weights as they lie in memory, ones where the plan has none.
    auto ones_or = [&](const void *w, int64_t row, int i) {
        uint4 v = piece_ones<DT>();
        if (w) {
            v = make_uint4(0, 0, 0, 0);
            if (col(i) < N) {
                v = piece_load<DT, false, ALL>(w, row, N, col(i));
                if constexpr (ALL) v = edge_piece<typename Elem<DT>::S>(v, N, col(i));
            }
        }
        return v;
    };
    uint4 w1[CH], w2[CH], gate[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        if constexpr (HOLD) {
            w1[i] = ones_or(a.w1, 0, i);
            w2[i] = ones_or(a.w2, 0, i);
        }
        gate[i] = piece_ones<DT>();
    }
    auto weight = [&](const uint4 *held, const void *w, int64_t row, int i, float *y) {
        if constexpr (HOLD) piece_floats<DT>(held[i], y);
        else piece_floats<DT>(ones_or(w, row, i), y);
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
    int group = -1;
    auto finish_group = [&]() {
        if (!a.dgate || group < 0) return;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (a.gpart) {
                float *p = a.gpart + ((int64_t)worker * 2 + (group == r0 / a.gate_rows ? 0 : 1)) * a.ldp;
#pragma unroll
                for (int e = 0; e < VE; e += 4)
                    if (col(i) + e < N)  // ldp is a multiple of four
                        *(float4 *)(p + col(i) + e) = make_float4(gsum[i][e], gsum[i][e + 1], gsum[i][e + 2], gsum[i][e + 3]);
            } else {
                piece_store<DT, ALL>(a.dgate, group, N, col(i), piece_pack<DT>(gsum[i]));
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) gsum[i][e] = 0.0f;
        }
    };
    Raw cur = {}, nxt = {};
    if constexpr (HOLD) load(r0, nxt);
    const bool to_block = a.dB || a.dgate || (POST && (a.slot[0] >= 0 || a.slot[2] >= 0));
    int change = r0;  // the row at which the next group begins
    for (int row = r0; row < r1; ++row) {
        keep_number(t);
        if constexpr (HOLD) {
            keep_packed(w1);
            keep_packed(w2);
            keep_packed(gate);
        }
        if constexpr (HOLD) {
            cur = nxt;
            if (row + 1 < r1) load(row + 1, nxt);
        } else {
            load(row, cur);
        }
        settle(cur);
        // (the same in every lane)
        auto scalar = [](float x) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x))); };
        const float m1 = POST ? scalar(cur.st.x) : 0.0f, rr1 = POST ? scalar(cur.st.y) : 1.0f;
        const float m2 = PRE ? scalar(cur.st.z) : 0.0f, rr2 = PRE ? scalar(cur.st.w) : 1.0f;
        if (a.gate_rows && row >= change) {
            finish_group();
            group = (int)((uint32_t)row / (uint32_t)a.gate_rows);
            const int64_t next = (int64_t)(group + 1) * a.gate_rows;
            change = next < a.M ? (int)next : a.M;
            if constexpr (HOLD) {
#pragma unroll
                for (int i = 0; i < CH; ++i) gate[i] = ones_or(a.gate, group, i);
            }
        }
        // R - mean, and B - mean (B without a norm), of a piece.
        auto second = [&](int i, float *x) {
            if constexpr (KEPT8) {
                const float sc = ck_scale(cur.rs[i]);
#pragma unroll
                for (int k = 0; k < VE / 4; ++k) unpack_bytes(cur.r[i][k], sc, m2, x + 4 * k);
            } else {
#pragma unroll
                for (int k = 0; k < RP; ++k) piece_floats<KE>(cur.r[i * RP + k], x + k * RV);
#pragma unroll
                for (int e = 0; e < VE; ++e) x[e] -= m2;
            }
        };
        auto first = [&](int i, float *x) {
            if constexpr (KEPT8) {
                const float sc = ck_scale(cur.bs[i]);
#pragma unroll
                for (int k = 0; k < VE / 4; ++k) unpack_bytes(cur.b[i][k], sc, m1, x + 4 * k);
            } else {
                piece_floats<DT>(cur.b[i], x);
                if constexpr (POST) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) x[e] -= m1;
                }
            }
        };
        // Normalised values are x r: r is taken out of the sums over the row and
        // into the factors that go with a whole row.
        float d[CH][VE];
        // dR, from dY through the second norm and from dS.
        if constexpr (PRE) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float x[VE], w[VE];
                second(i, x);
                weight(w2, a.w2, 0, i, w);
                piece_floats<DT>(cur.dy[i], d[i]);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if constexpr (ALL) sum[3][i][e] += d[i][e];
                    sum[1][i][e] = fmaf(d[i][e] * rr2, x[e], sum[1][i][e]);
                    d[i][e] *= w[e];
                    if constexpr (ALL) s0 += d[i][e];
                    s1 = fmaf(d[i][e], x[e], s1);
                }
            }
            const bool layer = ALL && a.pre == MM_NORM_LAYER;
            const float2 s = sums(layer, s0, s1);
            const float mean = s.x * inv_n, proj = s.y * inv_n * rr2 * rr2;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float x[VE], y[VE];
                second(i, x);
                piece_floats<DT>(cur.ds[i], y);
                if (layer) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) d[i][e] -= mean;
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) d[i][e] = fmaf(rr2, fmaf(-proj, x[e], d[i][e]), y[e]);
                if (ragged && (ALL || m2 != 0.0f)) {
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        if (col(i) + e >= N) d[i][e] = 0.0f;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_floats<DT>(cur.ds[i], d[i]);
        }
        if (a.dX) {
#pragma unroll
            for (int i = 0; i < CH; ++i) piece_store<DT, ALL>(a.dX, row, N, col(i), piece_pack<DT>(d[i]));
        }
        if (!to_block) continue;
        float s0 = 0.0f, s1 = 0.0f;
        const float ar = a.alpha * rr1;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            // d becomes dn1, then d1
            float x[VE], w[VE], y[VE];
            if (POST || a.dgate) first(i, x);
            if constexpr (POST) weight(w1, a.w1, 0, i, w);
            if (a.dgate) {
                if (ALL && a.b1) {  // n1 = x r w1 + b1
                    piece_floats<DT>(ones_or(a.b1, 0, i), y);
#pragma unroll
                    for (int e = 0; e < VE; ++e) gsum[i][e] = fmaf(a.alpha * d[i][e], fmaf(x[e] * rr1, POST ? w[e] : 1.0f, y[e]), gsum[i][e]);
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) gsum[i][e] = fmaf(ar * d[i][e], POST ? x[e] * w[e] : x[e], gsum[i][e]);
                }
            }
            weight(gate, a.gate, group < 0 ? 0 : group, i, y);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                d[i][e] *= a.alpha * y[e];
                if constexpr (POST) {
                    if constexpr (ALL) sum[2][i][e] += d[i][e];
                    sum[0][i][e] = fmaf(d[i][e] * rr1, x[e], sum[0][i][e]);
                    d[i][e] *= w[e];
                    if constexpr (ALL) s0 += d[i][e];
                    s1 = fmaf(d[i][e], x[e], s1);
                }
            }
        }
        if (!a.dB) continue;
        if constexpr (POST) {
            const bool layer = ALL && a.post == MM_NORM_LAYER;
            const float2 s = sums(layer, s0, s1);
            const float mean = s.x * inv_n, proj = s.y * inv_n * rr1 * rr1;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float x[VE];
                first(i, x);
                if (layer) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) d[i][e] -= mean;
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) d[i][e] = rr1 * fmaf(-proj, x[e], d[i][e]);
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) piece_store<DT, ALL>(a.dB, row, N, col(i), piece_pack<DT>(d[i]));
    }
    finish_group();
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

template <int DT, int KEPT, int TPR, int COLS>
static hipError_t bwd(const NormBwd &a, hipStream_t s) {
    constexpr int NT = norm_bwd_block(TPR), R = NT / TPR;
    const dim3 g((unsigned)((a.workers + R - 1) / R)), b(NT);
    const bool pre = a.pre != MM_NORM_NONE, post = a.post != MM_NORM_NONE;
    const bool all = a.pre == MM_NORM_LAYER || a.post == MM_NORM_LAYER || a.slot[2] >= 0 || a.slot[3] >= 0 || a.b1 ||
                     a.N % Elem<DT>::kVE != 0;
    if (!pre) hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS, false, true, true>), g, b, 0, s, a);
    else if (post && all) hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS, true, true, true>), g, b, 0, s, a);
    else if (post) hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS, true, true, false>), g, b, 0, s, a);
    else if (all) hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS, true, false, true>), g, b, 0, s, a);
    else hipLaunchKernelGGL((k_norm_bwd<DT, KEPT, TPR, COLS, true, false, false>), g, b, 0, s, a);
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

#define MM_NORM_INSTANCE(DT, NAME)                                                                              \
    hipError_t norm_fwd_##NAME(bool train, const NormFwdTrain &a, hipStream_t s) { return fwd<DT>(train, a, s); } \
    hipError_t norm_bwd_##NAME(int kept, const NormBwd &a, hipStream_t s) { return bwd<DT>(kept, a, s); }

}  // namespace mm
