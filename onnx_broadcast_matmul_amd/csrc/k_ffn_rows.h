// k_ffn_rows.h -- the gated block and the scaled INT8 product over few rows
// (one decoded token to kFfnRows of them).
//
// The weights are the traffic, and memory's rate the bound: each is read once
// (one token, [N, K]: gated BF16 4096 x 11008 35 us, 5.1 TB/s; INT8 11008 x 4096
// 12 us, of which 3 are the launch and the rest a workgroup's chain of K).  A workgroup owns NF x 16
// weight columns (the gated block: half gate, half up of the same features);
// its waves take every NWV-th block of K and their sums meet in LDS in wave
// order, so the result does not depend on timing.  X (a few rows) is re-read
// by every workgroup from cache.
//
// Weights stored [N, K] go straight from memory into MFMA operands: a lane
// holds 16 bytes of one weight row.  Weights stored [K, N] (KN) are loaded as
// 16-byte pieces of rows of one k, NF / panels x 16 columns wide, and turned
// through LDS that belongs to the wave alone (no barrier) by the transposing
// reads.  Either way the next block's loads are in flight while a block is
// multiplied.  Rows of any alignment are read in 16-byte pieces; only the end
// of K goes element by element.
//
// UA ([N, K] weights or X with rows off 4-byte alignment, an odd K): 16-byte
// loads off a dword boundary run at half the rate, so pieces are read from the
// dword they begin in, with the one behind, and shifted where they are used
// (M = 3, K = 2561, N = 5530: INT8 14.2 -> 7.8 us, BF16 gated 37.4 -> 26.6; at
// K = 2560 6.4 and 15.8).
//
// XQ (INT8 product): X comes in that float type, and every workgroup
// quantizes its rows into LDS by mm_quantize_rows' rule while its first
// weights are on their way.  Two reads of a few rows from cache cost less than
// a kernel of its own before this one.
#pragma once

#include <type_traits>

#include "activation.h"
#include "device.h"
#include "ffn.h"
#include "pieces.h"
#include "quantize.h"

namespace mm {

typedef int i32x4v __attribute__((ext_vector_type(4)));

template <int DT, int OD, bool GLU, bool KN, int NF, int MB, int NWV, int XQ, bool UA>
__global__ __launch_bounds__(64 * NWV, MB == 2 || (XQ && KN) ? 2 : XQ && NWV == 4 ? 3 : 4) void k_ffn_rows(FfnSlim a) {
#if defined(__HIP_DEVICE_COMPILE__)
    using E = Elem<DT>;
    using S = typename E::S;
    using OE = Elem<OD>;
    using OS = typename OE::S;
    constexpr bool INT = DT == MM_INT8;
    static_assert(XQ == 0 || INT, "only the INT8 product quantizes");
    constexpr int NT = 64 * NWV;
    constexpr int ES = (int)sizeof(S);
    constexpr int VE = 16 / ES;
    constexpr int NPAN = GLU ? 2 : 1;
    constexpr int CF = NF / NPAN;          // fragments (of 16 columns) of one panel
    constexpr int COLS = 16 * CF;          // output columns of the workgroup
    constexpr int U = KN || (UA && GLU) ? 2 : 4;  // MFMA steps of a block
    constexpr int SK = 4 * VE;             // k of one step: 16 bytes in each of 4 lane groups
    constexpr int BK = U * SK;             // k of a block
    using AccT = typename std::conditional<INT, i32x4v, f32x4>::type;
    using gptr = GlobalPtr<S>;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t M = a.M, N = a.N, K = a.K;
    // Neighbouring columns on one XCD, except for wide gated blocks with [N, K]
    // weights, whose two streams do better spread over the XCDs (M = 1, K =
    // 4096, N = 11008: 41.4 us so, 38.9 spread; M = 13, K = 2048, N = 5461:
    // 13.2 and 14.9; INT8, K = N = 4096: 6.6 and 7.6).
    const int64_t n0 = (GLU && !KN && NWV == 4 ? (int64_t)blockIdx.x : xcd_remap(blockIdx.x, gridDim.x)) * COLS;

    // ---- weights
    // [N, K]: fragment f of a lane is row n0 + 16 (f % CF) + r of its panel;
    // rows past the end read the last one and are not stored.
    // [K, N]: a block is BK rows of COLS columns of each panel, CPR pieces a row.
    constexpr int CPR = COLS / VE;
    constexpr int PIECES = KN ? BK * CPR * NPAN / 64 : NF * U;  // 16-byte pieces per lane and block
    static_assert(!KN || (BK * CPR) % 64 == 0, "whole pieces per lane");
    static_assert(!UA || (!KN && ES < 4), "only [N, K] rows of narrow types are shifted");
    gptr w[KN ? NPAN : NF];
    int wsh[UA ? NF : 1];  // UA: bytes from the dword that w points to to the piece
    if constexpr (KN) {
#pragma unroll
        for (int p = 0; p < NPAN; ++p) w[p] = (gptr)a.B[p] + n0;
    } else {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const int64_t n = n0 + 16 * (f % CF) + r;
            w[f] = (gptr)a.B[f / CF] + (n < N ? n : N - 1) * a.ldb + g * VE;
            if constexpr (UA) {
                wsh[f] = (int)((uintptr_t)w[f] & 3);
                w[f] -= wsh[f] / ES;
            }
        }
    }
    const bool back = (KN ? N : K) >= VE;  // weight rows are at least a piece long
    const int64_t left_n = N - n0;
    // The dword behind a shifted piece's 16 bytes, or (nothing to shift) its
    // own last one: never beyond the dwords that hold the piece.
    auto next_dword = [&](gptr p, int sh) {
        return *(const __attribute__((address_space(1))) uint32_t *)((const __attribute__((address_space(1))) char *)p +
                                                                    (sh ? 16 : 12));
    };
    auto shifted = [&](const uint4 &v, uint32_t e, int sh) {
        return make_uint4(__builtin_amdgcn_alignbyte(v.y, v.x, sh), __builtin_amdgcn_alignbyte(v.z, v.y, sh),
                          __builtin_amdgcn_alignbyte(v.w, v.z, sh), __builtin_amdgcn_alignbyte(e, v.w, sh));
    };
    auto load_w = [&](int64_t kb, uint4 *t, uint32_t *te) {
        const int64_t k0 = kb * BK, krem = K - k0;
        if constexpr (KN) {
            constexpr int PP = PIECES / NPAN;
            // Pieces that cross a row's end read on into the next rows, where
            // the matrix goes on for that long (see k_ffn.h).
            const bool whole = krem >= BK && (left_n >= COLS || (krem - BK) * a.ldb >= VE);
            if (whole) {
#pragma unroll
                for (int p = 0; p < NPAN; ++p)
#pragma unroll
                    for (int i = 0; i < PP; ++i) {
                        const int y = lane + 64 * i, row = y / CPR, c = y % CPR;
                        t[p * PP + i] = whole_piece<S>(w[p] + (k0 + row) * a.ldb + (c * VE < left_n ? c * VE : 0));
                    }
            } else {
#pragma unroll
                for (int p = 0; p < NPAN; ++p)
#pragma unroll
                    for (int i = 0; i < PP; ++i) {
                        const int y = lane + 64 * i, row = y / CPR, c = y % CPR;
                        t[p * PP + i] = row_piece<S>(w[p] + (k0 + row) * a.ldb + c * VE, row < krem ? left_n - c * VE : 0, back);
                    }
            }
        } else if (krem >= BK) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    t[u * NF + f] = whole_piece<S>(w[f] + k0 + u * SK);
                    if constexpr (UA) te[u * NF + f] = next_dword(w[f] + k0 + u * SK, wsh[f]);
                }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    t[u * NF + f] = row_piece<S>(w[f] + (UA ? wsh[f] / ES : 0) + k0 + u * SK, krem - (u * 4 + g) * VE, back);
        }
    };

    constexpr int WLDS = KN ? BK * COLS * ES * NPAN : 0;  // bytes of one wave's block
    constexpr int RLDS = NWV * NF * MB * 1024;            // the waves' sums, after the last block
    __shared__ __attribute__((aligned(1024))) char pool[NWV * WLDS > RLDS ? NWV * WLDS : RLDS];
    char *mine = pool + wave * WLDS;
    // Piece c of row k at c ^ (k / (256 / row bytes)): the rows that one
    // transposing read takes then fall on distinct banks.
    constexpr int RB = COLS * ES;          // bytes of a row
    auto turn = [&](int k, int c) { return CPR >= 4 ? c ^ ((k / (256 / RB)) & (CPR - 1)) : c; };
    auto stage_w = [&](const uint4 *t) {
        if constexpr (KN) {
            constexpr int PP = PIECES / NPAN;
#pragma unroll
            for (int p = 0; p < NPAN; ++p)
#pragma unroll
                for (int i = 0; i < PP; ++i) {
                    const int y = lane + 64 * i, row = y / CPR, c = y % CPR;
                    *(uint4 *)(mine + p * BK * RB + row * RB + turn(row, c) * 16) = t[p * PP + i];
                }
        }
    };
    // Fragment f of step u: 16 bytes of consecutive k of column 16 (f % CF) + r.
    auto frag_w = [&](const uint4 *t, const uint32_t *te, bool whole, int u, int f) -> uint4 {
        if constexpr (UA) {
            return shifted(t[u * NF + f], te[u * NF + f], whole ? wsh[f] : 0);
        } else if constexpr (!KN) {
            return t[u * NF + f];
        } else {
            const char *P = mine + (f / CF) * BK * RB;
            const int jl = lane & 15, n = 16 * (f % CF);
            if constexpr (ES == 1) {
                typedef int i32x2v __attribute__((ext_vector_type(2)));
                uint2 h2[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = u * SK + g * 16 + h * 8 + (jl >> 1);
                    const char *at = P + k * RB + turn(k, n >> 4) * 16 + (jl & 1) * 8;
                    h2[h] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                                          (__attribute__((address_space(3))) i32x2v *)(at)));
                }
                return make_uint4(h2[0].x, h2[0].y, h2[1].x, h2[1].y);
            } else if constexpr (ES == 2) {
                uint2 h2[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = u * SK + g * 8 + h * 4 + (jl >> 2), c = n + (jl & 3) * 4;
                    const char *at = P + k * RB + turn(k, c >> 3) * 16 + ((c >> 2) & 1) * 8;
                    h2[h] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                                                          (__attribute__((address_space(3))) bf16x4 *)(at)));
                }
                return make_uint4(h2[0].x, h2[0].y, h2[1].x, h2[1].y);
            } else {
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = u * SK + g * 4 + e, c = n + r;
                    v[e] = *(const uint32_t *)(P + k * RB + turn(k, c >> 2) * 16 + (c & 3) * 4);
                }
                return make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    };

    uint4 cur[PIECES], nxt[PIECES];
    uint32_t cur_e[UA ? PIECES : 1] = {}, nxt_e[UA ? PIECES : 1] = {};  // UA: the dwords behind them
    const int64_t nball = (K + BK - 1) / BK;

    // ---- X
    // XQ: the rows side by side, `group` threads each; a thread's first pieces
    // stay in registers.  They are asked for before the first weights, whose
    // longer way from memory the quantization then hides.
    constexpr int XKEEP = 4;
    int group = NT;
    uint4 xkeep[XQ ? XKEEP : 1];
    if constexpr (XQ != 0) {
        using XS = typename Elem<XQ>::S;
        while (NT / group < (int)M) group >>= 1;  // at most NWV rows: a wave or more each
        if (tid / group < (int)M) {
#pragma unroll
            for (int j = 0; j < XKEEP; ++j)
                xkeep[j] = quant_load<XQ>((const XS *)a.A[0] + tid / group * K, (int64_t)(tid % group + j * group) * Elem<XQ>::kVE, K);
        }
    }
    if (wave < nball) load_w(wave, cur, cur_e);
    constexpr int XCAP = XQ ? kFfnQuantLds : 16;
    __shared__ __attribute__((aligned(16))) char xq[XCAP];
    __shared__ uint32_t xtop[XQ ? 16 * MB : 1];
    const int xp = (int)((K + 63) / 64 * 64 + 16);  // row pitch of the quantized rows
    if constexpr (XQ != 0) {
        using XE = Elem<XQ>;
        using XS = typename XE::S;
        constexpr int XV = XE::kVE;
        const int t = tid % group, m = tid / group;
        const XS *xm = (const XS *)a.A[0] + (int64_t)m * K;
        if (tid < 16 * MB) xtop[tid] = 0;
        __syncthreads();
        if (m < (int)M) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < XKEEP; ++j) top = quant_top<XQ>(xkeep[j], top);
            for (int c = t + XKEEP * group; c * XV < (int)K; c += group) top = quant_top<XQ>(quant_load<XQ>(xm, c * XV, K), top);
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
                top = o > top ? o : top;
            }
            if (lane == 0) atomicMax(&xtop[m], top);
        }
        __syncthreads();
        if (m < (int)M) {
            const float rr = quant_factor(xtop[m]);
            char *q = xq + m * xp;  // zeros up to the pitch, which the last step may read
#pragma unroll
            for (int j = 0; j < XKEEP; ++j)
                if ((t + j * group) * XV < xp) quant_store<XQ>(xkeep[j], rr, q + (t + j * group) * XV);
            for (int c = t + XKEEP * group; c * XV < xp; c += group) quant_store<XQ>(quant_load<XQ>(xm, c * XV, K), rr, q + c * XV);
        }
        __syncthreads();
    }
    constexpr bool XUA = UA && XQ == 0;
    gptr x[MB];
    int xr[MB], xsh[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int64_t m = 16 * i + r < M ? 16 * i + r : M - 1;  // rows past the end are not stored
        x[i] = (gptr)a.A[0] + m * a.lda + g * VE;
        xr[i] = (int)m * xp + g * 16;
        if constexpr (XUA) {
            xsh[i] = (int)((uintptr_t)x[i] & 3);
            x[i] -= xsh[i] / ES;
        }
    }
    auto load_x = [&](int64_t kb, uint4 *t, uint32_t *te) {
        const int64_t k0 = kb * BK, krem = K - k0;
        if constexpr (XQ != 0) {
            // Past K: zeros, or the (finite) bytes of a neighbour against
            // weights that are zero there.
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    const int at = xr[i] + (int)k0 + u * SK;
                    t[u * MB + i] = *(const uint4 *)(xq + (at <= XCAP - 16 ? at : 0));
                }
        } else if (krem >= BK) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    t[u * MB + i] = whole_piece<S>(x[i] + k0 + u * SK);
                    if constexpr (XUA) te[u * MB + i] = next_dword(x[i] + k0 + u * SK, xsh[i]);
                }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < MB; ++i)
                    t[u * MB + i] = row_piece<S>(x[i] + (XUA ? xsh[i] / ES : 0) + k0 + u * SK, krem - (u * 4 + g) * VE, K >= VE);
        }
    };

    AccT acc[NF][MB];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[f][i][e] = 0;
    auto mul = [&](const uint4 *tw, const uint32_t *twe, const uint4 *tx, const uint32_t *txe, bool whole) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const uint4 y = frag_w(tw, twe, whole, u, f);
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    uint4 z = tx[u * MB + i];
                    if constexpr (XUA) z = shifted(z, txe[u * MB + i], whole ? xsh[i] : 0);
                    AccT &c = acc[f][i];
                    if constexpr (INT) {
                        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4v, y), __builtin_bit_cast(i32x4v, z), c, 0, 0, 0);
                    } else if constexpr (DT == MM_BFLOAT16) {
                        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, y), __builtin_bit_cast(bf16x8, z), c, 0, 0, 0);
                    } else if constexpr (DT == MM_FLOAT16) {
                        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, y), __builtin_bit_cast(f16x8, z), c, 0, 0, 0);
                    } else {
                        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.x), __uint_as_float(z.x), c, 0, 0, 0);
                        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.y), __uint_as_float(z.y), c, 0, 0, 0);
                        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.z), __uint_as_float(z.z), c, 0, 0, 0);
                        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(y.w), __uint_as_float(z.w), c, 0, 0, 0);
                    }
                }
            }
    };
    for (int64_t kb = wave; kb < nball; kb += NWV) {
        uint4 tx[U * MB];
        uint32_t txe[XUA ? U * MB : 1] = {};
        load_x(kb, tx, txe);
        stage_w(cur);
        if (kb + NWV < nball) load_w(kb + NWV, nxt, nxt_e);
        mul(cur, cur_e, tx, txe, K - kb * BK >= BK);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) cur[i] = nxt[i];
#pragma unroll
        for (int i = 0; i < (UA ? PIECES : 1); ++i) cur_e[i] = nxt_e[i];
    }

    // ---- the waves' sums, in wave order
    // Element e of a lane is column 4 (lane / 16) + e, X row lane % 16.
    using P = typename std::conditional<INT, int, float>::type;
    auto red = (P(*)[NF][MB][256])pool;
    if constexpr (KN) __syncthreads();  // other waves may still read their blocks
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MB; ++i) *(AccT *)&red[wave][f][i][r * 16 + 4 * g] = acc[f][i];
    __syncthreads();
    for (int idx = tid; idx < MB * 16 * COLS; idx += NT) {
        const int c = idx % COLS, m16 = idx / COLS;
        const int i = m16 >> 4, at = (m16 & 15) * 16 + (c & 15);
        const int64_t m = m16, n = n0 + c;
        if (m >= M || n >= N) continue;
        const int64_t o = m * a.ldy + n;
        if constexpr (GLU) {
            float sg = 0.0f, su = 0.0f;
#pragma unroll
            for (int v = 0; v < NWV; ++v) {
                sg += red[v][c >> 4][i][at];
                su += red[v][CF + (c >> 4)][i][at];
            }
            if (a.G()) {
                if (OD != MM_FLOAT && a.kept32()) {
                    ((float *)a.G())[o] = sg;
                    ((float *)a.U())[o] = su;
                } else {
                    ((OS *)a.G())[o] = OE::from_f32(sg);
                    ((OS *)a.U())[o] = OE::from_f32(su);
                }
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
        } else {
            int sum = 0;
#pragma unroll
            for (int v = 0; v < NWV; ++v) sum += (int)red[v][c >> 4][i][at];
            const float bias = a.bias() ? OE::to_f32(((const OS *)a.bias())[n]) : 0.0f;
            // K == 0 takes no scales: the result is the bias.
            const float sa = XQ ? quant_scale(xtop[XQ ? m16 : 0]) : K > 0 ? a.sa()[m] : 0.0f;
            ((OS *)a.Y[0])[o] = OE::from_f32(scaled_value(sum, sa, K > 0 ? a.sb()[n] : 0.0f, bias));
        }
    }
#endif
}

// Waves of a workgroup: 8, or 4 where the columns make more than the 512
// workgroups of 8 that fit the GPU at once, so that all start together ([N, K]
// weights, M = 1, K = 4096, N = 11008: INT8 13.9 against 11.9 us, gated BF16
// 38.9 against 37.8; INT8 K = 11008, N = 4096: 12.8 with 8, 14.7 with 4).
constexpr int64_t kRowsFit = 512;

template <int DT, int OD, bool GLU, bool KN, int NF, int MB, int NWV, int XQ, bool UA = false>
static hipError_t launch_rows(const FfnArgs &a, hipStream_t s) {
    constexpr int COLS = 16 * NF / (GLU ? 2 : 1);
    const int64_t wgs = (a.N + COLS - 1) / COLS;
    if (wgs <= 0 || a.M <= 0) return hipSuccess;
    if (wgs > 0x7fffffff || a.M > 16 * MB) return hipErrorInvalidValue;
    if constexpr (!KN && NWV == 8) {
        if (wgs > kRowsFit) return launch_rows<DT, OD, GLU, KN, NF, MB, 4, XQ, UA>(a, s);
    }
    constexpr int ES = (int)sizeof(typename Elem<DT>::S);
    if constexpr (!KN && ES < 4 && !UA) {
        uintptr_t low = (uintptr_t)a.B[0] | (uintptr_t)a.B[1] | (uintptr_t)(a.ldb * ES);
        if (XQ == 0) low |= (uintptr_t)a.A[0] | (uintptr_t)(a.lda * ES);
        if (low & 3) return launch_rows<DT, OD, GLU, KN, NF, MB, NWV, XQ, true>(a, s);
    }
    if constexpr (KN && NF > (GLU ? 2 : 1)) {
        if (rows_halve(wgs)) return launch_rows<DT, OD, GLU, KN, NF / 2, MB, NWV, XQ>(a, s);
    }
    hipLaunchKernelGGL((k_ffn_rows<DT, OD, GLU, KN, NF, MB, NWV, XQ, UA>), dim3((unsigned)wgs), dim3(64 * NWV), 0, s,
                       slim_args<FfnSlim>(a, GLU ? kUseGlu : kUseScaled, false, false));
    return hipGetLastError();
}

}  // namespace mm
