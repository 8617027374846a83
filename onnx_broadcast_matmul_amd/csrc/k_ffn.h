// k_ffn.h -- tiled products of the feed-forward operators on the gfx950
// matrix cores: the gated block (two weight matrices, one fused epilogue), the
// two-term input gradient, the pair of weight gradients, and the INT8 product
// with row and column scales.
//
// One workgroup owns a BM x BN tile (for the gated block BN counts the gate
// and the up columns: BN / 2 hidden features).  K moves through STAGES LDS
// buffers of BKB bytes per staged row, and the pipeline looks one stage
// further ahead than the one computed: at stage kt's barrier every wave's
// loads of stage kt + 1 have landed, so the first fragments of kt + 1 are
// read while the last MFMAs of kt run and the matrix cores do not wait for
// LDS at the stage's start.  The loads of kt + STAGES - 1 are issued after
// that barrier, into the buffer whose last reads ended before it.
//
// Operands are staged as they lie in memory: K-contiguous rows (chunk c of
// row r at c ^ aswz(r)) or M/N-contiguous rows of one k each (chunk c at
// c ^ kn_swizzle(k)), read back as 16-byte MFMA operands directly or through
// the transposing LDS reads.
//
// DMA = true needs 16-byte aligned rows and bases and moves global memory
// straight into LDS.  DMA = false takes any alignment: every thread loads its
// chunks into registers one stage ahead (whole 16-byte chunks where they lie
// inside the row, single elements at its end) and writes them to the same LDS
// layout, so odd sizes run on the same matrix-core loop (512 x 2560 x 5504 gated,
// BF16: 41 us, with K = 2561 65).
//
// What bounds it.  Large products: power.  8192 x 4096 x 11008 in BF16 takes 1.20
// ms gated (1.23 PFLOP/s), 1.17 for dX, 1.32 for dWg and dWu, and 0.36 in INT8
// (2.07 POP/s); the matrix cores are busy 67-73 % of the cycles at the clock
// that random operands leave (zeros, which take less power, run at 1.5-1.6
// PFLOP/s).  A persistent form, which loads the next tile's first stages during
// the epilogue, gained nothing there and took 10 % more for INT8.  Products
// of about one tile per CU: the 256 x 128 tile's shorter runs of MFMAs (48 % busy:
// 4096 x 2048 x 5504, dX 0.20 ms) and the ends of a tile, which no other work
// covers (1000 x 1024 x 4096 gated: 23 us, 15 of them in the K loop).
#pragma once

#include <type_traits>

#include "activation.h"
#include "device.h"
#include "ffn.h"
#include "pieces.h"

namespace mm {

// 16-byte chunk swizzle of M/N-contiguous rows (one k each) of cpr chunks:
// 16-bit transposing reads cover 4 rows x 4 chunks per half-wave, 8-bit ones
// 8 rows x 2 neighbouring chunks, FP32 column reads rows k and k + 4.
template <int ES>
__device__ __forceinline__ int row_swizzle(int k, int cpr) {
    if constexpr (ES == 4) return cpr >= 16 ? 8 * ((k >> 2) & 1) : 0;
    else if constexpr (ES == 1) return cpr >= 16 ? 2 * (k & 7) : 2 * ((k >> 1) & 3);
    else return cpr >= 16 ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
}

// Which products a kernel computes.
//   kGlu:    H = act(A B0) * (A B1), optionally also A B0 and A B1, in OD or
//            (flags) as their FP32 sums: 4096 x 2048 x 5504 BF16 171 us without
//            them, 181 and 196 with (8192 x 4096 x 11008: 1199, 1241, 1287)
//   kSum2:   Y0 = A0 B0 + A1 B1 (the K loop runs over both terms)
//   kPair:   Y0 = A0 B0 and Y1 = A1 B1 (half of the grid each)
//   kScaled: Y = sa[m] sb[n] (A B) + bias[n], INT8 operands
// SPLIT: a workgroup takes a range of K stages and writes FP32 (INT8
// operands: INT32) partial sums to the workspace.
// KG groups of WGM x WGN waves share the tile; group g takes every KG-th MFMA
// step of a stage, and their sums are added in group order at the end.
// BATCH (kScaled): more than one product.
enum FfnMode { kGlu = 0, kSum2 = 1, kPair = 2, kScaled = 3 };

template <int DT, int OD, int MODE, bool SPLIT, bool TA, bool TB, int BM, int BN, int WGM, int WGN, int KG, int BKB,
          int STAGES, int PW, bool DMA, bool BATCH>
__global__ __launch_bounds__(64 * WGM * WGN * KG) void k_ffn(typename std::conditional<BATCH, FfnSlimBatch, FfnSlim>::type a) {
#if defined(__HIP_DEVICE_COMPILE__)
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr bool INT = DT == MM_INT8;
    constexpr int NWG = WGM * WGN;         // waves of one K group
    constexpr int NW = NWG * KG;
    constexpr int NT = 64 * NW;
    constexpr int ES = (int)sizeof(S);
    constexpr int VE = 16 / ES;
    constexpr int BK = BKB / ES;
    constexpr int CA = BKB / 16;           // chunks of a K-contiguous row
    constexpr int KS = BKB / 32;           // MFMA steps per stage
    constexpr int NPAN = MODE == kGlu ? 2 : 1;  // B panels (gate, up)
    constexpr int PN = BN / NPAN;          // columns of one panel = output columns of the tile
    constexpr int WM = BM / WGM, WNP = PN / WGN;
    constexpr int FM = WM / 32, FNP = WNP / 32, FN = FNP * NPAN;
    constexpr int RBA = BM * ES, CPRA = RBA / 16;  // M-contiguous A rows
    constexpr int RBB = PN * ES, CPRB = RBB / 16;  // N-contiguous B rows
    constexpr int A_BYTES = BM * BKB;
    constexpr int P_BYTES = PN * BKB;      // one B panel
    constexpr int STAGE_BYTES = A_BYTES + NPAN * P_BYTES;
    static_assert(CA == 4 || CA == 8 || CA == 16, "K-contiguous rows are 64, 128 or 256 bytes");
    static_assert(KS % (2 * KG) == 0, "an even number of steps per group and stage");
    static_assert(FM >= 1 && FNP >= 1 && BM % (32 * WGM) == 0 && PN % (32 * WGN) == 0, "wave tile");
    static_assert(STAGES >= 3 && STAGES * STAGE_BYTES <= 160 * 1024, "LDS");
    static_assert(!TA || (CPRA >= 8 && CPRA <= 64), "transposed A rows");
    static_assert(TB || (CPRB >= 8 && CPRB <= 64), "B rows");
    auto aswz = [](int row) { return CA == 16 ? (row & 15) : CA == 8 ? ((row >> 1) & 7) : ((row >> 2) & 3); };

    __shared__ __attribute__((aligned(1024))) char lds[STAGES * STAGE_BYTES];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kg = wave / NWG;
    const int wr = (wave % NWG) / WGN, wc = wave % WGN;

    const int64_t M = a.M, N = a.N, K = a.K;
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + PN - 1) / PN;
    const int64_t per = tiles_m * tiles_n;
    const int64_t nsplit = SPLIT ? a.split : 1;
    int64_t id = xcd_remap(blockIdx.x, (int64_t)gridDim.x);
    const int64_t sidx = SPLIT ? id % nsplit : 0;
    if constexpr (SPLIT) id /= nsplit;
    const int64_t b = id / per;  // batch (kScaled) or which of the pair
    const int64_t t = id % per;
    // 8 tile rows sweep the tile columns together, so that they share B.
    constexpr int64_t GM = 8;
    const int64_t group = t / (GM * tiles_n);
    const int64_t first_m = group * GM;
    const int64_t gsize = (tiles_m - first_m) < GM ? (tiles_m - first_m) : GM;
    const int64_t tm = first_m + (t % (GM * tiles_n)) % gsize;
    const int64_t tn = (t % (GM * tiles_n)) / gsize;
    const int64_t m0 = tm * BM, n0 = tn * PN;

    int64_t oa = 0, ob = 0;
    if constexpr (BATCH) batch_offsets(a.bd, b, oa, ob);
    // Tile origins of the two A and B operands (the modes that have one use [0]).
    const int64_t ta_off = oa + (TA ? m0 : m0 * a.lda), tb_off = ob + (TB ? n0 * a.ldb : n0);
    const int pick = MODE == kPair ? (int)b : 0;
    const char *At0 = (const char *)((const S *)a.A[pick] + ta_off);
    const char *Bt0 = (const char *)((const S *)a.B[pick] + tb_off);
    const char *At1 = MODE == kSum2 ? (const char *)((const S *)a.A[1] + ta_off) : At0;
    const char *Bt1 = MODE == kSum2 || MODE == kGlu ? (const char *)((const S *)a.B[1] + tb_off) : Bt0;

    // Stages of this workgroup: all of them (kSum2: both terms' in turn), or
    // its partition's.
    const int64_t kend = K;
    const int nk1 = (int)((K + BK - 1) / BK);
    const int nkall = MODE == kSum2 ? 2 * nk1 : nk1;
    const int st0 = SPLIT ? (int)sidx * a.kstages : 0;
    const int nk = SPLIT ? (nkall - st0 < a.kstages ? nkall - st0 : a.kstages) : nkall;

    using AccT = typename std::conditional<INT, i32x16, f32x16>::type;
    AccT acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

    // ---- fragments
    uint4 fa[2][FM], fb[2][FN];
    auto read_k = [&](const char *Xs, int row, int c) -> uint4 {
        return *(const uint4 *)(Xs + row * BKB + ((c ^ aswz(row)) * 16));
    };
    // 16 bytes of consecutive k of index base + lane % 32, from rows of one k
    // each.  Transposing reads: in each 16-lane group the lanes address the
    // pieces of a (16 / ES / 2) x 16 block and lane i receives column i.
    auto read_mn = [&](const char *Xs, int rbytes, int cpr, int base, int ks) -> uint4 {
        const int G = lane >> 4, jl = lane & 15;
        if constexpr (ES == 1) {
            typedef int i32x2v __attribute__((ext_vector_type(2)));
            const int n = base + (G & 1) * 16 + (jl & 1) * 8;
            uint2 h2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = ks * 32 + (G >> 1) * 16 + h * 8 + (jl >> 1);
                const char *addr = Xs + k * rbytes + ((n >> 4) ^ row_swizzle<ES>(k, cpr)) * 16 + ((n >> 3) & 1) * 8;
                h2[h] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                                      (__attribute__((address_space(3))) i32x2v *)(addr)));
            }
            return make_uint4(h2[0].x, h2[0].y, h2[1].x, h2[1].y);
        } else if constexpr (ES == 2) {
            const int n = base + (G & 1) * 16 + (jl & 3) * 4;
            uint2 h2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = ks * 16 + (G >> 1) * 8 + h * 4 + (jl >> 2);
                const char *addr = Xs + k * rbytes + ((n >> 3) ^ row_swizzle<ES>(k, cpr)) * 16 + ((n >> 2) & 1) * 8;
                h2[h] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                                                      (__attribute__((address_space(3))) bf16x4 *)(addr)));
            }
            return make_uint4(h2[0].x, h2[0].y, h2[1].x, h2[1].y);
        } else {
            const int n = base + (lane & 31), c = 2 * ks + (lane >> 5);
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = c * 4 + e;
                v[e] = *(const uint32_t *)(Xs + k * rbytes + ((n >> 2) ^ row_swizzle<ES>(k, cpr)) * 16 + (n & 3) * 4);
            }
            return make_uint4(v[0], v[1], v[2], v[3]);
        }
    };
    auto read_frags = [&](int buf, int ks, int slot) {
        const char *As = lds + buf * STAGE_BYTES;
        const char *Bs = As + A_BYTES;
        const int c = 2 * ks + (lane >> 5);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if constexpr (TA) fa[slot][i] = read_mn(As, RBA, CPRA, wr * WM + i * 32, ks);
            else fa[slot][i] = read_k(As, wr * WM + i * 32 + (lane & 31), c);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const char *Ps = Bs + (j / FNP) * P_BYTES;
            const int col = wc * WNP + (j % FNP) * 32;
            if constexpr (TB) fb[slot][j] = read_k(Ps, col + (lane & 31), c);
            else fb[slot][j] = read_mn(Ps, RBB, CPRB, col, ks);
        }
    };
    // B is the first MFMA operand: accumulator element r of a lane is output
    // row lane % 32 and column 8 (r / 4) + 4 (lane / 32) + r % 4 of the block.
    auto mfmas = [&](int slot) {
        if constexpr (DT == MM_FLOAT) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const uint4 &x = fa[slot][i];
                        const uint4 &y = fb[slot][j];
                        const float av = __uint_as_float(e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w);
                        const float bv = __uint_as_float(e == 0 ? y.x : e == 1 ? y.y : e == 2 ? y.z : y.w);
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(bv, av, acc[i][j], 0, 0, 0);
                    }
        } else {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if constexpr (INT) {
                        typedef int i32x4v __attribute__((ext_vector_type(4)));
                        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4v, fb[slot][j]),
                                                                         __builtin_bit_cast(i32x4v, fa[slot][i]),
                                                                         acc[i][j], 0, 0, 0);
                    } else if constexpr (DT == MM_BFLOAT16) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, fb[slot][j]),
                                                                           __builtin_bit_cast(bf16x8, fa[slot][i]),
                                                                           acc[i][j], 0, 0, 0);
                    } else {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, fb[slot][j]),
                                                                          __builtin_bit_cast(f16x8, fa[slot][i]),
                                                                          acc[i][j], 0, 0, 0);
                    }
                }
        }
    };
    // One stage's MFMA steps; the last step reads the next stage's first
    // fragments (after the last stage: stale bytes that nothing uses).  `mid`
    // runs after the first step's MFMAs: the loads of a later stage issued
    // there and not at the barrier let every wave start its MFMAs at once
    // (8192 x 4096 x 11008: gated 1300 -> 1274 us, dX 1216 -> 1200, INT8 365 ->
    // 355, dW the same).
    auto compute = [&](int buf, int next, auto mid) {
        constexpr bool SCHED = DT != MM_FLOAT;
        constexpr int RPS = FM * (TA ? 2 : 1) + FN * (TB ? 1 : 2);  // LDS reads per step
        constexpr int MPS = FM * FN;                              // MFMAs per step
        constexpr int R2 = (RPS + 1) / 2;
#pragma unroll
        for (int j = 0; j < KS / KG; ++j) {
            if (j + 1 < KS / KG) read_frags(buf, kg + (j + 1) * KG, (j + 1) & 1);
            else read_frags(next, kg, (j + 1) & 1);
            mfmas(j & 1);
            if (j == 0) mid();
            if constexpr (SCHED) {
                {
#pragma unroll
                    for (int q = 0; q < (R2 < MPS ? R2 : MPS); ++q) {
                        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    }
                    if constexpr (MPS > R2) __builtin_amdgcn_sched_group_barrier(0x008, MPS - R2, 0);
                }
            }
        }
    };

    // A stage's first k and operands: kSum2 runs over the first term's stages,
    // then the second's.
    auto stage_second = [&](int st) { return MODE == kSum2 && st0 + st >= nk1; };
    auto stage_k0 = [&](int st) { return (int64_t)(st0 + st - (stage_second(st) ? nk1 : 0)) * BK; };

    if constexpr (DMA) {
        constexpr int A_INSTR = A_BYTES / 1024 / PW;  // 1 KB loads per producer and stage
        constexpr int B_INSTR = NPAN * P_BYTES / 1024 / PW;
        constexpr int LPW = A_INSTR + B_INSTR;
        constexpr int A_RPB = TA ? 1024 / RBA : 1024 / BKB;
        constexpr int B_RPB = TB ? 1024 / BKB : 1024 / RBB;
        static_assert(PW >= 1 && PW <= NW && A_INSTR * PW * 1024 == A_BYTES && A_INSTR >= 1, "A loads");
        static_assert(B_INSTR * PW * 1024 == NPAN * P_BYTES && B_INSTR >= NPAN && B_INSTR % NPAN == 0, "B loads");
        static_assert((STAGES - 2) * LPW < 64, "vmcnt range");
        const uint32_t lds_base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char *)lds);
        const bool producer = wave < PW;
        // 1 KB block of load q of this producer: q * PW + wave, so that a B
        // load's panel depends on q only.
        uint32_t a_off[A_INSTR], b_off[B_INSTR];
        int a_k[A_INSTR], b_k[B_INSTR];
#pragma unroll
        for (int q = 0; q < A_INSTR; ++q) {
            const int blk = q * PW + wave;
            if constexpr (!TA) {
                const int row = blk * A_RPB + lane / CA;
                const int c = (lane % CA) ^ aswz(row);
                a_off[q] = m0 + row < M ? (uint32_t)((int64_t)row * a.lda * ES + c * 16) : kOutOfRange;
                a_k[q] = c * VE;
            } else {
                const int row = blk * A_RPB + lane / CPRA;
                const int c = (lane % CPRA) ^ row_swizzle<ES>(row, CPRA);
                a_off[q] = m0 + c * VE < M ? (uint32_t)((int64_t)row * a.lda * ES + c * 16) : kOutOfRange;
                a_k[q] = row;
            }
        }
#pragma unroll
        for (int q = 0; q < B_INSTR; ++q) {
            const int blk = (q * PW + wave) % (P_BYTES / 1024);
            if constexpr (!TB) {
                const int row = blk * B_RPB + lane / CPRB;
                const int c = (lane % CPRB) ^ row_swizzle<ES>(row, CPRB);
                b_off[q] = n0 + c * VE < N ? (uint32_t)((int64_t)row * a.ldb * ES + c * 16) : kOutOfRange;
                b_k[q] = row;
            } else {
                const int row = blk * B_RPB + lane / CA;
                const int c = (lane % CA) ^ aswz(row);
                b_off[q] = n0 + row < N ? (uint32_t)((int64_t)row * a.ldb * ES + c * 16) : kOutOfRange;
                b_k[q] = c * VE;
            }
        }
        auto issue = [&](int st) {
            if (!producer) return;
            const uint32_t sbase = lds_base + (st % STAGES) * STAGE_BYTES;
            const int64_t k0 = stage_k0(st);
            const bool second = stage_second(st);
            const int64_t ka = (TA ? k0 * a.lda : k0) * ES, kb = (TB ? k0 : k0 * a.ldb) * ES;
            const i32x4 ra = buffer_rsrc((second ? At1 : At0) + ka);
            const i32x4 rb0 = buffer_rsrc((second ? Bt1 : Bt0) + kb);
            const i32x4 rb1 = MODE == kGlu ? buffer_rsrc(Bt1 + kb) : rb0;
            if (k0 + BK <= kend) {
#pragma unroll
                for (int q = 0; q < A_INSTR; ++q) load_to_lds16(ra, sbase + (q * PW + wave) * 1024, a_off[q]);
#pragma unroll
                for (int q = 0; q < B_INSTR; ++q)
                    load_to_lds16(q * NPAN >= B_INSTR ? rb1 : rb0, sbase + A_BYTES + (q * PW + wave) * 1024, b_off[q]);
            } else {
                const int rem = (int)(kend - k0);
#pragma unroll
                for (int q = 0; q < A_INSTR; ++q)
                    load_to_lds16(ra, sbase + (q * PW + wave) * 1024, a_k[q] < rem ? a_off[q] : kOutOfRange);
#pragma unroll
                for (int q = 0; q < B_INSTR; ++q)
                    load_to_lds16(q * NPAN >= B_INSTR ? rb1 : rb0, sbase + A_BYTES + (q * PW + wave) * 1024,
                                  b_k[q] < rem ? b_off[q] : kOutOfRange);
            }
        };
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s)
            if (s < nk) issue(s);
        // Stage 0 has landed in every wave's share before its first fragments are read.
        if (nk >= STAGES - 1) wait_vmcnt<(STAGES - 2) * LPW>();
        else wait_vmcnt<0>();
        asm volatile("s_barrier" ::: "memory");
        if (nk > 0) read_frags(0, kg, 0);
        for (int kt = 0; kt < nk; ++kt) {
            // Loads of stage kt + 1 are complete once at most those of the
            // STAGES - 3 stages issued after it are outstanding.
            if (nk - 2 - kt >= STAGES - 3) wait_vmcnt<(STAGES - 3) * LPW>();
            else wait_vmcnt<0>();
            // Every wave's reads of stage kt - 1 have ended: lgkmcnt(0).
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            compute(kt % STAGES, (kt + 1) % STAGES, [&]() {
                if (kt + STAGES - 1 < nk) issue(kt + STAGES - 1);
            });
        }
    } else {
        // Chunks of A and of each B panel per thread and stage.
        constexpr int AC = A_BYTES / 16 / NT, BC = P_BYTES / 16 / NT;
        static_assert(AC * NT * 16 == A_BYTES && BC * NT * 16 == P_BYTES, "whole chunks per thread");
        uint4 rga[AC], rgb[NPAN][BC];
        // One operand's chunks of a stage starting at k0 (KC: K-contiguous
        // rows).  A whole stage loads whole chunks without a test: rows past
        // the matrix read its last row, and chunks that cross a row's end
        // read on into the next rows (where the matrix goes on for that long);
        // both reach only outputs that are not stored.  The last stage may
        // neither read past the matrix nor bring in values past K: it goes
        // straight to LDS when it is its turn to be stored.  (Brought through
        // the same registers, its shifts made every stage wait for its loads:
        // 1.7-2.4 times the time per stage.)
        auto whole_stage = [&](bool kc, int cpr, int64_t ld, int64_t left_mn, int64_t k0) {
            const int64_t krem = kend - k0;
            return krem >= BK && (kc || left_mn >= (int64_t)cpr * VE || (krem - BK) * ld >= VE);
        };
        auto gather = [&](auto kc_t, auto cpr_t, auto count_t, const char *base, int64_t ld, int64_t left_mn, int64_t k0,
                          uint4 *out) {
            constexpr bool KC = decltype(kc_t)::value;
            constexpr int CPR = decltype(cpr_t)::value, COUNT = decltype(count_t)::value;
            if (!whole_stage(KC, CPR, ld, left_mn, k0)) return;
            const GlobalPtr<S> g = (GlobalPtr<S>)base;
#pragma unroll
            for (int i = 0; i < COUNT; ++i) {
                const int y = tid + NT * i;
                int row = y / CPR;
                const int c = (y % CPR) ^ (KC ? aswz(row) : row_swizzle<ES>(row, CPR));
                int64_t at;
                if constexpr (KC) {
                    if (row >= left_mn) row = (int)left_mn - 1;
                    at = (int64_t)row * ld + k0 + c * VE;
                } else {
                    // Columns wholly past the matrix: its first ones.
                    at = (k0 + row) * ld + (c * VE < left_mn ? c * VE : 0);
                }
                out[i] = whole_piece<S>(g + at);
            }
        };
        auto scatter = [&](auto kc_t, auto cpr_t, auto count_t, const char *base, int64_t ld, int64_t left_mn,
                           int64_t row_len, int64_t k0, const uint4 *in, char *dst) {
            constexpr bool KC = decltype(kc_t)::value;
            constexpr int CPR = decltype(cpr_t)::value, COUNT = decltype(count_t)::value;
            if (whole_stage(KC, CPR, ld, left_mn, k0)) {
#pragma unroll
                for (int i = 0; i < COUNT; ++i) *(uint4 *)(dst + (tid + NT * i) * 16) = in[i];
                return;
            }
            const GlobalPtr<S> g = (GlobalPtr<S>)base;
            const int64_t krem = kend - k0;
#pragma unroll
            for (int i = 0; i < COUNT; ++i) {
                const int y = tid + NT * i;
                const int row = y / CPR;
                const int c = (y % CPR) ^ (KC ? aswz(row) : row_swizzle<ES>(row, CPR));
                const int64_t left = KC ? (row < left_mn ? krem - c * VE : 0) : (row < krem ? left_mn - c * VE : 0);
                const int64_t at = KC ? (int64_t)row * ld + k0 + c * VE : (k0 + row) * ld + c * VE;
                *(uint4 *)(dst + y * 16) = row_piece<S>(g + at, left, row_len >= VE);
            }
        };
        using AKC = std::integral_constant<bool, !TA>;
        using BKC = std::integral_constant<bool, TB>;
        using ACPR = std::integral_constant<int, TA ? CPRA : CA>;
        using BCPR = std::integral_constant<int, TB ? CA : CPRB>;
        auto load = [&](int st) {
            const int64_t k0 = stage_k0(st);
            const bool second = stage_second(st);
            gather(AKC(), ACPR(), std::integral_constant<int, AC>(), second ? At1 : At0, a.lda, M - m0, k0, rga);
#pragma unroll
            for (int p = 0; p < NPAN; ++p)
                gather(BKC(), BCPR(), std::integral_constant<int, BC>(), second || p == 1 ? Bt1 : Bt0, a.ldb, N - n0, k0,
                       rgb[p]);
        };
        auto store = [&](int st) {
            char *sb = lds + (st % STAGES) * STAGE_BYTES;
            const int64_t k0 = stage_k0(st);
            const bool second = stage_second(st);
            scatter(AKC(), ACPR(), std::integral_constant<int, AC>(), second ? At1 : At0, a.lda, M - m0, TA ? M : K, k0,
                    rga, sb);
#pragma unroll
            for (int p = 0; p < NPAN; ++p)
                scatter(BKC(), BCPR(), std::integral_constant<int, BC>(), second || p == 1 ? Bt1 : Bt0, a.ldb, N - n0,
                        TB ? K : N, k0, rgb[p], sb + A_BYTES + p * P_BYTES);
        };
        // Stages 0 and 1 go through the same registers one after the other: two
        // memory latencies before the first MFMA, and a partial last stage's
        // own where it is stored, which products of few stages feel (333 x 1000
        // x 1501 INT8, four stages: 8.5 us, of which the bytes take 0.7).
        if (nk > 0) {
            load(0);
            store(0);
        }
        if (nk > 1) {
            load(1);
            store(1);
        }
        if (nk > 2) load(2);
        __syncthreads();
        if (nk > 0) read_frags(0, kg, 0);
        for (int kt = 0; kt < nk; ++kt) {
            // Stage kt + 2 goes to a buffer last read before the previous
            // barrier and is visible after the next one.
            __syncthreads();
            if (kt + 2 < nk) store(kt + 2);
            if (kt + 3 < nk) load(kt + 3);
            compute(kt % STAGES, (kt + 1) % STAGES, []() {});
        }
    }

    // ---- epilogue
    // A wave's blocks go through LDS (chunk c of tile row r at c ^ r % OCPR)
    // so that the workgroup writes whole 16-byte chunks of output rows; tiles
    // larger than the stage buffers go in row passes.
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    using OE = Elem<OD>;
    // K groups meet through LDS, their sums added in group order.  Of four
    // groups each takes a quarter of every accumulator (QG quarters of four
    // columns) and carries it through the epilogue, so that all eight waves
    // work there and not two (300 x 512 x 1364 FP32, gelu: 15.4 -> 14.3 us); of two
    // groups the first takes all (halves gained nothing).
    constexpr int QG = KG > 2 ? 4 / KG : 4;
    auto mine = [&](int q) { return KG <= 2 || q / QG == kg; };
    static_assert((KG - 1) * BM * BN * 4 <= STAGES * STAGE_BYTES, "K group exchange");
    if constexpr (KG == 2) {
        using T = typename std::conditional<INT, int, float>::type;
        T *xch = (T *)lds;
        auto at = [&](int i, int j, int r) { return (((wave % NWG) * FM + i) * FN * 16 + j * 16 + r) * 64 + lane; };
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) xch[at(i, j, r)] = acc[i][j][r];
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kg == 0) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] += xch[at(i, j, r)];
        }
    } else if constexpr (KG > 2) {
        using T = typename std::conditional<INT, int, float>::type;
        uint4 *xch = (uint4 *)lds;
        // What group s holds of group d's quarter q.
        auto at = [&](int d, int s, int i, int j, int q) {
            return (((((d * (KG - 1) + (s < d ? s : s - 1)) * NWG + wave % NWG) * FM + i) * FN + j) * QG + q % QG) * 64 + lane;
        };
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (!mine(q)) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const T part[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                        uint4 x;
                        __builtin_memcpy(&x, part, 16);
                        xch[at(q / QG, kg, i, j, q)] = x;
                    }
            }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (mine(q)) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        T sum[4];
#pragma unroll
                        for (int g = 0; g < KG; ++g) {
                            T part[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                            if (g != kg) {
                                const uint4 x = xch[at(kg, g, i, j, q)];
                                __builtin_memcpy(part, &x, 16);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[e] = g ? sum[e] + part[e] : part[e];
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] = sum[e];
                    }
            }
    }
    auto emit = [&](auto zero, int jbase, auto value, void *outp, int64_t ldo, bool vec) {
        using O = decltype(zero);
        constexpr int OS = (int)sizeof(O), OV = 16 / OS;
        constexpr int OCPR = PN * OS / 16;
        constexpr int NP = (BM * PN * OS + STAGES * STAGE_BYTES - 1) / (STAGES * STAGE_BYTES);
        constexpr int PR = BM / NP;
        static_assert(BM % NP == 0 && (OCPR & (OCPR - 1)) == 0, "epilogue passes");
        O *out = (O *)outp;
#pragma unroll
        for (int pass = 0; pass < NP; ++pass) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int rl = wr * WM + i * 32 + (lane & 31) - pass * PR;
                if ((KG > 2 || kg == 0) && (NP == 1 || (rl >= 0 && rl < PR))) {
                    char *trow = lds + rl * (PN * OS);
#pragma unroll
                    for (int j = 0; j < FNP; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (!mine(q)) continue;
                            const int cl = wc * WNP + j * 32 + 8 * q + 4 * (lane >> 5);
                            char *dst = trow + ((cl / OV) ^ (rl & (OCPR - 1))) * 16 + (cl % OV) * OS;
                            const AccT &v = acc[i][jbase + j];
                            if constexpr (std::is_same<O, int32_t>::value) {
                                *(uint4 *)dst = make_uint4((uint32_t)v[4 * q], (uint32_t)v[4 * q + 1],
                                                           (uint32_t)v[4 * q + 2], (uint32_t)v[4 * q + 3]);
                            } else {
                                float w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[e] = value(i, cl + e, v[4 * q + e]);
                                using PK = Elem<OS == 4 ? MM_BFLOAT16 : OD>;
                                if constexpr (OS == 4) *(float4 *)dst = make_float4(w[0], w[1], w[2], w[3]);
                                else *(uint2 *)dst = make_uint2(PK::pack2(w[0], w[1]), PK::pack2(w[2], w[3]));
                            }
                        }
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            for (int idx = tid; idx < PR * OCPR; idx += NT) {
                const int rl = idx / OCPR, c = idx % OCPR;
                const int64_t row = m0 + pass * PR + rl, col = n0 + (int64_t)c * OV;
                if (row < M && col < N) {
                    const uint4 v = *(const uint4 *)(lds + rl * (PN * OS) + (c ^ (rl & (OCPR - 1))) * 16);
                    O *dst = out + row * ldo + col;
                    if (vec) {
                        const u32x4 w = {v.x, v.y, v.z, v.w};
                        __builtin_nontemporal_store(w, (u32x4 *)dst);
                    } else if (col + OV <= N) {
                        __builtin_memcpy(dst, &v, 16);  // any alignment
                    } else {
                        O e[OV];
                        __builtin_memcpy(e, &v, 16);
#pragma unroll
                        for (int q = 0; q < OV; ++q)
                            if (col + q < N) dst[q] = e[q];
                    }
                }
            }
        }
    };
    auto plain = [](int, int, auto v) { return (float)v; };
    if constexpr (SPLIT && MODE == kGlu) {
        // Partials of G, then of U, for every partition.
        float *w = (float *)a.part() + sidx * 2 * M * N;
        emit(0.0f, 0, plain, w, N, N % 4 == 0);
        emit(0.0f, FNP, plain, w + M * N, N, N % 4 == 0);
    } else if constexpr (SPLIT) {
        using T = typename std::conditional<INT, int32_t, float>::type;
        int64_t nprod = MODE == kPair ? 2 : 1;
        if constexpr (BATCH) nprod = a.batch;
        emit((T)0, 0, plain, (T *)a.part() + (sidx * nprod + b) * M * N, N, N % 4 == 0);
    } else if constexpr (MODE == kGlu) {
        if (a.G()) {
            if (OD != MM_FLOAT && a.kept32()) {
                emit(0.0f, 0, plain, a.G(), a.ldy, a.kept_vec());
                emit(0.0f, FNP, plain, a.U(), a.ldy, a.kept_vec());
            } else {
                emit((typename OE::S)0, 0, plain, a.G(), a.ldy, a.kept_vec());
                emit((typename OE::S)0, FNP, plain, a.U(), a.ldy, a.kept_vec());
            }
        }
        auto apply = [&](auto kind) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FNP; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (mine(r / 4))
                            acc[i][j][r] = act_value<decltype(kind)::value, DT == MM_FLOAT>(acc[i][j][r]) * acc[i][FNP + j][r];
        };
        if (KG > 2 || kg == 0) switch (a.act) {
        case MM_ACT_SILU: apply(std::integral_constant<int, MM_ACT_SILU>()); break;
        case MM_ACT_GELU: apply(std::integral_constant<int, MM_ACT_GELU>()); break;
        case MM_ACT_GELU_TANH: apply(std::integral_constant<int, MM_ACT_GELU_TANH>()); break;
        case MM_ACT_RELU: apply(std::integral_constant<int, MM_ACT_RELU>()); break;
        default: apply(std::integral_constant<int, MM_ACT_SIGMOID>()); break;
        }
        emit((typename OE::S)0, 0, plain, a.Y[0], a.ldy, a.y_vec());
    } else if constexpr (MODE == kScaled) {
        // Scales of this lane's rows, and of the tile's columns in LDS after
        // the main loop's last reads.  K == 0: the matrices are empty, their
        // batch offsets tell no scales apart, and zeros in the scales' place
        // leave the bias alone.
        __shared__ __attribute__((aligned(16))) float cs[PN], cb[PN];
        const int64_t sb0 = K > 0 ? ob / K + n0 : 0;  // scale of column n of B matrix i: i N + n
        for (int x = tid; x < PN; x += NT) {
            const bool in = n0 + x < N;
            cs[x] = in && K > 0 ? a.sb()[sb0 + x] : 0.0f;
            cb[x] = in && a.bias() ? OE::to_f32(((const typename OE::S *)a.bias())[n0 + x]) : 0.0f;
        }
        float rs[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int64_t row = m0 + wr * WM + i * 32 + (lane & 31);
            rs[i] = row < M && K > 0 ? a.sa()[oa / a.lda + row] : 0.0f;
        }
        __syncthreads();
        emit((typename OE::S)0, 0, [&](int i, int cl, int v) { return scaled_value(v, rs[i], cs[cl], cb[cl]); },
             (typename OE::S *)a.Y[0] + b * M * a.ldy, a.ldy, a.y_vec());
    } else {
        emit((typename OE::S)0, 0, plain, MODE == kPair ? a.Y[pick] : a.Y[0], a.ldy, a.y_vec());
    }
#endif
}

// Launch one entry; DMA where the operands allow it (`vec`).
template <int DT, int OD, int MODE, bool SPLIT, bool TA, bool TB, int BM, int BN, int WGM, int WGN, int KG, int BKB,
          int STAGES, int PW>
static hipError_t launch_ffn(bool vec, const FfnArgs &a, hipStream_t s) {
    constexpr int PN = MODE == kGlu ? BN / 2 : BN;
    constexpr int ES = (int)sizeof(typename Elem<DT>::S);
    const int64_t tiles = a.batch * ((a.M + BM - 1) / BM) * ((a.N + PN - 1) / PN) * (SPLIT ? a.split : 1);
    if (tiles <= 0) return hipSuccess;
    if (tiles > 0x7fffffff) return hipErrorInvalidValue;
    // Buffer offsets are 32-bit: the rows that one stage of a tile spans.
    const int64_t a_span = (TA ? (int64_t)(BKB / ES) : (int64_t)BM) * a.lda;
    const int64_t b_span = (TB ? (int64_t)PN : (int64_t)(BKB / ES)) * a.ldb;
    const bool fits = a_span * ES < 0x7fff0000LL && b_span * ES < 0x7fff0000LL;
    const dim3 g((unsigned)tiles), blk(64 * WGM * WGN * KG);
    auto go = [&](auto dma) {
        constexpr bool D = decltype(dma)::value;
        if constexpr (MODE == kScaled) {
            if (a.batch != 1) {
                hipLaunchKernelGGL((k_ffn<DT, OD, MODE, SPLIT, TA, TB, BM, BN, WGM, WGN, KG, BKB, STAGES, PW, D, true>), g,
                                   blk, 0, s, slim_batch(a, SPLIT, false));
                return hipGetLastError();
            }
        }
        const FfnUse use = MODE == kGlu ? kUseGlu : MODE == kScaled ? kUseScaled : kUsePlain;
        hipLaunchKernelGGL((k_ffn<DT, OD, MODE, SPLIT, TA, TB, BM, BN, WGM, WGN, KG, BKB, STAGES, PW, D, false>), g, blk,
                           0, s, slim_args<FfnSlim>(a, use, SPLIT, false));
        return hipGetLastError();
    };
    if (vec && fits) return go(std::true_type());
    if constexpr (BM * BN < 256 * 256) return go(std::false_type());
    // The register-staged form would not fit the registers of this tile.
    return launch_ffn<DT, OD, MODE, SPLIT, TA, TB, 128, 128, 2, 2, 1, 64, 4, 4>(false, a, s);
}

// The entries of kFfnTiles for one kind of product.
template <int DT, int OD, int MODE, bool SPLIT, bool TA, bool TB>
static hipError_t launch_entry(int tile, bool vec, const FfnArgs &a, hipStream_t s) {
    switch (tile) {
    case 0:
        // FLOAT fills the matrix cores with smaller tiles, and partial sums
        // of 256 x 256 tiles are never wanted.
        if constexpr (DT != MM_FLOAT && !SPLIT) return launch_ffn<DT, OD, MODE, SPLIT, TA, TB, 256, 256, 2, 4, 1, 64, 4, 4>(vec, a, s);
        break;
    case 1: return launch_ffn<DT, OD, MODE, SPLIT, TA, TB, 128, 128, 2, 2, 1, 64, 4, 4>(vec, a, s);
    case 2: return launch_ffn<DT, OD, MODE, SPLIT, TA, TB, 64, 128, 2, 2, 2, 128, 3, 4>(vec, a, s);
    case 3:
        // A 32-row tile of a transposed 16-bit A has rows too short to stage.
        if constexpr (!TA || DT == MM_FLOAT) return launch_ffn<DT, OD, MODE, SPLIT, TA, TB, 32, 128, 1, 2, 4, 256, 3, 8>(vec, a, s);
        break;
    case 4:
        if constexpr (DT != MM_FLOAT) return launch_ffn<DT, OD, MODE, SPLIT, TA, TB, 256, 128, 4, 2, 1, 128, 3, 4>(vec, a, s);
        break;
    }
    return hipErrorInvalidValue;
}

}  // namespace mm
