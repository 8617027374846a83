// k_big.h -- large 16-bit products of the linear layer on tiles of 256 x 256 or
// 256 x 128: the forward pass with its epilogue and dX (A of K-contiguous rows),
// and dW (both operands as rows of one k).
//
// Four waves, one on each SIMD, hold 128 x 128 of the larger tile each: 256
// accumulator registers, and LDS reads of 256 bytes for every MFMA of 16 x 16 x 32,
// where eight waves of 128 x 64 need 384 for as many products.  One wave alone has to keep its matrix core fed, so
// the order of everything is written down: a half stage is 64 MFMAs of 32 k, and the
// reads of the next half's fragments and the loads of a later stage stand one
// between every two to four of them.  (In groups between groups of eight MFMAs they
// cost their own issue time: 8192 x 11008 x 4096 BF16 without an epilogue 611 us, so
// 540; the eight-wave kernel in k_ffn.h 650.)
//
// A stage is 64 k, two LDS buffers hold one each.  Midway through stage kt, when
// every wave holds the fragments of its second half, its buffer is free: a barrier,
// after which the loads of kt + 2 go there, most of them in the next 64 MFMAs,
// which leaves 1 to 1.5 stages for their way, and the fragments of kt + 1 are read,
// whose loads every wave has waited for before that barrier.  Tiles of 128 columns
// take half as long, so they have a third buffer and a stage more (8192 x 4096 x
// 11008 790 -> 595 us, 2048 x 4096 x 4096 63 -> 55).
//
// Rows of 64 k, 128 bytes, keep a load's 64 lanes on 8 rows; with rows half as
// long every load took longer to issue (595 us for 540).
//
// What bounds it: the matrix cores, 1.26 to 1.48 PFLOP/s from 8192 x 4096 x 10240
// on, where a product of 8192^3 reaches 1.55 at the clock that random operands
// leave.  A round of tiles of 256 x 256 takes 10 us and 21 ns for each k, one of 256 x
// 128 7 us and 12 ns; the 10 us are the first loads' way and the epilogue, during
// which a CU's one workgroup feeds no matrix core (8192 x 4096 x 10240, 475 us: tanh
// gelu 14 us more, a residual, whose 168 MB are read in bursts, 37, Z in 16 bits 20,
// as a checkpoint 30, in FP32 50).
#pragma once

#include <type_traits>

#include "activation.h"
#include "checkpoint.h"
#include "device.h"
#include "ffn.h"

namespace mm {

// 16-byte chunk swizzles of staged rows: K-contiguous ones (8 chunks) and rows of
// one k (32 or 16 chunks, read by four k x two chunks in each 16 lanes, lanes 16 apart
// eight k apart).
__device__ __forceinline__ int big_swizzle_k(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int big_swizzle_mn(int k) { return 2 * (k & 3) + 8 * ((k >> 3) & 1); }

// TA, TB as in k_ffn.h.  LINEAR: the linear layer's epilogue (kUseLinear arguments).
template <int DT, bool TA, bool TB, bool LINEAR, int BN>
__global__ __launch_bounds__(256, 1) void k_big(FfnSlim a) {
#if defined(__HIP_DEVICE_COMPILE__)
    using E = Elem<DT>;
    using S = typename E::S;
    constexpr int BM = 256, BK = 64, PANEL = BM * BK * 2, STAGE = PANEL + BN * BK * 2;
    constexpr int FN = BN / 32, NB = BN / 32, LOADS = 8 + NB;  // blocks of 16 columns a wave, loads of B, of both
    constexpr int NBUF = BN == 256 ? 2 : 3;
    __shared__ __attribute__((aligned(1024))) char lds[NBUF * STAGE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave >> 1, wc = wave & 1;
    const int r16 = lane & 15, kg = lane >> 4;

    const int64_t M = a.M, N = a.N, K = a.K;
    const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
    const int64_t id = xcd_remap(blockIdx.x, (int64_t)gridDim.x);
    // 8 tile rows sweep the tile columns together, so that they share B.
    constexpr int64_t GM = 8;
    const int64_t first_m = id / (GM * tiles_n) * GM;
    const int64_t gsize = tiles_m - first_m < GM ? tiles_m - first_m : GM;
    const int64_t m0 = (first_m + id % (GM * tiles_n) % gsize) * BM, n0 = id % (GM * tiles_n) / gsize * BN;
    const char *At = (const char *)((const S *)a.A[0] + (TA ? m0 : m0 * a.lda));
    const char *Bt = (const char *)((const S *)a.B[0] + (TB ? n0 * a.ldb : n0));
    const int nk = (int)((K + BK - 1) / BK);

    // ---- staging: 1 KB blocks wave * 8 + q, q < 8, of A's panel, wave * NB + q, q <
    // NB, of B's
    const uint32_t lds_base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char *)lds);
    // The chunk of a block that this lane loads: its row of the panel and place in
    // it; a row of one k has `width` elements.
    auto place = [&](bool mn, int width, int blk, int &row, int &c) {
        row = mn ? blk * (512 / width) + lane / (width / 8) : blk * 8 + lane / 8;
        c = mn ? (lane % (width / 8)) ^ big_swizzle_mn(row) : (lane % 8) ^ big_swizzle_k(row);
    };
    auto offset = [&](bool mn, int width, int blk, int64_t ld, int64_t left) {
        int row, c;
        place(mn, width, blk, row, c);
        return (mn ? c * 8 : row) < left ? (uint32_t)(row * ld * 2 + c * 16) : kOutOfRange;
    };
    uint32_t a_off[8], b_off[NB];
#pragma unroll
    for (int q = 0; q < 8; ++q) a_off[q] = offset(TA, BM, wave * 8 + q, a.lda, M - m0);
#pragma unroll
    for (int q = 0; q < NB; ++q) b_off[q] = offset(!TB, BN, wave * NB + q, a.ldb, N - n0);
    auto rsrc_a = [&](int st) { return buffer_rsrc(At + (int64_t)st * BK * 2 * (TA ? a.lda : 1)); };
    auto rsrc_b = [&](int st) { return buffer_rsrc(Bt + (int64_t)st * BK * 2 * (TB ? 1 : a.ldb)); };
    // Load q of a stage: A's blocks, then B's.  `rem`: k left in it.
    auto issue = [&](int buf, const i32x4 &ra, const i32x4 &rb, int q, int rem) {
        const bool is_a = q < 8, mn = is_a ? TA : !TB;
        const int blk = is_a ? wave * 8 + q : wave * NB + q - 8;
        uint32_t off = is_a ? a_off[q & 7] : b_off[(q - 8) & (NB - 1)];
        if (rem < BK) {
            int row, c;
            place(mn, is_a ? BM : BN, blk, row, c);
            if ((mn ? row : c * 8) >= rem) off = kOutOfRange;
        }
        load_to_lds16(is_a ? ra : rb, lds_base + buf * STAGE + (is_a ? 0 : PANEL) + blk * 1024, off);
    };
    auto issue_all = [&](int st) {  // into buffer st < NBUF
        const i32x4 ra = rsrc_a(st), rb = rsrc_b(st);
        const int rem = K - (int64_t)st * BK < BK ? (int)(K - (int64_t)st * BK) : BK;
#pragma unroll
        for (int q = 0; q < LOADS; ++q) issue(st, ra, rb, q, rem);
    };

    // ---- fragments: 16 bytes of consecutive k of row (column) base + lane % 16
    uint4 fa[2][8], fb[2][FN];
    f32x4 acc[8][FN];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
    // Half ks of panel P, fragment f of this wave's rows from `first`.  Rows 16
    // apart have one swizzle.  part: both (2), or half 0 or 1 of a transposing
    // read's result.
    auto read = [&](bool mn, int width, const char *P, int first, int ks, int f, int part, uint4 &v) {
        if (!mn) {
            const int row = first + r16;
            v = *(const uint4 *)(P + row * 128 + (((ks * 4 + kg) ^ big_swizzle_k(row)) * 16) + f * 2048);
            return;
        }
        const int k = ks * 32 + kg * 8 + part * 4 + (r16 >> 2), n = first + f * 16 + (r16 & 3) * 4;
        const char *at = P + k * (width * 2) + ((n >> 3) ^ big_swizzle_mn(k)) * 16 + ((n >> 2) & 1) * 8;
        const uint2 h = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                                                      (__attribute__((address_space(3))) bf16x4 *)(at)));
        if (part == 0) {
            v.x = h.x;
            v.y = h.y;
        } else {
            v.z = h.x;
            v.w = h.y;
        }
    };
    constexpr int VS = BN == 256 ? 4 : 3, EARLY = BN == 256 ? 14 : 10;  // from one load's slot to the next; before the half
    constexpr int RA = TA ? 16 : 8, RB = TB ? FN : 2 * FN, READS = RA + RB;
    // Read r < READS of a half's fragments, A's and B's in turn as far as both go.
    auto read_nth = [&](const char *X, int ks, int r, int slot) {
        constexpr int both = 2 * (RA < RB ? RA : RB);
        const bool is_a = r < both ? r % 2 == 0 : RA > RB;
        const int x = r < both ? r / 2 : r - both / 2;
        if (is_a) read(TA, BM, X, wr * 128, ks, TA ? x / 2 : x, TA ? x % 2 : 2, fa[slot][TA ? x / 2 : x]);
        else read(!TB, BN, X + PANEL, wc * (BN / 2), ks, TB ? x : x / 2, TB ? 2 : x % 2, fb[slot][TB ? x : x / 2]);
    };
    auto mfma = [&](int s, int i, int j) {
        if constexpr (DT == MM_BFLOAT16)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[s][j]),
                                                                __builtin_bit_cast(bf16x8, fa[s][i]), acc[i][j], 0, 0, 0);
        else
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, fb[s][j]),
                                                               __builtin_bit_cast(f16x8, fa[s][i]), acc[i][j], 0, 0, 0);
    };
    // The MFMAs of the fragments in slot `s`, the reads of the next half (ks_next of
    // stage buffer X) into the other slot, and loads.
    auto half = [&](auto s_t, auto reads_t, const char *X, int ks_next, auto load) {
        constexpr int s = decltype(s_t)::value;
        constexpr int DSP = READS * 5 / 2 <= 8 * FN ? 2 : 1;  // slots from one read to the next
#pragma unroll
        for (int n = 0; n < 8 * FN; ++n) {
            if (decltype(reads_t)::value && n % DSP == 0 && n / DSP < READS) read_nth(X, ks_next, n / DSP, s ^ 1);
            if (n % VS == 1) load(n / VS);
            __builtin_amdgcn_sched_barrier(0);
            mfma(s, n / FN, n % FN);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using Yes = std::true_type;
    using No = std::false_type;
    auto nothing = [](int) {};
    if (nk > 0) {
        issue_all(0);
        if (nk > 1) issue_all(1);
        if (NBUF > 2 && nk > 2) issue_all(2);
        if (nk >= NBUF) wait_vmcnt<(NBUF - 1) * LOADS>();
        else wait_vmcnt<0>();
        asm volatile("s_barrier" ::: "memory");
#pragma unroll
        for (int r = 0; r < READS; ++r) read_nth(lds, 0, r, 0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        half(S0(), Yes(), lds, 1, nothing);
        // Second half of stage kt and first half of kt + 1, while kt + NBUF is
        // asked for: most of its loads in the first half, the others behind them.
        int kt = 0, buf = 0;  // (a stage and its buffer)
        auto stage = [&](auto more_t, int rem) {
            constexpr bool more = decltype(more_t)::value;
            const int next = buf + 1 == NBUF ? 0 : buf + 1;
            const char *X = lds + next * STAGE;
            const i32x4 ra = rsrc_a(kt + NBUF), rb = rsrc_b(kt + NBUF);
            // kt + 1 has come; in between lie the stages up to kt + NBUF - 1.
            wait_vmcnt<more ? (NBUF - 2) * LOADS : 0>();
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            half(S1(), Yes(), X, 0, [&](int q) {
                if (more && q < EARLY) issue(buf, ra, rb, q, rem);
            });
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            half(S0(), Yes(), X, 1, [&](int q) {
                if (more && q < LOADS - EARLY) issue(buf, ra, rb, EARLY + q, rem);
            });
            buf = next;
            ++kt;
        };
        while (kt + NBUF + 1 < nk) stage(Yes(), BK);
        if (kt + NBUF < nk) stage(Yes(), (int)(K - (int64_t)(kt + NBUF) * BK));  // asks for the last one
        while (kt + 1 < nk) stage(No(), BK);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        half(S1(), No(), lds, 0, nothing);
    }
    // Every wave's reads and loads of the last stages have ended: LDS is free.
    wait_vmcnt<0>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

    // ---- epilogue.  Element e of block (i, j) is row wr 128 + 16 i + lane % 16,
    // column wc BN / 2 + 16 j + 4 (lane / 16) + e.  The sums go through LDS in FP32, half
    // of each wave's rows at a time, and come back as eight columns of a row, from
    // which everything is formed and written in whole 16-byte chunks; four threads
    // hold a checkpoint block of Z.  (In the registers where the matrix cores leave
    // them there is room for nothing beside them.)  Chunk c of 16 bytes of a row r
    // lies at (c / 2 + BN / 8 (c % 2)) ^ (r % 16): neither side meets a bank twice.
    typedef uint32_t U4 __attribute__((ext_vector_type(4)));
    typedef uint32_t U2 __attribute__((ext_vector_type(2)));
    constexpr int CT = BN / 8, RT = 256 / CT;     // threads a row, rows at a time
    constexpr int GR = 4, STEPS = 128 / (GR * RT);  // rows a thread works on at a time, such steps for half the rows
    const int c8 = tid % CT;
    const int64_t col = n0 + c8 * 8;
    const int in = N - col >= 8 ? 8 : N > col ? (int)(N - col) : 0;
    // 8 columns of `size` bytes each, their words in w.
    auto put8 = [&](void *out, int size, int64_t row, bool vec, const uint32_t *w) {
        char *dst = (char *)out + (row * a.ldy + col) * size;
        if (vec && in == 8) {
            if (size == 1) {
                U2 v = {w[0], w[1]};
                __builtin_nontemporal_store(v, (U2 *)dst);
            } else {
#pragma unroll
                for (int h = 0; h < size / 2; ++h) {
                    U4 v = {w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]};
                    // (halves of 32 bytes meet in the cache)
                    if (size == 4) *((U4 *)dst + h) = v;
                    else __builtin_nontemporal_store(v, (U4 *)dst + h);
                }
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < in) {
                if (size == 4) __builtin_memcpy(dst + 4 * e, &w[e], 4);
                else if (size == 2) *(uint16_t *)(dst + 2 * e) = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
                else *(uint8_t *)(dst + e) = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
            }
    };
    float bias[8];
    if constexpr (LINEAR) {
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = a.lin_bias() && e < in ? E::to_f32(((const S *)a.lin_bias())[col + e]) : 0.0f;
    }
    // Step g: local row of a thread's x-th, and that row of the tile.
    auto local = [&](int g, int x) { return (g % STEPS * GR + x) * RT + tid / CT; };
    auto row_of = [&](int g, int x) {
        const int rl = local(g, x);
        return m0 + (rl >> 6) * 128 + g / STEPS * 64 + (rl & 63);
    };
    // The next step's residuals are on their way while a step's values are formed.
    uint4 rv[GR];
    auto ask = [&](int g) {
#pragma unroll
        for (int x = 0; x < GR; ++x) {
            const int64_t row = row_of(g, x);
            rv[x] = make_uint4(0, 0, 0, 0);
            if (row >= M || in == 0) continue;
            const S *r = (const S *)a.R() + row * a.ldy + col;
            if (a.r_vec() && in == 8) {
                rv[x] = *(const uint4 *)r;
            } else {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = e < in ? r[e] : 0;
                rv[x] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
        }
    };
    if constexpr (LINEAR) {
        if (a.R()) ask(0);
    }
    char *const put_at = lds + (wr * 64 + r16) * (BN * 4);
    auto put_half = [&](auto first_t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                *(f32x4 *)(put_at + i * (BN * 64) + (((wc * (CT / 2) + 2 * j + (kg >> 1) + CT * (kg & 1)) ^ r16) * 16)) =
                    acc[decltype(first_t)::value + i][j];
    };
#pragma unroll 1
    for (int g = 0; g < 2 * STEPS; ++g) {
        if (g == 0) {
            put_half(std::integral_constant<int, 0>());
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        } else if (g == STEPS) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            put_half(std::integral_constant<int, 4>());
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        float v[GR][8];
        uint4 r[GR];
#pragma unroll
        for (int x = 0; x < GR; ++x) {
            const int rl = local(g, x);
            const char *at = lds + rl * (BN * 4) + ((c8 ^ (rl & 15)) * 16);
            const f32x4 lo = *(const f32x4 *)at, hi = *(const f32x4 *)(at + BN * 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[x][e] = lo[e];
                v[x][4 + e] = hi[e];
            }
        }
        if constexpr (LINEAR) {
            auto each = [&](auto f) {
#pragma unroll
                for (int x = 0; x < GR; ++x)
#pragma unroll
                    for (int e = 0; e < 8; ++e) f(v[x][e], e);
            };
#pragma unroll
            for (int x = 0; x < GR; ++x) r[x] = rv[x];
            if (a.R() && g + 1 < 2 * STEPS) ask(g + 1);
            each([&](float &z, int e) { z += bias[e]; });
            if (a.G() && a.q8()) {
                // Columns past the last hold 0, or NaN where the whole row is NaN or
                // infinite: neither changes a block.
                uint32_t ex[GR], w[GR][2];
#pragma unroll
                for (int x = 0; x < GR; ++x) {
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = max(top, ck_magnitude(v[x][e]));
                    ex[x] = ck_exponent(block_top<8>(top));
                    const float inv = ck_inverse(ex[x]);
                    w[x][0] = ck_word(v[x][0], v[x][1], v[x][2], v[x][3], inv);
                    w[x][1] = ck_word(v[x][4], v[x][5], v[x][6], v[x][7], inv);
                }
#pragma unroll
                for (int x = 0; x < GR; ++x) {
                    const int64_t row = row_of(g, x);
                    if (row >= M || in == 0) continue;
                    if ((c8 & 3) == 0) ((uint8_t *)a.zs())[row * ((a.ldy + 31) / 32) + col / 32] = (uint8_t)ex[x];
                    put8(a.G(), 1, row, a.kept_vec(), w[x]);
                }
            } else if (a.G()) {
#pragma unroll
                for (int x = 0; x < GR; ++x) {
                    const int64_t row = row_of(g, x);
                    if (row >= M || in == 0) continue;
                    uint32_t w[8];
                    if (a.kept32()) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[x][e]);
                        put8(a.G(), 4, row, a.kept_vec(), w);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = E::pack2(v[x][2 * e], v[x][2 * e + 1]);
                        put8(a.G(), 2, row, a.kept_vec(), w);
                    }
                }
            }
            auto apply = [&](auto kind) {
                each([&](float &z, int) { z = act_only<decltype(kind)::value, false>(z); });
            };
            switch (a.act) {
            case MM_ACT_SILU: apply(std::integral_constant<int, MM_ACT_SILU>()); break;
            case MM_ACT_GELU: apply(std::integral_constant<int, MM_ACT_GELU>()); break;
            case MM_ACT_GELU_TANH: apply(std::integral_constant<int, MM_ACT_GELU_TANH>()); break;
            case MM_ACT_RELU: apply(std::integral_constant<int, MM_ACT_RELU>()); break;
            case MM_ACT_SIGMOID: apply(std::integral_constant<int, MM_ACT_SIGMOID>()); break;
            }
            if (a.R()) {
#pragma unroll
                for (int x = 0; x < GR; ++x) {
                    const uint32_t w[4] = {r[x].x, r[x].y, r[x].z, r[x].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[x][e] += E::to_f32((S)(w[e / 2] >> (16 * (e % 2))));
                }
            }
        }
#pragma unroll
        for (int x = 0; x < GR; ++x) {
            const int64_t row = row_of(g, x);
            if (row >= M || in == 0) continue;
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = E::pack2(v[x][2 * e], v[x][2 * e + 1]);
            put8(a.Y[0], 2, row, a.y_vec(), w);
        }
    }
#endif
}

template <int DT, bool TA, bool TB, bool LINEAR, int BN>
static hipError_t launch_big(const FfnArgs &a, hipStream_t s) {
    const int64_t tiles = (a.M + 255) / 256 * ((a.N + BN - 1) / BN);
    if (tiles <= 0) return hipSuccess;
    if (tiles > 0xffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_big<DT, TA, TB, LINEAR, BN>), dim3((unsigned)tiles), dim3(256), 0, s,
                       slim_args<FfnSlim>(a, LINEAR ? kUseLinear : kUsePlain, false, false));
    return hipGetLastError();
}

// Whether the kernel takes a product (entries 0 and 4, whole K): buffer offsets are
// 32-bit, and operand rows whole, aligned 16-byte chunks (`vec`).
inline bool big_fits(bool ta, bool tb, int tile, bool split, bool vec, const FfnArgs &a) {
    if ((tile != 0 && tile != 4) || split) return false;
    const int64_t span_a = (ta ? 64 : 256) * a.lda * 2, span_b = (tb ? 256 : 64) * a.ldb * 2;
    return vec && span_a < 0x7fff0000LL && span_b < 0x7fff0000LL;
}

}  // namespace mm
