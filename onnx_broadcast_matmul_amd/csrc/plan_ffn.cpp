// plan_ffn.cpp -- plans and executions of the feed-forward operators: the
// scaled INT8 product, row quantization and the gated block.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "ffn_choice.h"

namespace mm {

// Time model of the tiled products: a CU runs up to kOcc workgroups of an
// entry together, and a round of o workgroups per CU takes kFixed + kStep[o - 1]
// for each 32 bytes of K.  Measured with forced entries on grids of 256 and
// 512 workgroups, 1 and 8 KiB of K, over the forward, dX, dW and INT8 kinds,
// which lie within 10 % of each other; rows that are not 16-byte aligned run
// the register-staged form (entry 0 has none and runs entry 1's).
static const int kOcc[kNumFfnTiles] = {1, 2, 2, 1, 1};
static const double kLaunch = 2.5;                                      // us
static const double kFixed[kNumFfnTiles] = {7.5, 3.2, 2.5, 1.4, 5.5};  // us
static const double kFixedLinear[kNumFfnTiles] = {10.0, 3.2, 2.5, 1.4, 7.0};
static const double kStep[2][4][kNumFfnTiles][2] = {                    // us: aligned, not aligned
    {{{0.41, 0}, {0.17, 0.285}, {0.147, 0.165}, {0.095, 0}, {0.240, 0}},
     {{0.41, 0}, {0.17, 0.285}, {0.145, 0.160}, {0.095, 0}, {0.222, 0}},
     {{1e9, 0}, {0.54, 0.970}, {0.260, 0.490}, {0.148, 0}, {1e9, 0}},
     {{0.335, 0}, {0.17, 0.285}, {0.147, 0.165}, {0.095, 0}, {0.190, 0}}},
    {{{1e9, 0}, {0.27, 0.345}, {0.200, 0.222}, {0.098, 0}, {0.345, 0}},
     {{1e9, 0}, {0.23, 0.305}, {0.122, 0.182}, {0.080, 0}, {0.310, 0}},
     {{1e9, 0}, {0.60, 1.050}, {0.355, 0.585}, {0.171, 0}, {1e9, 0}},
     {{1e9, 0}, {0.27, 0.345}, {0.200, 0.222}, {0.098, 0}, {0.345, 0}}}};

int type_class(int dtype) { return dtype == MM_FLOAT ? kClass32 : dtype == MM_INT8 ? kClass8 : kClass16; }

static double est_us(int cls, bool aligned, int tile, double wgs, double steps) {
    const double *step = kStep[aligned ? 0 : 1][cls][tile];
    const int occ = kOcc[tile];
    const double per_cu = ceil(wgs / kNumCUs), fixed = (cls == kClassLinear16 && aligned ? kFixedLinear : kFixed)[tile];
    const double full = floor(per_cu / occ), rest = per_cu - full * occ;
    double us = kLaunch + full * (fixed + step[occ - 1] * steps);
    if (rest > 0) us += fixed + step[(int)rest - 1] * steps;
    return us;
}

// Time of the few-row kernel: a workgroup's chain of K (kChain us for each KiB
// of a weight row, which memory latency sets), or the weights' stream at kRate
// TB/s once the workgroups fill the GPU; each [up to 16 rows, more].  Fitted to
// M = 1..32, K = 500..11008, N = 128..11008, weights that come from memory.
// [K, N] weights: by how often rows_halve halves a workgroup's columns.  The
// gated block's workgroups of 32 columns take as long again where a CU has
// two, those of 16 longer the more of them share the cache lines.  Rows (of
// `row` bytes) off 4-byte alignment cost 16-bit types more.
double rows_us(int cls, bool nk, int64_t M, int64_t N, int64_t kbytes, int64_t row, double wbytes) {
    static const double kChain[3][2] = {{1.0, 1.75}, {0.6, 1.2}, {1.2, 1.85}}, kRate[3][2] = {{4.9, 3.2}, {3.5, 2.2}, {4.9, 3.2}};
    static const double kChain8[3][2] = {{2.0, 2.45}, {1.5, 2.0}, {1.35, 1.75}}, kRate8[3][2] = {{5.0, 4.4}, {4.5, 4.0}, {3.5, 3.0}};
    const int r = M > 16 ? 1 : 0;
    const double kib = (double)kbytes / 1024.0;
    const bool odd = cls == kClass16 && row % 4 != 0;
    if (nk) return std::max(3.0 + kChain[cls][r] * kib, wbytes / (kRate[cls][r] * (odd ? 0.5 : 1.0) * 1e6));
    const bool i8 = cls == kClass8;
    int h = 0;
    int64_t cols = i8 ? 64 : 32;
    for (; h < (i8 ? 2 : 1) && rows_halve(cdiv(N, cols)); cols /= 2) ++h;
    if (i8) return 3.0 + std::max(kChain8[h][r] * kib, wbytes / (kRate8[h][r] * 1e6));
    const double wgs = (double)cdiv(N, cols);
    const double chain = h ? (r ? 1.3 + 0.0085 * wgs : 1.2 + 0.0075 * wgs) : (r ? 3.5 : 2.8) * ceil(wgs / kNumCUs);
    return 3.0 + chain * kib * (odd ? 1.25 : 1.0);
}

// The linear layer's few-row kernel reads one matrix where the gated block's reads
// two.  Fitted to M = 1..32, K = 512..11008, N = 512..11008: within 15 % but for
// FP32 ones that leave a third of the CUs without work.
double linear_rows_us(int cls, bool nk, int64_t M, int64_t N, int64_t kbytes, int64_t row, double wbytes) {
    const bool f32 = cls == kClass32;
    const int r = M > 16 ? 1 : 0;
    const double kib = (double)kbytes / 1024.0;
    if (nk) {
        static const double kChain[2][2] = {{0.75, 1.15}, {0.8, 1.25}}, kRate[2][2] = {{4.0, 2.8}, {4.1, 2.7}};
        const bool odd = !f32 && row % 4 != 0;
        return std::max(3.0 + kChain[f32][r] * kib, wbytes / (kRate[f32][r] * (odd ? 0.5 : 1.0) * 1e6));
    }
    // [K, N]: us for each KiB of a column, from the workgroups there are, of 32 or
    // of half as many columns.
    const double wgs = (double)cdiv(N, 32), rounds = ceil(wgs / kNumCUs);
    if (rows_halve(cdiv(N, 32))) {
        static const double kBase[2][2] = {{0.65, 1.2}, {0.8, 1.35}}, kEach[2][2] = {{0.0035, 0.003}, {0.0025, 0.0013}};
        return 3.0 + (kBase[f32][r] + kEach[f32][r] * 2.0 * wgs) * kib;
    }
    static const double kBase[2][2] = {{1.0, 1.6}, {-0.6, 1.15}}, kEach[2][2] = {{0.8, 0.65}, {2.45, 1.05}};
    return 3.0 + (kBase[f32][r] + kEach[f32][r] * rounds) * kib;
}

// The tiles' time over the same few rows: the weights stream at kStream
// TB/s at best ([K, N] ones at 0.72 of it in the register-staged form, at half
// with rows off 4-byte alignment), and a second launch follows a split.
double tiles_us(int cls, const FfnChoice &c, bool nk, bool aligned, int64_t row, double wbytes) {
    static const double kStream[4] = {4.0, 2.7, 4.0, 4.0};
    const double part = aligned || nk ? 1.0 : row % 4 == 0 ? 0.72 : 0.5;
    return std::max(c.us + (c.split > 1 ? 3.0 : 0.0), wbytes / (kStream[cls] * part * 1e6));
}

// Entry and split with the least estimated time for `batch` products of
// [M, cols] over `kbytes` bytes of K (terms: that many times in one K loop;
// cols counts gate and up columns).  Partials cost their write, read and a
// launch.
FfnChoice choose(int cls, bool aligned, int64_t batch, int64_t M, int64_t cols, int64_t kbytes, int terms,
                        unsigned tiles, bool may_split) {
    FfnChoice best;
    double top = 1e30;
    for (int i = 0; i < kNumFfnTiles; ++i) {
        if (!(tiles >> i & 1)) continue;
        const FfnTile &t = kFfnTiles[i];
        const int64_t wgs = batch * cdiv(M, t.bm) * cdiv(cols, t.bn), stages = terms * cdiv(kbytes, t.bkb);
        int64_t most = 1;
        if (may_split && i > 0)
            most = std::max<int64_t>(1, std::min(stages * t.bkb / 512, 2 * kNumCUs / std::max<int64_t>(wgs, 1)));
        for (int64_t sp = 1; sp <= most; ++sp) {
            const int64_t per = std::max<int64_t>(1, cdiv(stages, sp)), parts = std::max<int64_t>(1, cdiv(stages, per));
            if (parts != sp) continue;
            double us = est_us(cls, aligned, i, (double)(wgs * parts), (double)(per * t.bkb / 32));
            if (parts > 1) us += 3.0 + (double)parts * (double)batch * (double)M * (double)cols * 8.0 / 3.5e6;
            if (us < top) {
                top = us;
                best.us = us;
                best.tile = i;
                best.split = (int32_t)parts;
                best.kstages = (int32_t)per;
            }
        }
    }
    return best;
}

int64_t balance(int cls, FfnChoice *c, int64_t M, int64_t N, int64_t kbytes, unsigned tiles, int *rest) {
    if (M <= 0 || N <= 0) return 0;
    const double steps = ceil((double)kbytes / 32.0);
    int64_t best = 0;
    FfnChoice main = *c;
    double top = 0.98 * c->us;  // (a second launch has to bring something)
    for (int i = 0; i < kNumFfnTiles; ++i) {
        if (!(tiles >> i & 1)) continue;
        const FfnTile &t = kFfnTiles[i];
        const int64_t slots = (int64_t)kNumCUs * kOcc[i], rows = cdiv(M, t.bm), total = rows * cdiv(N, t.bn);
        if (total > 64 * slots) continue;  // a round less would bring under 2 %
        const int64_t cols = total / slots * slots / rows;  // columns of tiles in whole rounds
        if (cols <= 0 || cols * t.bn >= N) continue;
        const double us = est_us(cls, true, i, (double)(rows * cols), steps);
        const FfnChoice r = choose(cls, true, 1, M, N - cols * t.bn, kbytes, 1, tiles, false);
        if (us + r.us >= top) continue;
        top = us + r.us;
        best = cols * t.bn;
        *rest = r.tile;
        main = *c;
        main.tile = i;
        main.us = top;
    }
    *c = main;
    return best;
}

// A requested number of partitions for an entry, as whole stages.
void set_split(FfnChoice *c, int64_t kbytes, int terms, int64_t split) {
    const int64_t stages = std::max<int64_t>(1, terms * cdiv(kbytes, kFfnTiles[c->tile].bkb));
    const int64_t per = cdiv(stages, std::max<int64_t>(1, std::min<int64_t>({split, stages, 4096})));
    c->kstages = (int32_t)per;
    c->split = (int32_t)cdiv(stages, per);
}

mm_status tile_option(const mm_plan_options *opt, int *tile) {
    const int req = opt ? opt->tile : 0;
    if (req == 0) return MM_OK;
    if (req < 0 || req > kNumFfnTiles)
        return fail(MM_ERR_BAD_OPTION, "tile %d out of range 1..%d", req, kNumFfnTiles);
    *tile = req - 1;
    return MM_OK;
}

// A backward product's entry and split: the requested ones, the time model's
// where they are 0.
mm_status choose_backward(const char *name, int cls, bool aligned, int64_t batch, int64_t M, int64_t cols,
                                 int64_t kbytes, int terms, unsigned tiles, int treq, int sreq, FfnChoice *c) {
    if (treq < 0 || treq > kNumFfnTiles)
        return fail(MM_ERR_BAD_OPTION, "%s tile %d out of range 1..%d", name, treq, kNumFfnTiles);
    if (sreq < 0) return fail(MM_ERR_BAD_OPTION, "%s split_k %d is negative", name, sreq);
    if (treq > 0) tiles &= 1u << (treq - 1);
    if (!tiles) return fail(MM_ERR_BAD_OPTION, "%s has no kernel of tile %d in this type", name, treq);
    if (sreq > 1) tiles &= ~1u;  // no 256 x 256 partials
    if (!tiles) return fail(MM_ERR_BAD_OPTION, "tile 1 does not split K");
    *c = choose(cls, aligned, batch, M, cols, kbytes, terms, tiles, sreq == 0);
    if (sreq > 0) set_split(c, kbytes, terms, sreq);
    return MM_OK;
}

// Options that a forced algorithm would drop: partitions of the unsplit ones,
// a tile entry of the few-row kernel.
mm_status forced_alone(const mm_plan_options *opt) {
    if (!opt) return MM_OK;
    const bool rows = opt->force_algo == MM_ALGO_SKINNY_M;
    if ((rows || opt->force_algo == MM_ALGO_GENERAL) && opt->split_k > 1)
        return fail(MM_ERR_BAD_OPTION, "%s does not split K (split_k %d)", rows ? "SKINNY_M" : "GENERAL", opt->split_k);
    if (rows && opt->tile != 0) return fail(MM_ERR_BAD_OPTION, "SKINNY_M has no tiles (tile %d)", opt->tile);
    return MM_OK;
}

// Algorithm, tile and split of a scaled product whose output is not empty.
static mm_status select_scaled(mm_plan_s *p, const mm_plan_options *opt) {
    const int64_t M = p->kernel_m, N = p->N, K = p->K;
    const int force = opt ? opt->force_algo : MM_ALGO_AUTO;
    const int sreq = opt ? opt->split_k : 0, treq = opt ? opt->tile : 0;
    if (sreq < 0) return fail(MM_ERR_BAD_OPTION, "split_k %d is negative", sreq);
    if (force != MM_ALGO_AUTO && force != MM_ALGO_SKINNY_M && force != MM_ALGO_GENERAL && force != MM_ALGO_SPLIT_K)
        return fail(MM_ERR_BAD_OPTION, "the scaled INT8 product runs on the skinny-M, general and split-K kernels only");
    const bool rows_ok = p->batch == 1 && M <= kFfnRows;
    if (force == MM_ALGO_SKINNY_M && !rows_ok)
        return fail(MM_ERR_BAD_OPTION, "SKINNY_M takes one product of at most %d rows", kFfnRows);
    int only = -1;
    mm_status st = tile_option(opt, &only);
    if (st == MM_OK) st = forced_alone(opt);
    if (st != MM_OK) return st;
    // Partials are added by a grid of at most 65535 products.
    if (p->batch > 65535 && K > 0 && (force == MM_ALGO_SPLIT_K || sreq > 1))
        return fail(MM_ERR_BAD_OPTION, "split K takes at most 65535 products (got %lld)", (long long)p->batch);
    const bool may_split = force != MM_ALGO_GENERAL && K > 0 && p->batch <= 65535;
    const unsigned all = (1u << kNumFfnTiles) - 1;
    unsigned tiles = only >= 0 ? 1u << only : all;
    if (force == MM_ALGO_SPLIT_K || sreq > 1) tiles &= ~1u;  // no 256 x 256 partials
    if (!tiles) return fail(MM_ERR_BAD_OPTION, "tile 1 does not split K");
    const bool aligned = (p->tb ? K : N) % 16 == 0 && (p->a_type != MM_INT8 || K % 16 == 0);
    FfnChoice c = choose(kClass8, aligned, p->batch, M, N, K, 1, tiles, may_split && sreq == 0);
    const double wbytes = (double)K * (double)N;
    // The few-row kernel may save the quantization's own launch.
    const double saved = p->a_type != MM_INT8 && rows_quantize(p->a_type, p->dtype, p->tb != 0, M, K, N) ? 2.5 : 0.0;
    if (force == MM_ALGO_SKINNY_M ||
        (force == MM_ALGO_AUTO && rows_ok && K > 0 && treq == 0 && sreq == 0 &&
         rows_us(kClass8, p->tb != 0, M, N, K, p->tb ? K : N, wbytes) <=
             tiles_us(kClass8, c, p->tb != 0, aligned, p->tb ? K : N, wbytes) + saved)) {
        p->algo = MM_ALGO_SKINNY_M;
        if (!launchable((double)cdiv(N, 16), 512)) return fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
        return MM_OK;
    }
    if (may_split && sreq > 0) set_split(&c, K, 1, sreq);
    p->tile = c.tile;
    p->algo = c.split > 1 || (force == MM_ALGO_SPLIT_K && may_split) ? MM_ALGO_SPLIT_K : MM_ALGO_GENERAL;
    if (p->algo == MM_ALGO_SPLIT_K) {
        p->split = c.split;
        p->kstages = c.kstages;
        p->kchunk = (int64_t)c.kstages * kFfnTiles[c.tile].bkb;
        p->workspace_bytes = round_up((int64_t)p->split * p->batch * M * N * 4, 256);
    }
    if (!tile_launchable(c, p->batch, M, N) || (p->algo == MM_ALGO_SPLIT_K && !pieces_launchable(M, cdiv(N, 4))))
        return fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
    return MM_OK;
}

}  // namespace mm

using namespace mm;

extern "C" {

mm_status mm_scaled_int_plan_create(const int64_t *a_shape, int a_rank, const int64_t *b_shape, int b_rank,
                                    const mm_scaled_int_desc *d, const mm_plan_options *opt, mm_plan_t *out) {
    clear_error();
    if (!out) return fail(MM_ERR_NULL_ARG, "out is NULL");
    *out = nullptr;
    if (!d) return fail(MM_ERR_NULL_ARG, "descriptor is NULL");
    if ((!a_shape && a_rank > 0) || (!b_shape && b_rank > 0)) return fail(MM_ERR_NULL_ARG, "shape pointer is NULL");
    if (d->a_type != MM_INT8 && !float_type(d->a_type))
        return fail(MM_ERR_DTYPE, "A is INT8, or FLOAT, FLOAT16 or BFLOAT16 to be quantized (got %d)", d->a_type);
    if (!float_type(d->out_type))
        return fail(MM_ERR_DTYPE, "the output is FLOAT, FLOAT16 or BFLOAT16 (got %d)", d->out_type);
    if (d->reserved != 0 || (opt && opt->reserved != 0)) return fail(MM_ERR_BAD_OPTION, "reserved field must be 0");
    if ((d->trans_b != 0 && d->trans_b != 1) || (d->has_bias != 0 && d->has_bias != 1))
        return fail(MM_ERR_BAD_OPTION, "trans_b and has_bias must be 0 or 1");
    if (d->trans_b && b_rank == 1) return fail(MM_ERR_BAD_OPTION, "trans_b needs a B of rank two or more");
    int64_t bs[MM_MAX_RANK] = {};
    if (b_rank >= 1 && b_rank <= MM_MAX_RANK) {
        for (int i = 0; i < b_rank; ++i) bs[i] = b_shape[i];
        if (d->trans_b) std::swap(bs[b_rank - 1], bs[b_rank - 2]);
    }
    mm_plan_s *p = new (std::nothrow) mm_plan_s();
    if (!p) return fail(MM_ERR_ALLOC, "host allocation failed");
    p->dtype = d->out_type;
    p->is_scaled = true;
    p->a_type = d->a_type;
    p->b_type = MM_INT8;
    p->tb = d->trans_b;
    p->has_bias = d->has_bias != 0;
    mm_status st = resolve(a_shape, a_rank, bs, b_rank, p);
    if (st == MM_OK) st = check_limits(p);
    if (st == MM_OK && p->K > 131071)
        st = fail(MM_ERR_TOO_LARGE, "K = %lld: INT32 sums hold at most 131071 INT8 products", (long long)p->K);
    if (st == MM_OK) {
        double a_rows = 1.0;
        for (int i = 0; i + 1 < a_rank; ++i) a_rows *= (double)a_shape[i];
        if (a_rows > INT32_MAX || too_large(p->batch * p->kernel_m, p->N) || too_large(p->K, p->N) ||
            a_rows * (double)p->K > 1099511627776.0 || p->kernel_m > kMaxSize || p->N > kMaxSize)
            st = fail(MM_ERR_TOO_LARGE, "a matrix of more than 2^40 elements, or a size of 2^31 - 64 or more");
    }
    if (st == MM_OK && p->out_numel == 0) {
        p->algo = MM_ALGO_EMPTY;
    } else if (st == MM_OK) {
        st = select_scaled(p, opt);
        p->fused_quant = p->a_type != MM_INT8 && p->algo == MM_ALGO_SKINNY_M &&
                         rows_quantize(p->a_type, p->dtype, p->tb != 0, p->kernel_m, p->K, p->N);
        if (st == MM_OK && p->a_type != MM_INT8 && !p->fused_quant) {
            p->a_rows = 1;
            for (int i = 0; i + 1 < a_rank; ++i) p->a_rows *= a_shape[i];
            p->q_pitch = round_up(p->K, 16);
            p->q_off = p->workspace_bytes;
            p->qs_off = p->q_off + round_up(p->a_rows * p->q_pitch, 256);
            p->workspace_bytes = p->qs_off + round_up(p->a_rows * 4, 256);
            // The batch strides of A count elements of its dense rows.
            if (p->K > 0)
                for (int i = 0; i < p->bd.nb; ++i) p->bd.sa[i] = p->bd.sa[i] / p->K * p->q_pitch;
        }
    }
    if (st == MM_OK) st = alloc_workspace(p, true);
    if (st != MM_OK) {
        delete p;
        return st;
    }
    *out = p;
    return MM_OK;
}

mm_status mm_quantize_rows(const void *X, int dtype, int64_t rows, int64_t cols, void *Q, float *scale, void *stream) {
    clear_error();
    if (rows < 0 || cols < 0) return fail(MM_ERR_NEG_DIM, "rows and cols must not be negative");
    if (!float_type(dtype)) return fail(MM_ERR_DTYPE, "quantize_rows takes FLOAT, FLOAT16 or BFLOAT16 (got %d)", dtype);
    if (rows > INT32_MAX || cols > INT32_MAX || too_large(rows, cols))
        return fail(MM_ERR_TOO_LARGE, "rows and cols must each be below 2^31, their product at most 2^40");
    if (rows == 0) return MM_OK;
    if (!scale || (cols > 0 && (!X || !Q))) return fail(MM_ERR_NULL_ARG, "X, Q or scale is NULL");
    return launched(launch_quantize_rows(dtype, X, rows, cols, Q, cols, scale, (hipStream_t)stream));
}

mm_status mm_scaled_int_execute(mm_plan_t p, const void *A, const void *B, const float *a_scale, const float *b_scale,
                                const void *bias, void *Y, void *stream) {
    clear_error();
    if (!p) return fail(MM_ERR_NULL_ARG, "plan is NULL");
    if (!p->is_scaled) return fail(MM_ERR_BAD_OPTION, "not a scaled INT8 plan");
    if (p->algo == MM_ALGO_EMPTY) return MM_OK;
    const bool quant = p->a_type != MM_INT8, pass = quant && !p->fused_quant;
    if (!Y) return fail(MM_ERR_NULL_ARG, "Y is NULL for a non-empty output");
    if (p->K > 0 && (!A || !B)) return fail(MM_ERR_NULL_ARG, "A or B is NULL");
    if (!b_scale || (!quant && !a_scale)) return fail(MM_ERR_NULL_ARG, "a scale is NULL");
    if (quant && a_scale) return fail(MM_ERR_BAD_OPTION, "the plan quantizes A itself: a_scale must be NULL");
    if (p->has_bias && !bias) return fail(MM_ERR_NULL_ARG, "the plan has a bias but bias is NULL");
    if (!p->has_bias && bias) return fail(MM_ERR_BAD_OPTION, "the plan has no bias");
    hipStream_t s = (hipStream_t)stream;
    if (p->workspace_bytes > 0) {
        mm_status st = alloc_workspace(p, false);
        if (st != MM_OK) return st;
    }
    char *ws = (char *)p->ws;
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.A[0] = pass ? ws + p->q_off : A;
    a.B[0] = B;
    a.Y[0] = Y;
    a.M = p->kernel_m;
    a.N = p->N;
    a.K = p->K;
    a.lda = std::max<int64_t>(pass ? p->q_pitch : p->K, 1);
    a.ldb = p->tb ? p->K : p->N;
    a.ldy = p->N;
    a.batch = p->batch;
    a.y_vec = aligned16(Y) && (p->N * elem_size(p->dtype)) % 16 == 0;
    a.sa = pass ? (const float *)(ws + p->qs_off) : a_scale;
    a.sb = b_scale;
    a.bias = bias;
    a.kstages = p->kstages;
    a.split = p->split;
    a.bd = p->bd;
    if (pass) {
        mm_status st = launched(launch_quantize_rows(p->a_type, A, p->a_rows, p->K, ws + p->q_off, p->q_pitch,
                                                     (float *)(ws + p->qs_off), s));
        if (st != MM_OK) return st;
    }
    if (p->algo == MM_ALGO_SKINNY_M) return launched(launch_scaled_rows(p->dtype, p->tb != 0, p->fused_quant, a, s));
    const bool vec = aligned16(a.A[0]) && a.lda % 16 == 0 && aligned16(B) && a.ldb % 16 == 0;
    if (p->algo == MM_ALGO_SPLIT_K) {
        a.W = ws;
        hipError_t e = launch_scaled_split(p->tb != 0, p->tile, vec, a, s);
        if (e == hipSuccess) e = launch_scaled_reduce(p->dtype, a, s);
        return launched(e);
    }
    return launched(launch_scaled(p->dtype, p->tb != 0, p->tile, vec, a, s));
}

mm_status mm_glu_plan_create(const mm_glu_desc *d, int dtype, const mm_plan_options *opt, mm_plan_t *out) {
    return mm_glu_plan_create_ex(d, dtype, opt, nullptr, out);
}

mm_status mm_glu_plan_create_ex(const mm_glu_desc *d, int dtype, const mm_plan_options *opt,
                                const mm_glu_options *glu, mm_plan_t *out) {
    clear_error();
    if (!out) return fail(MM_ERR_NULL_ARG, "out is NULL");
    *out = nullptr;
    if (!d) return fail(MM_ERR_NULL_ARG, "descriptor is NULL");
    if (!float_type(dtype))
        return fail(MM_ERR_DTYPE, "the gated block takes FLOAT, FLOAT16 and BFLOAT16 (got %d)", dtype);
    if (d->reserved != 0 || (opt && opt->reserved != 0)) return fail(MM_ERR_BAD_OPTION, "reserved field must be 0");
    if ((d->trans_w != 0 && d->trans_w != 1) || (d->training != 0 && d->training != 1))
        return fail(MM_ERR_BAD_OPTION, "trans_w and training must be 0 or 1");
    if (d->activation < MM_ACT_SILU || d->activation > MM_ACT_SIGMOID)
        return fail(MM_ERR_BAD_OPTION, "unknown activation %d", d->activation);
    if (d->rows < 0 || d->in_features < 0 || d->hidden < 0)
        return fail(MM_ERR_NEG_DIM, "rows, in_features and hidden must not be negative");
    const int64_t M = d->rows, K = d->in_features, N = d->hidden;
    const int64_t row = d->trans_w ? K : N;
    if (d->w_pitch != 0 && d->w_pitch < row)
        return fail(MM_ERR_BAD_OPTION, "w_pitch %lld is below the weights' row length %lld", (long long)d->w_pitch,
                    (long long)row);
    if (M > kMaxSize || K > kMaxSize || N > kMaxSize || d->w_pitch > kMaxSize)
        return fail(MM_ERR_TOO_LARGE, "rows, in_features, hidden and w_pitch must each be below 2^31 - 64");
    if (too_large(M, K) || too_large(M, N) || too_large(K, N) || too_large(d->trans_w ? N : K, d->w_pitch))
        return fail(MM_ERR_TOO_LARGE, "a matrix of more than 2^40 elements");
    const int force = opt ? opt->force_algo : MM_ALGO_AUTO;
    const bool rows_ok = M <= kFfnRows;
    const int treq = opt ? opt->tile : 0, sreq = opt ? opt->split_k : 0;
    if (force != MM_ALGO_AUTO && force != MM_ALGO_GENERAL && force != MM_ALGO_SKINNY_M && force != MM_ALGO_SPLIT_K)
        return fail(MM_ERR_BAD_OPTION, "the gated block runs on the skinny-M, general and split-K kernels only");
    if (force == MM_ALGO_SKINNY_M && !rows_ok)
        return fail(MM_ERR_BAD_OPTION, "SKINNY_M takes at most %d rows", kFfnRows);
    if (sreq < 0) return fail(MM_ERR_BAD_OPTION, "split_k %d is negative", sreq);
    int only = -1;
    mm_status st = tile_option(opt, &only);
    if (st == MM_OK && M > 0 && N > 0) st = forced_alone(opt);
    if (st != MM_OK) return st;
    unsigned tiles = dtype == MM_FLOAT ? 0xe : 0x1f;  // FLOAT has the three smaller entries
    if (only >= 0) tiles &= 1u << only;
    if (!tiles) return fail(MM_ERR_BAD_OPTION, "tile %d has no FLOAT kernel", treq);
    if (force == MM_ALGO_SPLIT_K || sreq > 1) tiles &= ~1u;  // no 256 x 256 partials
    if (!tiles) return fail(MM_ERR_BAD_OPTION, "tile 1 does not split K");
    const mm_glu_options bt = glu ? *glu : mm_glu_options{};
    if (bt.kept_type != 0 && bt.kept_type != dtype && bt.kept_type != MM_FLOAT)
        return fail(MM_ERR_DTYPE, "G and U are kept in the plan's type or in FLOAT (got %d)", bt.kept_type);
    if (!d->training && (bt.dx_tile || bt.dx_split_k || bt.dw_tile || bt.dw_split_k))
        return fail(MM_ERR_BAD_OPTION, "backward tiling of a plan without training");
    mm_plan_s *p = new (std::nothrow) mm_plan_s();
    if (!p) return fail(MM_ERR_ALLOC, "host allocation failed");
    p->dtype = dtype;
    p->is_glu = true;
    p->tb = d->trans_w;
    p->act = d->activation;
    p->training = d->training != 0;
    p->kept = bt.kept_type ? bt.kept_type : dtype;
    p->w_pitch = d->w_pitch ? d->w_pitch : row;
    p->out_rank = 2;
    p->out_shape[0] = M;
    p->out_shape[1] = N;
    p->M = p->kernel_m = M;
    p->N = N;
    p->K = K;
    p->out_numel = M * N;
    p->total_batch = p->batch = 1;
    const int64_t es = elem_size(dtype);
    const int cls = type_class(dtype);
    if (p->out_numel == 0) {
        p->algo = MM_ALGO_EMPTY;
    } else {
        const bool aligned = (K * es) % 16 == 0 && (p->w_pitch * es) % 16 == 0 && (p->tb || (N * es) % 16 == 0);
        const bool may_split = force != MM_ALGO_GENERAL && K > 0;
        FfnChoice c = choose(cls, aligned, 1, M, 2 * N, K * es, 1, tiles, may_split && sreq == 0);
        const double wbytes = 2.0 * (double)K * (double)N * (double)es;
        if (force == MM_ALGO_SKINNY_M || (force == MM_ALGO_AUTO && rows_ok && treq == 0 && sreq == 0 &&
                                          rows_us(cls, p->tb != 0, M, N, K * es, p->w_pitch * es, wbytes) <=
                                              tiles_us(cls, c, p->tb != 0, aligned, p->w_pitch * es, wbytes))) {
            p->algo = MM_ALGO_SKINNY_M;
            if (!launchable((double)cdiv(N, 8), 512)) st = fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
        } else {
            if (may_split && sreq > 0) set_split(&c, K * es, 1, sreq);
            p->tile = c.tile;
            p->split = c.split;
            p->kstages = c.kstages;
            p->algo = c.split > 1 || (force == MM_ALGO_SPLIT_K && may_split) ? MM_ALGO_SPLIT_K : MM_ALGO_GENERAL;
            if (!tile_launchable(c, 1, M, 2 * N) || (p->algo == MM_ALGO_SPLIT_K && !pieces_launchable(M, cdiv(N, 4))))
                st = fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
            if (p->algo == MM_ALGO_SPLIT_K) {
                p->kchunk = (int64_t)c.kstages * kFfnTiles[c.tile].bkb / es;
                p->workspace_bytes = round_up((int64_t)c.split * 2 * M * N * 4, 256);
            }
        }
    }
    if (st == MM_OK && p->training) {
        p->d_off = p->workspace_bytes;
        p->d_pitch = round_up(N, 16 / es);
        p->d_bytes = round_up(M * p->d_pitch * es, 256);
        // dW's reduction runs over the rows of X; a 16-bit 32-row tile of its
        // transposed operand has rows too short to stage.
        const unsigned dx_tiles = dtype == MM_FLOAT ? 0xe : 0x1f, dw_tiles = dtype == MM_FLOAT ? 0xe : 0x17;
        const bool dx_al = (p->w_pitch * es) % 16 == 0 && ((p->tb ? K : N) * es) % 16 == 0, dw_al = (K * es) % 16 == 0;
        st = choose_backward("dX", cls, dx_al, 1, M, K, N * es, 2, dx_tiles, bt.dx_tile, bt.dx_split_k, &p->dx);
        if (st == MM_OK)
            st = choose_backward("dW", cls, dw_al, 2, p->tb ? N : K, p->tb ? K : N, M * es, 1, dw_tiles, bt.dw_tile,
                                 bt.dw_split_k, &p->dw);
    }
    if (st == MM_OK && p->training) {
        if (!tile_launchable(p->dx, 1, M, K) || !tile_launchable(p->dw, 2, p->tb ? N : K, p->tb ? K : N) ||
            !pieces_launchable(M, cdiv(p->d_pitch * es, 16)) || (p->dx.split > 1 && !pieces_launchable(M, cdiv(K, 4))) ||
            (p->dw.split > 1 && !pieces_launchable(p->tb ? N : K, cdiv(p->tb ? K : N, 4))))
            st = fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
        int64_t part = 0;
        if (p->dx.split > 1) part = (int64_t)p->dx.split * M * K * 4;
        if (p->dw.split > 1) part = std::max(part, (int64_t)p->dw.split * 2 * K * N * 4);
        p->workspace_bytes += 2 * p->d_bytes + part;
    }
    if (st == MM_OK) st = alloc_workspace(p, true);
    if (st != MM_OK) {
        delete p;
        return st;
    }
    *out = p;
    return MM_OK;
}

mm_status mm_glu_get_options(mm_plan_t p, mm_glu_options *glu) {
    clear_error();
    if (!p || !glu) return fail(MM_ERR_NULL_ARG, "plan or glu is NULL");
    if (!p->is_glu || !p->training) return fail(MM_ERR_BAD_OPTION, "not a gated-block plan with training");
    *glu = mm_glu_options{p->kept, p->dx.tile + 1, p->dx.split, p->dw.tile + 1, p->dw.split};
    return MM_OK;
}

mm_status mm_glu_execute(mm_plan_t p, const void *X, const void *Wg, const void *Wu, void *H, void *G, void *U,
                         void *stream) {
    clear_error();
    if (!p) return fail(MM_ERR_NULL_ARG, "plan is NULL");
    if (!p->is_glu) return fail(MM_ERR_BAD_OPTION, "not a gated-block plan");
    if (p->algo == MM_ALGO_EMPTY) return MM_OK;
    if (!H) return fail(MM_ERR_NULL_ARG, "H is NULL for a non-empty output");
    if (!G != !U) return fail(MM_ERR_NULL_ARG, "G and U are given together or not at all");
    if (p->K > 0 && (!X || !Wg || !Wu)) return fail(MM_ERR_NULL_ARG, "X, Wg or Wu is NULL");
    hipStream_t s = (hipStream_t)stream;
    const int64_t es = elem_size(p->dtype);
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.A[0] = X;
    a.B[0] = Wg;
    a.B[1] = Wu;
    a.Y[0] = H;
    a.G = G;
    a.U = U;
    a.M = p->M;
    a.N = p->N;
    a.K = p->K;
    a.lda = p->K;
    a.ldb = p->w_pitch;
    a.ldy = p->N;
    a.batch = 1;
    a.split = p->split;
    a.kstages = p->kstages;
    a.act = p->act;
    a.y_vec = aligned16(H) && (p->N * es) % 16 == 0;
    a.kept_vec = aligned16(G) && aligned16(U) && (p->N * elem_size(p->kept)) % 16 == 0;
    a.kept32 = p->kept != p->dtype;
    if (p->algo == MM_ALGO_SKINNY_M) return launched(launch_glu_rows(p->dtype, p->tb != 0, a, s));
    const bool vec = aligned16(X) && aligned16(Wg) && aligned16(Wu) && (p->K * es) % 16 == 0 &&
                     (p->w_pitch * es) % 16 == 0 && (p->tb || (p->N * es) % 16 == 0);
    if (p->algo != MM_ALGO_SPLIT_K) return launched(launch_glu_fwd(p->dtype, p->tb != 0, p->tile, false, vec, a, s));
    mm_status st = alloc_workspace(p, false);
    if (st != MM_OK) return st;
    a.W = p->ws;
    hipError_t e = launch_glu_fwd(p->dtype, p->tb != 0, p->tile, true, vec, a, s);
    if (e == hipSuccess) e = launch_glu_reduce(p->dtype, a, s);
    return launched(e);
}

mm_status mm_glu_backward(mm_plan_t p, const void *X, const void *Wg, const void *Wu, const void *G, const void *U,
                          const void *dH, void *dX, void *dWg, void *dWu, void *stream) {
    clear_error();
    if (!p) return fail(MM_ERR_NULL_ARG, "plan is NULL");
    if (!p->is_glu) return fail(MM_ERR_BAD_OPTION, "not a gated-block plan");
    if (!p->training) return fail(MM_ERR_BAD_OPTION, "the plan was created without training");
    if (!dWg != !dWu) return fail(MM_ERR_NULL_ARG, "dWg and dWu are given together or not at all");
    const int64_t M = p->M, N = p->N, K = p->K, es = elem_size(p->dtype);
    const bool want_x = dX && M > 0 && K > 0, want_w = dWg && N > 0 && K > 0;
    if (!want_x && !want_w) return MM_OK;
    hipStream_t s = (hipStream_t)stream;
    if (p->out_numel > 0) {
        if (!G || !U || !dH) return fail(MM_ERR_NULL_ARG, "G, U or dH is NULL");
        if (want_x && (!Wg || !Wu)) return fail(MM_ERR_NULL_ARG, "Wg or Wu is NULL");
        if (want_w && !X) return fail(MM_ERR_NULL_ARG, "X is NULL");
        mm_status st = alloc_workspace(p, false);
        if (st != MM_OK) return st;
    }
    char *dG = (char *)p->ws + p->d_off, *dU = dG + p->d_bytes;
    if (p->out_numel > 0) {
        mm_status st = launched(launch_glu_dact(p->dtype, p->kept, p->act, G, U, dH, dG, dU, M, N, p->d_pitch, s));
        if (st != MM_OK) return st;
    }
    void *part = dU + p->d_bytes;
    const bool w_vec = (p->w_pitch * es) % 16 == 0;
    if (want_x) {
        // dX [M, K] = dG Wg' + dU Wu', the reduction over the hidden features:
        // weights stored [K, N] are K-contiguous rows, [N, K] rows of one n.
        FfnArgs a;
        memset(&a, 0, sizeof(a));
        a.A[0] = dG;
        a.A[1] = dU;
        a.B[0] = Wg;
        a.B[1] = Wu;
        a.Y[0] = dX;
        a.M = M;
        a.N = K;
        a.K = N;
        a.lda = std::max<int64_t>(p->d_pitch, 1);
        a.ldb = p->w_pitch;
        a.ldy = K;
        a.batch = 1;
        a.y_vec = aligned16(dX) && (K * es) % 16 == 0;
        const bool vec = w_vec && aligned16(Wg) && aligned16(Wu) && ((p->tb ? K : N) * es) % 16 == 0;
        a.W = part;
        a.split = p->dx.split;
        a.kstages = p->dx.kstages;
        hipError_t e = launch_glu_dx(p->dtype, !p->tb, p->dx.tile, a.split > 1, vec, a, s);
        if (e == hipSuccess && a.split > 1) e = launch_sum_reduce(p->dtype, a, s);
        mm_status st = launched(e);
        if (st != MM_OK) return st;
    }
    if (want_w) {
        // Weights [N, K]: dW = dG^T X; [K, N]: dW = X^T dG.  The reduction
        // over the rows reads both operands as rows of one k.
        FfnArgs a;
        memset(&a, 0, sizeof(a));
        a.A[0] = p->tb ? dG : X;
        a.A[1] = p->tb ? dU : X;
        a.B[0] = p->tb ? X : dG;
        a.B[1] = p->tb ? X : dU;
        a.Y[0] = dWg;
        a.Y[1] = dWu;
        a.M = p->tb ? N : K;
        a.N = p->tb ? K : N;
        a.K = M;
        a.lda = std::max<int64_t>(p->tb ? p->d_pitch : K, 1);
        a.ldb = std::max<int64_t>(p->tb ? K : p->d_pitch, 1);
        a.ldy = p->w_pitch;
        a.batch = 2;
        a.y_vec = aligned16(dWg) && aligned16(dWu) && w_vec && (a.N * es) % 16 == 0;
        const bool vec = aligned16(X) && (K * es) % 16 == 0;
        a.W = part;
        a.split = p->dw.split;
        a.kstages = p->dw.kstages;
        hipError_t e = launch_glu_dw(p->dtype, p->dw.tile, a.split > 1, vec, a, s);
        if (e == hipSuccess && a.split > 1) e = launch_sum_reduce(p->dtype, a, s);
        mm_status st = launched(e);
        if (st != MM_OK) return st;
    }
    return MM_OK;
}

}  // extern "C"
