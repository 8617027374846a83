// plan_linear.cpp -- plans and executions of the linear layer with its
// epilogue, and the 8-bit checkpoints.
#include <string.h>

#include <algorithm>
#include <new>

#include "ffn_choice.h"

using namespace mm;

namespace mm {

// A product as one launch, or (col > 0) as columns [0, col) in whole rounds of
// workgroups and the rest on another entry: `run` gets each part's arguments.
template <class Run>
static hipError_t in_rounds(const FfnArgs &a, int64_t es, int64_t col, bool tb, Run run) {
    if (col <= 0) return run(a, false);
    FfnArgs first = a, rest = a;
    first.N = col;
    rest.N = a.N - col;
    rest.B[0] = (const char *)a.B[0] + (tb ? col * a.ldb : col) * es;
    rest.Y[0] = (char *)a.Y[0] + col * es;
    if (a.G) rest.G = (char *)a.G + col * (a.q8 ? 1 : a.kept32 ? 4 : es);
    if (a.zs) rest.zs = (char *)a.zs + col / MM_CHECKPOINT_BLOCK;
    if (a.R) rest.R = (const char *)a.R + col * es;
    if (a.bias) rest.bias = (const char *)a.bias + col * es;
    const hipError_t e = run(first, false);
    return e == hipSuccess ? run(rest, true) : e;
}

}  // namespace mm

extern "C" {

int64_t mm_checkpoint_blocks(int64_t cols) { return cols < 0 ? -1 : cdiv(cols, MM_CHECKPOINT_BLOCK); }

static mm_status checkpoint_sizes(const char *call, int dtype, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(MM_ERR_NEG_DIM, "rows and cols must not be negative");
    if (!float_type(dtype)) return fail(MM_ERR_DTYPE, "%s takes FLOAT, FLOAT16 or BFLOAT16 (got %d)", call, dtype);
    if (rows > INT32_MAX || cols > INT32_MAX || too_large(rows, cols))
        return fail(MM_ERR_TOO_LARGE, "rows and cols must each be below 2^31, their product at most 2^40");
    return MM_OK;
}

mm_status mm_checkpoint_pack(const void *X, int dtype, int64_t rows, int64_t cols, void *q, void *scale, void *stream) {
    clear_error();
    mm_status st = checkpoint_sizes("checkpoint_pack", dtype, rows, cols);
    if (st != MM_OK || rows == 0 || cols == 0) return st;
    if (!X || !q || !scale) return fail(MM_ERR_NULL_ARG, "X, q or scale is NULL");
    return launched(launch_checkpoint_pack(dtype, X, rows, cols, q, scale, (hipStream_t)stream));
}

mm_status mm_checkpoint_unpack(const void *q, const void *scale, int64_t rows, int64_t cols, int dtype, void *X,
                               void *stream) {
    clear_error();
    mm_status st = checkpoint_sizes("checkpoint_unpack", dtype, rows, cols);
    if (st != MM_OK || rows == 0 || cols == 0) return st;
    if (!X || !q || !scale) return fail(MM_ERR_NULL_ARG, "q, scale or X is NULL");
    return launched(launch_checkpoint_unpack(dtype, q, scale, rows, cols, X, (hipStream_t)stream));
}

mm_status mm_linear_plan_create(const mm_linear_desc *d, int dtype, const mm_plan_options *opt, mm_plan_t *out) {
    clear_error();
    if (!out) return fail(MM_ERR_NULL_ARG, "out is NULL");
    *out = nullptr;
    if (!d) return fail(MM_ERR_NULL_ARG, "descriptor is NULL");
    if (!float_type(dtype))
        return fail(MM_ERR_DTYPE, "the linear layer takes FLOAT, FLOAT16 and BFLOAT16 (got %d)", dtype);
    if (d->reserved != 0 || (opt && opt->reserved != 0)) return fail(MM_ERR_BAD_OPTION, "reserved field must be 0");
    auto flag = [](int32_t v) { return v == 0 || v == 1; };
    if (!flag(d->trans_w) || !flag(d->has_bias) || !flag(d->has_residual) || !flag(d->training))
        return fail(MM_ERR_BAD_OPTION, "trans_w, has_bias, has_residual and training must be 0 or 1");
    if (d->activation < MM_ACT_NONE || d->activation > MM_ACT_SIGMOID || d->x_activation < MM_ACT_NONE ||
        d->x_activation > MM_ACT_SIGMOID)
        return fail(MM_ERR_BAD_OPTION, "unknown activation %d or %d", d->activation, d->x_activation);
    if (d->z_type != 0 && d->z_type != dtype && d->z_type != MM_FLOAT && d->z_type != MM_INT8)
        return fail(MM_ERR_DTYPE, "Z is kept in the plan's type, in FLOAT or as a checkpoint (got %d)", d->z_type);
    if (d->x_type != 0 && d->x_type != dtype && d->x_type != MM_INT8)
        return fail(MM_ERR_DTYPE, "X is given in the plan's type or as a checkpoint (got %d)", d->x_type);
    if (d->z_type != 0 && (!d->training || d->activation == MM_ACT_NONE))
        return fail(MM_ERR_BAD_OPTION, "only a training plan with an activation keeps Z");
    if (d->x_type != 0 && !d->training) return fail(MM_ERR_BAD_OPTION, "x_type is for a training plan");
    if (d->x_activation != MM_ACT_NONE && d->x_type != MM_INT8)
        return fail(MM_ERR_BAD_OPTION, "x_activation is for an X given as a checkpoint");
    if (!d->training && (d->dx_tile || d->dx_split_k || d->dw_tile || d->dw_split_k))
        return fail(MM_ERR_BAD_OPTION, "backward tiling of a plan without training");
    if (d->rows < 0 || d->in_features < 0 || d->out_features < 0)
        return fail(MM_ERR_NEG_DIM, "rows, in_features and out_features must not be negative");
    const int64_t M = d->rows, K = d->in_features, N = d->out_features;
    const int64_t row = d->trans_w ? K : N;
    if (d->w_pitch != 0 && d->w_pitch < row)
        return fail(MM_ERR_BAD_OPTION, "w_pitch %lld is below the weights' row length %lld", (long long)d->w_pitch,
                    (long long)row);
    if (M > kMaxSize || K > kMaxSize || N > kMaxSize || d->w_pitch > kMaxSize)
        return fail(MM_ERR_TOO_LARGE, "rows, in_features, out_features and w_pitch must each be below 2^31 - 64");
    if (too_large(M, K) || too_large(M, N) || too_large(K, N) || too_large(d->trans_w ? N : K, d->w_pitch))
        return fail(MM_ERR_TOO_LARGE, "a matrix of more than 2^40 elements");
    const int force = opt ? opt->force_algo : MM_ALGO_AUTO;
    const int treq = opt ? opt->tile : 0, sreq = opt ? opt->split_k : 0;
    // A checkpoint of Z is formed by the kernels that hold a block of it.
    const bool z8 = d->z_type == MM_INT8, rows_ok = M <= kFfnRows && !z8;
    if (force != MM_ALGO_AUTO && force != MM_ALGO_GENERAL && force != MM_ALGO_SKINNY_M && force != MM_ALGO_SPLIT_K)
        return fail(MM_ERR_BAD_OPTION, "the linear layer runs on the skinny-M, general and split-K kernels only");
    if (force == MM_ALGO_SKINNY_M && !rows_ok)
        return fail(MM_ERR_BAD_OPTION, "SKINNY_M takes at most %d rows, and no checkpoint of Z", kFfnRows);
    if (sreq < 0) return fail(MM_ERR_BAD_OPTION, "split_k %d is negative", sreq);
    int only = -1;
    mm_status st = tile_option(opt, &only);
    if (st == MM_OK && M > 0 && N > 0) st = forced_alone(opt);
    if (st != MM_OK) return st;
    const unsigned any = dtype == MM_FLOAT ? 0xe : 0x1f;  // FLOAT has the three smaller entries
    unsigned tiles = any;
    if (only >= 0) tiles &= 1u << only;
    if (!tiles) return fail(MM_ERR_BAD_OPTION, "tile %d has no FLOAT kernel", treq);
    if (force == MM_ALGO_SPLIT_K || sreq > 1) tiles &= ~1u;  // no 256 x 256 partials
    if (!tiles) return fail(MM_ERR_BAD_OPTION, "tile 1 does not split K");
    mm_plan_s *p = new (std::nothrow) mm_plan_s();
    if (!p) return fail(MM_ERR_ALLOC, "host allocation failed");
    p->dtype = dtype;
    p->is_linear = true;
    p->tb = d->trans_w;
    p->act = d->activation;
    p->has_bias = d->has_bias != 0;
    p->has_residual = d->has_residual != 0;
    p->training = d->training != 0;
    p->kept = p->training && p->act != MM_ACT_NONE ? (d->z_type ? d->z_type : dtype) : 0;
    p->x_type = d->x_type ? d->x_type : dtype;
    p->x_act = d->x_activation;
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
    const int cls = dtype == MM_FLOAT ? kClass32 : kClassLinear16;
    if (p->out_numel == 0) {
        p->algo = MM_ALGO_EMPTY;
    } else {
        const bool aligned = (K * es) % 16 == 0 && (p->w_pitch * es) % 16 == 0 && (p->tb || (N * es) % 16 == 0);
        const bool may_split = force != MM_ALGO_GENERAL && K > 0;
        const double wbytes = (double)K * (double)N * (double)es;
        auto pick = [&](unsigned from) { return choose(cls, aligned, 1, M, N, K * es, 1, from, may_split && sreq == 0); };
        FfnChoice c = pick(tiles);
        if (force == MM_ALGO_SKINNY_M ||
            (force == MM_ALGO_AUTO && rows_ok && treq == 0 && sreq == 0 &&
             linear_rows_us(type_class(dtype), p->tb != 0, M, N, K * es, p->w_pitch * es, wbytes) <=
                 tiles_us(cls, c, p->tb != 0, aligned, p->w_pitch * es, wbytes))) {
            p->algo = MM_ALGO_SKINNY_M;
            if (!launchable((double)cdiv(N, 16), 512)) st = fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
        } else {
            auto settle = [&](const FfnChoice &from) {
                c = from;
                if (may_split && sreq > 0) set_split(&c, K * es, 1, sreq);
            };
            settle(c);
            // Whole products of the 32-row entry do not hold checkpoint blocks
            // (split ones do: their joining forms them).
            if (z8 && c.tile == 3 && c.split == 1 && !(force == MM_ALGO_SPLIT_K && may_split)) {
                if (only >= 0) st = fail(MM_ERR_BAD_OPTION, "tile 4 forms no checkpoint of Z without a split");
                else settle(pick(tiles & ~8u));
            }
            if (c.split == 1 && treq == 0 && sreq == 0 && force == MM_ALGO_AUTO && aligned)
                p->tail_col = balance(cls, &c, M, N, K * es, z8 ? any & ~8u : any, &p->tail_tile);
            p->tile = c.tile;
            p->split = c.split;
            p->kstages = c.kstages;
            p->algo = c.split > 1 || (force == MM_ALGO_SPLIT_K && may_split) ? MM_ALGO_SPLIT_K : MM_ALGO_GENERAL;
            if (st == MM_OK &&
                (!tile_launchable(c, 1, M, N) || (p->algo == MM_ALGO_SPLIT_K && !pieces_launchable(M, cdiv(N, 32) * 8))))
                st = fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
            if (p->algo == MM_ALGO_SPLIT_K) {
                p->kchunk = (int64_t)c.kstages * kFfnTiles[c.tile].bkb / es;
                p->workspace_bytes = round_up((int64_t)c.split * M * N * 4, 256);
            }
        }
    }
    if (st == MM_OK && p->training) {
        const int64_t ve = 16 / es;
        const bool dz = p->act != MM_ACT_NONE, x8 = p->x_type == MM_INT8;
        p->d_off = p->workspace_bytes;
        p->d_pitch = dz ? round_up(N, ve) : N;
        p->x_off = p->d_off + (dz ? round_up(M * p->d_pitch * es, 256) : 0);
        p->x_pitch = x8 ? round_up(K, ve) : K;
        p->p_off = p->x_off + (x8 ? round_up(M * p->x_pitch * es, 256) : 0);
        p->p_pitch = round_up(N, 4);
        p->s_off = p->p_off + (p->has_bias ? round_up(cdiv(M, linear_prep_rows(M, N, dtype)) * p->p_pitch * 4, 256) : 0);
        // dW's reduction runs over the rows of X; a 16-bit 32-row tile of its
        // transposed operand has rows too short to stage.
        const unsigned dw_tiles = dtype == MM_FLOAT ? 0xe : 0x17;
        const int64_t wm = p->tb ? N : K, wn = p->tb ? K : N;  // dW as stored
        const bool z_al = (p->d_pitch * es) % 16 == 0, x_al = (p->x_pitch * es) % 16 == 0;
        const bool w_al = (p->w_pitch * es) % 16 == 0 && (wn * es) % 16 == 0;
        st = choose_backward("dX", cls, z_al && w_al, 1, M, K, N * es, 1, any, d->dx_tile, d->dx_split_k, &p->dx);
        if (st == MM_OK)
            st = choose_backward("dW", cls, z_al && x_al, 1, wm, wn, M * es, 1, dw_tiles, d->dw_tile, d->dw_split_k, &p->dw);
        if (st == MM_OK && p->dx.split == 1 && d->dx_tile == 0 && d->dx_split_k == 0 && z_al && w_al)
            p->dx_tail_col = balance(cls, &p->dx, M, K, N * es, any, &p->dx_tail_tile);
        if (st == MM_OK && p->dw.split == 1 && d->dw_tile == 0 && d->dw_split_k == 0 && z_al && x_al)
            p->dw_tail_col = balance(cls, &p->dw, wm, wn, M * es, dw_tiles, &p->dw_tail_tile);
        LinearPrep prep = {};
        prep.dZ = prep.X = p;  // (not read)
        prep.M = M;
        prep.N = N;
        prep.K = K;
        prep.ldz = round_up(N, ve);
        prep.ldx = round_up(K, ve);
        prep.rows = linear_prep_rows(M, N, dtype);
        if (st == MM_OK &&
            (!tile_launchable(p->dx, 1, M, K) || !tile_launchable(p->dw, 1, wm, wn) ||
             !launchable((double)linear_prep_blocks(prep, dtype), 256) ||
             (p->dx.split > 1 && !pieces_launchable(M, cdiv(K, 32) * 8)) || (p->dw.split > 1 && !pieces_launchable(wm, cdiv(wn, 4)))))
            st = fail(MM_ERR_TOO_LARGE, "a launch of more than 2^32 threads");
        int64_t part = 0;
        if (p->dx.split > 1) part = (int64_t)p->dx.split * M * K * 4;
        if (p->dw.split > 1) part = std::max(part, (int64_t)p->dw.split * K * N * 4);
        p->workspace_bytes = p->s_off + part;
    }
    if (st == MM_OK) st = alloc_workspace(p, true);
    if (st != MM_OK) {
        delete p;
        return st;
    }
    *out = p;
    return MM_OK;
}

mm_status mm_linear_get_desc(mm_plan_t p, mm_linear_desc *d) {
    clear_error();
    if (!p || !d) return fail(MM_ERR_NULL_ARG, "plan or desc is NULL");
    if (!p->is_linear) return fail(MM_ERR_BAD_OPTION, "not a linear-layer plan");
    memset(d, 0, sizeof(*d));
    d->rows = p->M;
    d->in_features = p->K;
    d->out_features = p->N;
    d->w_pitch = p->w_pitch;
    d->trans_w = p->tb;
    d->activation = p->act;
    d->has_bias = p->has_bias;
    d->has_residual = p->has_residual;
    d->training = p->training;
    d->z_type = p->kept;
    if (p->training) {
        d->x_type = p->x_type;
        d->x_activation = p->x_act;
        d->dx_tile = p->dx.tile + 1;
        d->dx_split_k = p->dx.split;
        d->dw_tile = p->dw.tile + 1;
        d->dw_split_k = p->dw.split;
    }
    return MM_OK;
}

mm_status mm_linear_get_tails(mm_plan_t p, mm_linear_tails *t) {
    clear_error();
    if (!p || !t) return fail(MM_ERR_NULL_ARG, "plan or tails is NULL");
    if (!p->is_linear || !p->training) return fail(MM_ERR_BAD_OPTION, "not a linear-layer plan with training");
    *t = mm_linear_tails{p->dx_tail_col, p->dw_tail_col, p->dx_tail_tile + 1, p->dw_tail_tile + 1};
    return MM_OK;
}

mm_status mm_linear_execute(mm_plan_t p, const void *X, const void *W, const void *bias, const void *residual, void *Y,
                            void *Z, void *z_scale, void *stream) {
    clear_error();
    if (!p) return fail(MM_ERR_NULL_ARG, "plan is NULL");
    if (!p->is_linear) return fail(MM_ERR_BAD_OPTION, "not a linear-layer plan");
    if (!p->has_bias && bias) return fail(MM_ERR_BAD_OPTION, "the plan has no bias");
    if (!p->has_residual && residual) return fail(MM_ERR_BAD_OPTION, "the plan has no residual");
    if (!p->kept && Z) return fail(MM_ERR_BAD_OPTION, "the plan keeps no Z");
    if (z_scale && (!Z || p->kept != MM_INT8)) return fail(MM_ERR_BAD_OPTION, "z_scale goes with a Z kept as a checkpoint");
    if (p->algo == MM_ALGO_EMPTY) return MM_OK;
    if (!Y) return fail(MM_ERR_NULL_ARG, "Y is NULL for a non-empty output");
    if (p->K > 0 && (!X || !W)) return fail(MM_ERR_NULL_ARG, "X or W is NULL");
    if (p->has_bias && !bias) return fail(MM_ERR_NULL_ARG, "the plan has a bias but bias is NULL");
    if (p->has_residual && !residual) return fail(MM_ERR_NULL_ARG, "the plan has a residual but residual is NULL");
    if (Z && p->kept == MM_INT8 && !z_scale) return fail(MM_ERR_NULL_ARG, "Z is a checkpoint but z_scale is NULL");
    hipStream_t s = (hipStream_t)stream;
    const int64_t es = elem_size(p->dtype);
    FfnArgs a;
    memset(&a, 0, sizeof(a));
    a.A[0] = X;
    a.B[0] = W;
    a.Y[0] = Y;
    a.G = Z;
    a.zs = z_scale;
    a.R = residual;
    a.bias = bias;
    a.M = p->M;
    a.N = p->N;
    a.K = p->K;
    a.lda = std::max<int64_t>(p->K, 1);
    a.ldb = p->w_pitch;
    a.ldy = p->N;
    a.batch = 1;
    a.split = p->split;
    a.kstages = p->kstages;
    a.act = p->act;
    a.y_vec = aligned16(Y) && (p->N * es) % 16 == 0;
    a.q8 = p->kept == MM_INT8;
    a.kept32 = p->kept == MM_FLOAT && p->dtype != MM_FLOAT;
    a.kept_vec = aligned16(Z) && (p->N * (a.q8 ? 1 : a.kept32 ? 4 : es)) % 16 == 0;
    a.r_vec = aligned16(residual) && (p->N * es) % 16 == 0;
    if (p->algo == MM_ALGO_SKINNY_M) return launched(launch_linear_rows(p->dtype, p->tb != 0, a, s));
    const bool vec = aligned16(X) && aligned16(W) && (p->K * es) % 16 == 0 && (p->w_pitch * es) % 16 == 0 &&
                     (p->tb || (p->N * es) % 16 == 0);
    if (p->algo != MM_ALGO_SPLIT_K)
        return launched(in_rounds(a, es, p->tail_col, p->tb != 0, [&](const FfnArgs &part, bool rest) {
            return launch_linear(p->dtype, p->tb != 0, rest ? p->tail_tile : p->tile, false, vec, part, s);
        }));
    mm_status st = alloc_workspace(p, false);
    if (st != MM_OK) return st;
    a.W = p->ws;
    hipError_t e = launch_linear(p->dtype, p->tb != 0, p->tile, true, vec, a, s);
    if (e == hipSuccess) e = launch_linear_reduce(p->dtype, a, s);
    return launched(e);
}

mm_status mm_linear_backward(mm_plan_t p, const void *X, const void *x_scale, const void *W, const void *Z,
                             const void *z_scale, const void *dY, void *dX, void *dW, void *dbias, void *stream) {
    clear_error();
    if (!p) return fail(MM_ERR_NULL_ARG, "plan is NULL");
    if (!p->is_linear) return fail(MM_ERR_BAD_OPTION, "not a linear-layer plan");
    if (!p->training) return fail(MM_ERR_BAD_OPTION, "the plan was created without training");
    if (dbias && !p->has_bias) return fail(MM_ERR_BAD_OPTION, "the plan has no bias");
    if (Z && !p->kept) return fail(MM_ERR_BAD_OPTION, "the plan keeps no Z");
    const bool x8 = p->x_type == MM_INT8, z8 = p->kept == MM_INT8, act = p->act != MM_ACT_NONE;
    if (x_scale && !x8) return fail(MM_ERR_BAD_OPTION, "x_scale goes with an X given as a checkpoint");
    if (z_scale && !z8) return fail(MM_ERR_BAD_OPTION, "z_scale goes with a Z kept as a checkpoint");
    const int64_t M = p->M, N = p->N, K = p->K, es = elem_size(p->dtype);
    const bool want_x = dX && M > 0 && K > 0, want_w = dW && N > 0 && K > 0, want_b = dbias && N > 0;
    if (!want_x && !want_w && !want_b) return MM_OK;
    hipStream_t s = (hipStream_t)stream;
    const bool read_x = want_w && M > 0;
    if (p->out_numel > 0) {
        if (!dY) return fail(MM_ERR_NULL_ARG, "dY is NULL");
        if (act && (!Z || (z8 && !z_scale))) return fail(MM_ERR_NULL_ARG, "Z or z_scale is NULL");
        if (want_x && !W) return fail(MM_ERR_NULL_ARG, "W is NULL");
    }
    if (read_x && (!X || (x8 && !x_scale))) return fail(MM_ERR_NULL_ARG, "X or x_scale is NULL");
    if (p->workspace_bytes > 0) {
        mm_status st = alloc_workspace(p, false);
        if (st != MM_OK) return st;
    }
    char *ws = (char *)p->ws;
    const bool form_z = act && p->out_numel > 0, form_x = x8 && read_x;
    LinearPrep prep = {};
    prep.dY = dY;
    prep.Z = Z;
    prep.zs = z_scale;
    prep.dZ = form_z ? ws + p->d_off : nullptr;
    prep.part = want_b && M > 0 ? (float *)(ws + p->p_off) : nullptr;
    prep.xq = X;
    prep.xs = x_scale;
    prep.X = form_x ? ws + p->x_off : nullptr;
    prep.M = M;
    prep.N = N;
    prep.ldz = round_up(N, 16 / es);
    prep.ldp = p->p_pitch;
    prep.K = K;
    prep.ldx = p->x_pitch;
    prep.act = p->act;
    prep.z_type = p->kept;
    prep.x_act = p->x_act;
    prep.rows = linear_prep_rows(M, N, p->dtype);
    mm_status st = launched(launch_linear_prep(p->dtype, prep, s));
    if (st == MM_OK && want_b) {
        JoinArgs j = {};
        j.part = prep.part;
        j.P = cdiv(M, prep.rows);
        j.ldp = p->p_pitch;
        j.N = N;
        j.out = dbias;
        st = launched(launch_join(p->dtype, j, s));
    }
    if (st != MM_OK) return st;
    const void *dZ = act ? (const void *)(ws + p->d_off) : dY;
    const void *xv = x8 ? (const void *)(ws + p->x_off) : X;
    const bool z_vec = aligned16(dZ) && (p->d_pitch * es) % 16 == 0, w_vec = (p->w_pitch * es) % 16 == 0;
    if (want_x) {
        // dX [M, K] = dZ W', the reduction over the output features: weights
        // stored [K, N] are N-contiguous rows, [N, K] rows of one n.
        FfnArgs a;
        memset(&a, 0, sizeof(a));
        a.A[0] = dZ;
        a.B[0] = W;
        a.Y[0] = dX;
        a.M = M;
        a.N = K;
        a.K = N;
        a.lda = std::max<int64_t>(p->d_pitch, 1);
        a.ldb = p->w_pitch;
        a.ldy = K;
        a.batch = 1;
        a.y_vec = aligned16(dX) && (K * es) % 16 == 0;
        const bool vec = z_vec && w_vec && aligned16(W) && ((p->tb ? K : N) * es) % 16 == 0;
        a.W = ws + p->s_off;
        a.split = p->dx.split;
        a.kstages = p->dx.kstages;
        hipError_t e = in_rounds(a, es, p->dx_tail_col, !p->tb, [&](const FfnArgs &part, bool rest) {
            return launch_linear(p->dtype, !p->tb, rest ? p->dx_tail_tile : p->dx.tile, a.split > 1, vec, part, s);
        });
        if (e == hipSuccess && a.split > 1) e = launch_linear_reduce(p->dtype, a, s);
        st = launched(e);
        if (st != MM_OK) return st;
    }
    if (want_w) {
        // Weights [N, K]: dW = dZ^T X; [K, N]: dW = X^T dZ.  The reduction
        // over the rows reads both operands as rows of one k.
        FfnArgs a;
        memset(&a, 0, sizeof(a));
        a.A[0] = p->tb ? dZ : xv;
        a.B[0] = p->tb ? xv : dZ;
        a.Y[0] = dW;
        a.M = p->tb ? N : K;
        a.N = p->tb ? K : N;
        a.K = M;
        a.lda = std::max<int64_t>(p->tb ? p->d_pitch : p->x_pitch, 1);
        a.ldb = std::max<int64_t>(p->tb ? p->x_pitch : p->d_pitch, 1);
        a.ldy = p->w_pitch;
        a.batch = 1;
        a.y_vec = aligned16(dW) && w_vec && (a.N * es) % 16 == 0;
        const bool vec = z_vec && aligned16(xv) && (p->x_pitch * es) % 16 == 0;
        a.W = ws + p->s_off;
        a.split = p->dw.split;
        a.kstages = p->dw.kstages;
        hipError_t e = in_rounds(a, es, p->dw_tail_col, false, [&](const FfnArgs &part, bool rest) {
            return launch_linear_dw(p->dtype, rest ? p->dw_tail_tile : p->dw.tile, a.split > 1, vec, part, s);
        });
        if (e == hipSuccess && a.split > 1) e = launch_sum_reduce(p->dtype, a, s);
        st = launched(e);
        if (st != MM_OK) return st;
    }
    return MM_OK;
}

}  // extern "C"
