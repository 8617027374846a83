// plan_norm.cpp -- plans and executions of the fused norms.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "ffn_choice.h"
#include "norm.h"

namespace mm {

// Workers of the backward pass (see norm.h): as many as fill the GPU with threads.
// Their partial sums, up to 24 bytes a column each, are small against the rows (12
// bytes a column and row in 16-bit types) only where a worker has many of them.
static void deal_rows(const mm_plan_s *p, int32_t *per, int32_t *workers) {
    const int64_t M = p->M, most = (int64_t)kNumCUs * 1024 / norm_bwd_threads(p->N);
    int64_t n = std::max<int64_t>(1, cdiv(M, most));
    const int64_t gr = p->norm.gate_rows;
    if (gr > 0 && gr <= n) n = round_up(n, gr);
    *per = (int32_t)n;
    *workers = (int32_t)cdiv(M, n);
}

// Whether a gate's groups may be shared by workers.
static bool shared_groups(const mm_plan_s *p, int32_t per) { return p->norm.gate_rows > 0 && per % p->norm.gate_rows != 0; }

}  // namespace mm

using namespace mm;

extern "C" {

mm_status mm_norm_plan_create(const mm_norm_desc *d, int dtype, mm_plan_t *out) {
    clear_error();
    if (!out) return fail(MM_ERR_NULL_ARG, "out is NULL");
    *out = nullptr;
    if (!d) return fail(MM_ERR_NULL_ARG, "descriptor is NULL");
    if (!float_type(dtype)) return fail(MM_ERR_DTYPE, "norms take FLOAT, FLOAT16 and BFLOAT16 (got %d)", dtype);
    if (d->reserved != 0) return fail(MM_ERR_BAD_OPTION, "reserved field must be 0");
    if (d->rows < 0 || d->cols < 0 || d->gate_rows < 0)
        return fail(MM_ERR_NEG_DIM, "rows, cols and gate_rows must not be negative");
    for (int32_t v : {d->has_block, d->post_weight, d->post_bias, d->pre_weight, d->pre_bias, d->training})
        if (v != 0 && v != 1) return fail(MM_ERR_BAD_OPTION, "flags must be 0 or 1");
    for (int32_t v : {d->post_norm, d->pre_norm})
        if (v < MM_NORM_NONE || v > MM_NORM_LAYER) return fail(MM_ERR_BAD_OPTION, "unknown norm %d", v);
    if (d->post_norm == MM_NORM_NONE && d->pre_norm == MM_NORM_NONE) return fail(MM_ERR_BAD_OPTION, "neither norm is wanted");
    if (!d->has_block && (d->post_norm != MM_NORM_NONE || d->gate_rows != 0))
        return fail(MM_ERR_BAD_OPTION, "post_norm and gate are for a plan with a block");
    if ((d->post_norm == MM_NORM_NONE && (d->post_weight || d->post_bias)) ||
        (d->pre_norm == MM_NORM_NONE && (d->pre_weight || d->pre_bias)))
        return fail(MM_ERR_BAD_OPTION, "a weight or a bias of a norm that is absent");
    if (!(d->post_eps >= 0.0f) || !(d->pre_eps >= 0.0f) || isinf(d->post_eps) || isinf(d->pre_eps))
        return fail(MM_ERR_BAD_OPTION, "eps must be finite and not negative");
    if (!isfinite(d->residual_scale)) return fail(MM_ERR_BAD_OPTION, "residual_scale must be finite");
    if (d->kept_type != 0 && d->kept_type != dtype && d->kept_type != MM_FLOAT && d->kept_type != MM_INT8)
        return fail(MM_ERR_DTYPE, "R is kept in the plan's type, in FLOAT or as a checkpoint (got %d)", d->kept_type);
    if (d->kept_type != 0 && !d->training) return fail(MM_ERR_BAD_OPTION, "kept_type is for a training plan");
    if (d->cols > MM_NORM_MAX_COLS) return fail(MM_ERR_TOO_LARGE, "rows of more than %d columns", MM_NORM_MAX_COLS);
    if (d->rows > kMaxSize || too_large(d->rows, d->cols))
        return fail(MM_ERR_TOO_LARGE, "rows must be below 2^31 - 64, their elements at most 2^40");
    mm_plan_s *p = new (std::nothrow) mm_plan_s();
    if (!p) return fail(MM_ERR_ALLOC, "host allocation failed");
    p->dtype = dtype;
    p->is_norm = true;
    p->norm = *d;
    p->norm.gate_rows = std::min<int64_t>(d->gate_rows, std::max<int64_t>(d->rows, 1));
    p->training = d->training != 0;
    p->kept = d->kept_type ? d->kept_type : dtype;
    p->out_rank = 2;
    p->out_shape[0] = p->M = p->kernel_m = d->rows;
    p->out_shape[1] = p->N = d->cols;
    p->out_numel = d->rows * d->cols;
    p->total_batch = p->batch = 1;
    p->algo = p->out_numel == 0 ? MM_ALGO_EMPTY : MM_ALGO_DIRECT;
    mm_status st = MM_OK;
    if (p->out_numel > 0 && p->training) {
        int32_t per, workers;
        deal_rows(p, &per, &workers);
        const int64_t ldp = round_up(p->N, 4);
        const int64_t jobs = d->post_weight + d->post_bias + d->pre_weight + d->pre_bias;
        p->s_off = round_up((int64_t)workers * jobs * ldp * 4, 256);
        p->workspace_bytes = p->s_off + (shared_groups(p, per) ? round_up((int64_t)workers * 2 * ldp * 4, 256) : 0);
    }
    if (st == MM_OK) st = alloc_workspace(p, true);
    if (st != MM_OK) {
        delete p;
        return st;
    }
    *out = p;
    return MM_OK;
}

// An operand that the plan has (or not) against what was given.
static mm_status operand(const char *name, bool has, const void *given) {
    if (has && !given) return fail(MM_ERR_NULL_ARG, "%s is NULL", name);
    if (!has && given) return fail(MM_ERR_BAD_OPTION, "the plan has no %s", name);
    return MM_OK;
}

static mm_status checkpoint_pair(const mm_plan_s *p, const char *name, bool has, const void *q, const void *scale) {
    if ((q || scale) && (!p->training || !has)) return fail(MM_ERR_BAD_OPTION, "the plan makes no checkpoint of %s", name);
    if (!q != !scale) return fail(MM_ERR_NULL_ARG, "a checkpoint of %s needs numbers and scales", name);
    return MM_OK;
}

mm_status mm_norm_execute(mm_plan_t p, const mm_norm_forward_args *f, void *stream) {
    clear_error();
    if (!p || !f) return fail(MM_ERR_NULL_ARG, "plan or args is NULL");
    if (!p->is_norm) return fail(MM_ERR_BAD_OPTION, "not a norm plan");
    if (p->algo == MM_ALGO_EMPTY) return MM_OK;
    const mm_norm_desc &d = p->norm;
    const bool block = d.has_block != 0, pre = d.pre_norm != MM_NORM_NONE;
    mm_status st = operand("residual", true, f->residual);
    if (st == MM_OK) st = operand("block", block, f->block);
    if (st == MM_OK) st = operand("gate", d.gate_rows > 0, f->gate);
    if (st == MM_OK) st = operand("post_weight", d.post_weight != 0, f->post_weight);
    if (st == MM_OK) st = operand("post_bias", d.post_bias != 0, f->post_bias);
    if (st == MM_OK) st = operand("pre_weight", d.pre_weight != 0, f->pre_weight);
    if (st == MM_OK) st = operand("pre_bias", d.pre_bias != 0, f->pre_bias);
    if (st == MM_OK) st = operand("out", pre, f->out);
    if (st == MM_OK && f->stats) st = operand("stats", p->training, f->stats);
    if (st == MM_OK && f->sum_f32) st = operand("sum_f32", p->training && d.kept_type == MM_FLOAT, f->sum_f32);
    if (st == MM_OK) st = checkpoint_pair(p, "sum", true, f->sum_q, f->sum_scale);
    if (st == MM_OK) st = checkpoint_pair(p, "block", block, f->block_q, f->block_scale);
    if (st == MM_OK) st = checkpoint_pair(p, "out", pre, f->out_q, f->out_scale);
    if (st != MM_OK) return st;
    NormFwdTrain a;
    memset(&a, 0, sizeof(a));
    a.X = f->residual;
    a.B = f->block;
    a.gate = f->gate;
    a.w1 = f->post_weight;
    a.b1 = f->post_bias;
    a.w2 = f->pre_weight;
    a.b2 = f->pre_bias;
    a.R = f->sum;
    a.Y = f->out;
    a.M = (int32_t)p->M;
    a.N = (int32_t)p->N;
    a.gate_rows = (int32_t)d.gate_rows;
    a.alpha = d.residual_scale;
    a.eps1 = d.post_eps;
    a.eps2 = d.pre_eps;
    a.post = (uint8_t)d.post_norm;
    a.pre = (uint8_t)d.pre_norm;
    a.stats = f->stats;
    a.r32 = f->sum_f32;
    a.rq = f->sum_q;
    a.rs = f->sum_scale;
    a.bq = f->block_q;
    a.bs = f->block_scale;
    a.yq = f->out_q;
    a.ys = f->out_scale;
    const bool train = a.stats || a.r32 || a.rq || a.bq || a.yq;
    return launched(launch_norm_fwd(p->dtype, train, a, (hipStream_t)stream));
}

mm_status mm_norm_backward(mm_plan_t p, const mm_norm_backward_args *b, void *stream) {
    clear_error();
    if (!p || !b) return fail(MM_ERR_NULL_ARG, "plan or args is NULL");
    if (!p->is_norm) return fail(MM_ERR_BAD_OPTION, "not a norm plan");
    if (!p->training) return fail(MM_ERR_BAD_OPTION, "the plan was created without training");
    const mm_norm_desc &d = p->norm;
    const bool pre = d.pre_norm != MM_NORM_NONE, post = d.post_norm != MM_NORM_NONE, gate = d.gate_rows > 0;
    const bool k8 = p->kept == MM_INT8;
    mm_status st = MM_OK;
    const struct { const char *name; bool has; const void *given; } wanted[] = {
        {"dblock", d.has_block != 0, b->dblock}, {"dgate", gate, b->dgate},
        {"dpost_weight", d.post_weight != 0, b->dpost_weight}, {"dpost_bias", d.post_bias != 0, b->dpost_bias},
        {"dpre_weight", d.pre_weight != 0, b->dpre_weight}, {"dpre_bias", d.pre_bias != 0, b->dpre_bias}};
    for (const auto &w : wanted)
        if (st == MM_OK && w.given) st = operand(w.name, w.has, w.given);
    if (st != MM_OK) return st;
    if (!b->dresidual && !b->dblock && !b->dgate && !b->dpost_weight && !b->dpost_bias && !b->dpre_weight && !b->dpre_bias)
        return MM_OK;
    if (p->N == 0) return MM_OK;
    const bool to_block = b->dblock || b->dgate || b->dpost_weight || b->dpost_bias;
    const bool read_b = to_block && (post || b->dgate);
    if (p->M > 0) {
        if (!b->stats) return fail(MM_ERR_NULL_ARG, "stats is NULL");
        if (pre && (!b->sum || (k8 && !b->sum_scale))) return fail(MM_ERR_NULL_ARG, "sum or sum_scale is NULL");
        if (read_b && (!b->block || (k8 && !b->block_scale))) return fail(MM_ERR_NULL_ARG, "block or block_scale is NULL");
        if (!k8 && (b->sum_scale || b->block_scale)) return fail(MM_ERR_BAD_OPTION, "scales go with checkpoints");
        st = operand("gate", gate, b->gate);
        if (st == MM_OK) st = operand("post_weight", d.post_weight != 0, b->post_weight);
        if (st == MM_OK && (b->post_bias || b->dgate)) st = operand("post_bias", d.post_bias != 0, b->post_bias);
        if (st == MM_OK) st = operand("pre_weight", d.pre_weight != 0, b->pre_weight);
        if (st == MM_OK) st = operand("dout", pre, b->dout);
        if (st == MM_OK && !pre) st = operand("dsum", true, b->dsum);
        if (st != MM_OK) return st;
    }
    if (p->workspace_bytes > 0) {
        st = alloc_workspace(p, false);
        if (st != MM_OK) return st;
    }
    NormBwd a;
    memset(&a, 0, sizeof(a));
    NormJoin j;
    memset(&j, 0, sizeof(j));
    deal_rows(p, &a.per, &a.workers);
    a.stats = b->stats;
    if (pre) {
        a.R = b->sum;
        a.rs = b->sum_scale;
        a.w2 = b->pre_weight;
        a.dY = b->dout;
    }
    if (read_b) {
        a.B = b->block;
        a.bs = b->block_scale;
    }
    a.gate = b->gate;
    a.w1 = b->post_weight;
    a.b1 = b->dgate ? b->post_bias : nullptr;
    a.dS = b->dsum;
    a.dX = b->dresidual;
    a.dB = b->dblock;
    a.dgate = b->dgate;
    a.ldp = round_up(p->N, 4);
    a.M = (int32_t)p->M;
    a.N = (int32_t)p->N;
    a.gate_rows = (int32_t)d.gate_rows;
    a.alpha = d.residual_scale;
    a.post = (uint8_t)d.post_norm;
    a.pre = (uint8_t)d.pre_norm;
    a.part = (float *)p->ws;
    a.gpart = b->dgate && shared_groups(p, a.per) ? (float *)((char *)p->ws + p->s_off) : nullptr;
    void *const sums[4] = {b->dpost_weight, b->dpre_weight, b->dpost_bias, b->dpre_bias};
    for (int k = 0; k < 4; ++k) {
        a.slot[k] = -1;
        if (!sums[k]) continue;
        j.out[a.jobs] = sums[k];
        a.slot[k] = (int8_t)a.jobs++;
    }
    j.part = a.part;
    j.gpart = a.gpart;
    j.ldp = a.ldp;
    j.M = a.M;
    j.N = a.N;
    j.gate_rows = a.gate_rows;
    j.per = a.per;
    j.workers = a.workers;
    j.jobs = a.jobs;
    j.groups = gate ? (int32_t)cdiv(p->M, d.gate_rows) : 0;
    j.dgate = b->dgate;
    hipStream_t s = (hipStream_t)stream;
    st = launched(launch_norm_bwd(p->dtype, p->kept, a, s));
    if (st == MM_OK) st = launched(launch_norm_join(p->dtype, j, s));
    return st;
}

}  // extern "C"
