// Entry points of the gated norm and the block norm: checks, the choice of form and workspaces.
#include "rownorm.h"

namespace gdr {
namespace rownorm {
namespace {

// How the rows are spread, staged and walked.  A block keeps two rows' places (one on its way while the other is worked on)
// where both fit; the grid is what is resident at once.  Shifted rows: the same number of blocks for each remainder.
int period_of(int D) {
    int p = 8;
    while (p > 1 && D % 2 == 0) p /= 2, D /= 2;
    return D % 8 == 0 ? 1 : p;
}
// A row's threads: with 16 columns each (32 for the widest rows) the power of two up to 32 that covers it, or a multiple of 32;
// short rows share a block of at most 256.
norm::NormShape shape_of(int D) {
    norm::NormShape s = {};
    const int vectors = (D % 8 ? D + 7 : D) / 8 + (D % 8 && (D + 7) % 8 ? 1 : 0);
    s.nv = vectors <= 1024 ? 2 : 4;
    const int need = (vectors + s.nv - 1) / s.nv;
    s.tpr = 8;
    while (s.tpr < 32 && s.tpr < need) s.tpr *= 2;
    if (need > 32) s.tpr = (need + 31) / 32 * 32;
    s.rpb = s.tpr < 256 ? 256 / s.tpr : 1;
    s.threads = s.tpr * s.rpb;
    return s;
}
// Blocks an SM, as the forms' launch bounds have it: two of 256 threads, but three of the gated norm's forward and of
// whole-vector forwards; of smaller blocks as many more (8192 x 2560, gated norm's backward: 62 us with two of 160, 54 so).
// Of more threads one.  (Whole-vector forwards take 80 to 96 registers, which would leave room for a second block of up to 384
// threads, but their form is one for up to 512: 8192 rows of 4096 columns take 34 us in the gated norm's forward, of 4104 58.)
// Shifted rows have a form of 320 threads, two an SM with 96 registers (one of 288 with 112 is 4 % faster up to 4600 columns
// and a quarter slower from there to 5112, where one block is left).  Four vectors a thread: one block of any size, with 104 to
// 128 registers (two of 288 threads, which do not fit, as the grid: 4096 x 8193, gated norm's backward 174 us, 167 so).
int blocks_an_sm(const norm::NormShape &s, bool shift, bool two) {
    if (s.threads > 256) return s.nv == 2 && shift && s.threads <= 320 ? 2 : 1;
    return (two ? 2 : 3) * 256 / s.threads;
}
RowForm form_of(RowArgs *a, bool bwd, bool gated) {
    RowForm f = {};
    f.shift = a->D % 8 != 0;
    f.s = shape_of(a->D);
    size_t place = 0;
    for (const RowIn &in : a->in)
        if (in.p) place += (size_t)f.s.nv * f.s.threads * 8 * in.elem;
    const size_t all = 227 * 1024;
    const int most = blocks_an_sm(f.s, f.shift, bwd || (f.shift && !gated));
    auto resident = [&](size_t smem) {
        const int n = (int)(all / (smem + 2048));
        return n < most ? n : most;
    };
    a->stages = resident(2 * place) >= 1 ? 2 : 1;
    f.smem = a->stages * place;
    a->tpr = f.s.tpr, a->rpb = f.s.rpb, a->place = (int)place, a->period = period_of(a->D);
    const long long each = (a->rows + a->period - 1) / a->period, need = (each + f.s.rpb - 1) / f.s.rpb * a->period;
    const long long at_once = (long long)kSMs * resident(f.smem) / a->period * a->period;
    f.blocks = (int)(need < at_once ? need : at_once);
    return f;
}

// Partial rows of the parameters' gradients: at most this many blocks.
size_t parts_bytes(long long rows, int D, int outs) {
    const norm::NormShape s = shape_of(D);
    const int period = period_of(D);
    const long long each = (rows + period - 1) / period, need = (each + s.rpb - 1) / s.rpb * period, at_once = (long long)kSMs * blocks_an_sm(s, D % 8 != 0, true);
    return round_up((size_t)(need < at_once ? need : at_once) * outs * D * sizeof(float), 256);
}

// Rows of whole vectors, or tensors without gaps.
bool rows_ok(int D, int64_t ld, int64_t wide) { return D % 8 == 0 ? ld % 8 == 0 : ld == wide; }
bool width_ok(int D) { return D >= 1 && D <= (D % 8 ? GDR_NORM_MAX_D - 8 : GDR_NORM_MAX_D); }

gdr_status check_gated(const gdr_gated_norm_problem *p) {
    if (!p) return GDR_ERR_NULL;
    if (p->tokens < 0 || p->heads < 1 || !width_ok(p->D) || p->tokens > ((int64_t)1 << 40) / p->heads) return GDR_ERR_SHAPE;
    const int64_t wide = (int64_t)p->heads * p->D;
    if (p->x_ld < wide || p->gate_ld < wide) return GDR_ERR_SHAPE;
    if (!is_half(p->dtype) || (p->weight_dtype != p->dtype && p->weight_dtype != GDR_FP32)) return GDR_ERR_DTYPE;
    if (p->gate_act != GDR_GATE_SIGMOID && p->gate_act != GDR_GATE_SILU) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}
gdr_status check_block(const gdr_block_norm_problem *p) {
    if (!p) return GDR_ERR_NULL;
    if (p->rows < 0 || p->rows > ((int64_t)1 << 40) || !width_ok(p->D) || p->x_ld < p->D || p->gate_ld < p->D) return GDR_ERR_SHAPE;
    if (!is_half(p->dtype) || (p->weight_dtype != p->dtype && p->weight_dtype != GDR_FP32) ||
        (p->residual_dtype != p->dtype && p->residual_dtype != GDR_FP32))
        return GDR_ERR_DTYPE;
    if (p->gate_act != GDR_GATE_RAW && p->gate_act != GDR_GATE_SIGMOID && p->gate_act != GDR_GATE_SILU) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}
int act_of(unsigned gate_act) { return gate_act == GDR_GATE_SIGMOID ? ACT_SIGMOID : gate_act == GDR_GATE_SILU ? ACT_SILU : ACT_RAW; }
// Rows of all heads at one stride where the tokens follow one another.
RowIn heads_in(const void *p, int64_t ld, int heads, int D) {
    if (ld == (int64_t)heads * D) return {p, D, 1, 2};
    return {p, ld, heads, 2};
}
// An output over rows that other threads still read.
bool over(const void *out, size_t rows, size_t width, const void *in, size_t in_ld) { return touches(out, rows * width, in, rows, width, in_ld); }

}  // namespace
}  // namespace rownorm
}  // namespace gdr

using namespace gdr;
using namespace gdr::rownorm;

extern "C" {

gdr_status gdr_gated_norm_fwd(const gdr_gated_norm_problem *p, const void *x, const void *gate, const void *weight, void *y, void *stream) {
    gdr_status st = check_gated(p);
    if (st != GDR_OK) return st;
    if (p->tokens == 0) return GDR_OK;
    if (!x || !gate || !weight || !y) return GDR_ERR_NULL;
    const int64_t row = (int64_t)p->heads * p->D;
    if (!aligned16(x) || !aligned16(gate) || !aligned16(y) || !aligned16(weight) || !rows_ok(p->D, p->x_ld, row) || !rows_ok(p->D, p->gate_ld, row))
        return GDR_ERR_ALIGN;
    const size_t wide = (size_t)p->heads * p->D * 2;
    if (over(y, p->tokens, wide, x, p->x_ld * 2) || over(y, p->tokens, wide, gate, p->gate_ld * 2) ||
        overlap(y, p->tokens * wide, weight, p->D * esize(p->weight_dtype)))
        return GDR_ERR_UNSUPPORTED;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    RowArgs a = {};
    a.in[IN_X] = heads_in(x, p->x_ld, p->heads, p->D), a.in[IN_GATE] = heads_in(gate, p->gate_ld, p->heads, p->D);
    a.w = weight, a.y = y, a.rows = p->tokens * p->heads, a.D = p->D, a.eps = p->eps;
    a.w_f32 = p->weight_dtype == GDR_FP32, a.act = act_of(p->gate_act);
    RowForm f = form_of(&a, false, true);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return timed(K_GATED_FWD, cs, [&] { return p->dtype == GDR_BF16 ? gated_fwd_bf16(a, f, cs) : gated_fwd_fp16(a, f, cs); });
}

gdr_status gdr_gated_norm_bwd_workspace_size(const gdr_gated_norm_problem *p, size_t *bytes) {
    const gdr_status st = check_gated(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    *bytes = parts_bytes(p->tokens * p->heads, p->D, 1);
    return GDR_OK;
}

gdr_status gdr_gated_norm_bwd(const gdr_gated_norm_problem *p, const void *x, const void *gate, const void *weight, const void *dy,
                              void *dx, void *dgate, void *dweight, void *workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0;
    gdr_status st = gdr_gated_norm_bwd_workspace_size(p, &need);
    if (st != GDR_OK) return st;
    if (!weight || !dweight || (p->tokens && (!x || !gate || !dy || !dx || !dgate))) return GDR_ERR_NULL;
    const int64_t row = (int64_t)p->heads * p->D;
    if (!aligned16(x) || !aligned16(gate) || !aligned16(dy) || !aligned16(dx) || !aligned16(dgate) || !aligned16(weight) ||
        !aligned_to(dweight, esize(p->weight_dtype)) || !rows_ok(p->D, p->x_ld, row) || !rows_ok(p->D, p->gate_ld, row))
        return GDR_ERR_ALIGN;
    const size_t wide = (size_t)p->heads * p->D * 2, all = p->tokens * wide, wb = p->D * esize(p->weight_dtype);
    const void *outs[] = {dx, dgate, dweight};
    const size_t sizes[] = {all, all, wb};
    for (int i = 0; i < 3; ++i) {
        const void *o = outs[i];
        const size_t n = sizes[i];
        if (touches(o, n, x, p->tokens, wide, p->x_ld * 2) || touches(o, n, gate, p->tokens, wide, p->gate_ld * 2) || overlap(o, n, dy, all) ||
            overlap(o, n, weight, wb))
            return GDR_ERR_UNSUPPORTED;
        for (int k = 0; k < i; ++k)
            if (overlap(o, n, outs[k], sizes[k])) return GDR_ERR_UNSUPPORTED;
    }
    if (need && (!workspace || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    if (need && !aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->tokens == 0) return cuda_status(cudaMemsetAsync(dweight, 0, (size_t)p->D * esize(p->weight_dtype), cs));
    RowArgs a = {};
    a.in[IN_X] = heads_in(x, p->x_ld, p->heads, p->D), a.in[IN_GATE] = heads_in(gate, p->gate_ld, p->heads, p->D), a.in[IN_DY] = {dy, p->D, 1, 2};
    a.w = weight, a.dx = dx, a.dgate = dgate, a.rows = p->tokens * p->heads, a.D = p->D, a.eps = p->eps;
    a.part = static_cast<float *>(workspace);
    a.w_f32 = p->weight_dtype == GDR_FP32, a.act = act_of(p->gate_act);
    RowForm f = form_of(&a, true, true);
    st = timed(K_GATED_BWD, cs, [&] { return p->dtype == GDR_BF16 ? gated_bwd_bf16(a, f, cs) : gated_bwd_fp16(a, f, cs); });
    if (st != GDR_OK) return st;
    return timed(K_REDUCE, cs, [&] {
        const RowSums out = {dweight, p->D};
        return launch_reduce_rows(a.part, f.blocks, p->D, &out, 1, p->dtype == GDR_BF16, a.w_f32, cs);
    });
}

gdr_status gdr_block_norm_fwd(const gdr_block_norm_problem *p, const void *x, const void *residual, const void *weight,
                              const void *post_weight, const void *gate, void *y, void *residual_out, void *stream) {
    gdr_status st = check_block(p);
    if (st != GDR_OK) return st;
    if (p->rows == 0) return GDR_OK;
    if (!x || !residual || !weight || !y || !residual_out) return GDR_ERR_NULL;
    const size_t rs = esize(p->residual_dtype), n = (size_t)p->rows, D = p->D, wb = D * esize(p->weight_dtype);
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(post_weight) || !aligned16(gate) || !aligned16(y) ||
        !aligned16(residual_out) || !rows_ok(p->D, p->x_ld, p->D) || (gate && !rows_ok(p->D, p->gate_ld, p->D)))
        return GDR_ERR_ALIGN;
    // (residual_out may be the residual itself: a thread writes what only it has read; not another overlap of the two)
    if (over(y, n, 2 * D, x, p->x_ld * 2) || over(y, n, 2 * D, gate, p->gate_ld * 2) || overlap(y, n * 2 * D, residual, n * rs * D) ||
        overlap(y, n * 2 * D, residual_out, n * rs * D) || over(residual_out, n, rs * D, x, p->x_ld * 2) ||
        over(residual_out, n, rs * D, gate, p->gate_ld * 2) ||
        (residual_out != residual && overlap(residual_out, n * rs * D, residual, n * rs * D)) || overlap(y, n * 2 * D, weight, wb) ||
        overlap(y, n * 2 * D, post_weight, wb) || overlap(residual_out, n * rs * D, weight, wb) || overlap(residual_out, n * rs * D, post_weight, wb))
        return GDR_ERR_UNSUPPORTED;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    RowArgs a = {};
    a.in[IN_X] = {x, p->x_ld, 1, 2}, a.in[IN_RES] = {residual, p->D, 1, (int)rs};
    if (gate) a.in[IN_GATE] = {gate, p->gate_ld, 1, 2};
    a.w = weight, a.pw = post_weight, a.y = y, a.res_out = residual_out, a.rows = p->rows, a.D = p->D;
    a.eps = p->eps, a.rscale = p->residual_scale, a.w_f32 = p->weight_dtype == GDR_FP32, a.act = gate ? act_of(p->gate_act) : ACT_NONE;
    RowForm f = form_of(&a, false, false);
    f.f32 = p->residual_dtype == GDR_FP32, f.gate = gate != nullptr;
    a.wide = aligned_to(residual_out, 32);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return timed(K_BLOCK_FWD, cs, [&] { return p->dtype == GDR_BF16 ? block_fwd_bf16(a, f, cs) : block_fwd_fp16(a, f, cs); });
}

gdr_status gdr_block_norm_bwd_workspace_size(const gdr_block_norm_problem *p, size_t *bytes) {
    const gdr_status st = check_block(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    *bytes = parts_bytes(p->rows, p->D, 2);
    return GDR_OK;
}

gdr_status gdr_block_norm_bwd(const gdr_block_norm_problem *p, const void *x, const void *h, const void *weight, const void *post_weight,
                              const void *gate, const void *dy, const void *dresidual, void *dx, void *dresidual_in, void *dweight,
                              void *dpost_weight, void *dgate, void *workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0;
    gdr_status st = gdr_block_norm_bwd_workspace_size(p, &need);
    if (st != GDR_OK) return st;
    if (!weight || !dweight || ((post_weight != nullptr) != (dpost_weight != nullptr))) return GDR_ERR_NULL;
    if (p->rows && (!x || !h || !dy || !dx || !dresidual_in || ((gate != nullptr) != (dgate != nullptr)))) return GDR_ERR_NULL;
    const size_t rs = esize(p->residual_dtype), ws = esize(p->weight_dtype), n = (size_t)p->rows, D = p->D;
    if (!aligned16(x) || !aligned16(h) || !aligned16(weight) || !aligned16(post_weight) || !aligned16(gate) || !aligned16(dy) ||
        !aligned16(dresidual) || !aligned16(dx) || !aligned16(dresidual_in) || !aligned16(dgate) || !aligned_to(dweight, ws) ||
        !aligned_to(dpost_weight, ws) || !rows_ok(p->D, p->x_ld, p->D) || (gate && !rows_ok(p->D, p->gate_ld, p->D)))
        return GDR_ERR_ALIGN;
    const void *outs[] = {dx, dresidual_in, dgate, dweight, dpost_weight};
    const size_t sizes[] = {n * 2 * D, n * rs * D, n * 2 * D, D * ws, D * ws};
    for (int i = 0; i < 5; ++i) {
        const void *o = outs[i];
        const size_t b = sizes[i];
        if (touches(o, b, x, n, 2 * D, p->x_ld * 2) || touches(o, b, gate, n, 2 * D, p->gate_ld * 2) || overlap(o, b, h, n * rs * D) ||
            overlap(o, b, dy, n * 2 * D) || overlap(o, b, dresidual, n * rs * D) || overlap(o, b, weight, D * ws) || overlap(o, b, post_weight, D * ws))
            return GDR_ERR_UNSUPPORTED;
        for (int k = 0; k < i; ++k)
            if (overlap(o, b, outs[k], sizes[k])) return GDR_ERR_UNSUPPORTED;
    }
    if (need && (!workspace || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    if (need && !aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->rows == 0) {
        st = cuda_status(cudaMemsetAsync(dweight, 0, D * ws, cs));
        return st == GDR_OK && dpost_weight ? cuda_status(cudaMemsetAsync(dpost_weight, 0, D * ws, cs)) : st;
    }
    RowArgs a = {};
    a.in[IN_X] = {x, p->x_ld, 1, 2}, a.in[IN_H] = {h, p->D, 1, (int)rs}, a.in[IN_DY] = {dy, p->D, 1, 2};
    if (gate) a.in[IN_GATE] = {gate, p->gate_ld, 1, 2};
    if (dresidual) a.in[IN_DRES] = {dresidual, p->D, 1, (int)rs};
    a.w = weight, a.pw = post_weight, a.dx = dx, a.dres = dresidual_in, a.dgate = dgate, a.rows = p->rows, a.D = p->D;
    a.part = static_cast<float *>(workspace);
    a.eps = p->eps, a.rscale = p->residual_scale, a.w_f32 = p->weight_dtype == GDR_FP32, a.act = gate ? act_of(p->gate_act) : ACT_NONE;
    RowForm f = form_of(&a, true, false);
    f.f32 = p->residual_dtype == GDR_FP32, f.gate = gate != nullptr;
    a.wide = aligned_to(dresidual_in, 32);
    st = timed(K_BLOCK_BWD, cs, [&] { return p->dtype == GDR_BF16 ? block_bwd_bf16(a, f, cs) : block_bwd_fp16(a, f, cs); });
    if (st != GDR_OK) return st;
    return timed(K_REDUCE, cs, [&] {
        const RowSums out[2] = {{dweight, p->D}, {dpost_weight, p->D}};
        const int outs = post_weight ? 2 : 1;
        return launch_reduce_rows(a.part, f.blocks, (long long)outs * p->D, out, outs, p->dtype == GDR_BF16, a.w_f32, cs);
    });
}

}  // extern "C"
