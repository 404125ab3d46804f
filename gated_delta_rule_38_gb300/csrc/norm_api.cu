// Entry points of the RMS norm: checks, the choice of form and workspaces.
#include "norm.h"

namespace gdr {
namespace norm {
namespace {

gdr_status check_norm(const gdr_norm_problem *p) {
    if (!p) return GDR_ERR_NULL;
    if (p->rows < 0 || p->D < 1 || p->D > GDR_NORM_MAX_D || p->x_ld < p->D) return GDR_ERR_SHAPE;
    if (p->scale_group != 0 && p->scale_group != 128) return GDR_ERR_SHAPE;
    if (!is_half(p->dtype)) return GDR_ERR_DTYPE;
    if (p->weight_dtype != p->dtype && p->weight_dtype != GDR_FP32) return GDR_ERR_DTYPE;
    if (p->residual_dtype != p->dtype && p->residual_dtype != GDR_FP32) return GDR_ERR_DTYPE;
    if (p->y_dtype != p->dtype && p->y_dtype != GDR_E4M3) return GDR_ERR_DTYPE;
    return GDR_OK;
}

// Every pointer that is given is aligned to its elements; `vec` is cleared unless all allow 16-byte accesses.
bool norm_ptr(const void *p, size_t elem, size_t vec_bytes, bool *vec) {
    if (!p) return true;
    if (!aligned_to(p, elem)) return false;
    if (!aligned_to(p, vec_bytes)) *vec = false;
    return true;
}

}  // namespace
}  // namespace norm
}  // namespace gdr

using namespace gdr;
using namespace gdr::norm;

extern "C" {

gdr_status gdr_norm_fwd(const gdr_norm_problem *p, const void *x, const void *weight, const void *residual, void *y,
                        void *residual_out, float *scale, void *stream) {
    gdr_status st = check_norm(p);
    if (st != GDR_OK) return st;
    const bool quant = p->y_dtype == GDR_E4M3;
    if (p->rows == 0) return GDR_OK;
    if (!x || !weight || !y || (quant && !scale) || ((residual != nullptr) != (residual_out != nullptr)))
        return GDR_ERR_NULL;
    bool vec = p->D % 8 == 0 && p->x_ld % 8 == 0;
    const size_t rs = esize(p->residual_dtype);
    if (!norm_ptr(x, 2, 16, &vec) || !norm_ptr(weight, esize(p->weight_dtype), 16, &vec) ||
        !norm_ptr(residual, rs, 16, &vec) || !norm_ptr(residual_out, rs, 16, &vec) ||
        !norm_ptr(y, quant ? 1 : 2, quant ? 8 : 16, &vec) || !norm_ptr(scale, 4, 4, &vec))
        return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    NormArgs a = {};
    a.x = x, a.w = weight, a.res = residual, a.y = y, a.res_out = residual_out, a.scale = scale;
    a.rows = p->rows, a.x_ld = p->x_ld, a.D = p->D, a.eps = p->eps;
    a.group = p->scale_group;
    a.nscale = p->scale_group ? (p->D + 127) / 128 : 1;
    a.w_f32 = p->weight_dtype == GDR_FP32;
    const int res = !residual ? RES_NONE : p->residual_dtype == GDR_FP32 ? RES_F32 : RES_HALF;
    const NormShape s = norm_shape(p->D, !vec);
    a.tpr = s.tpr;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return timed(K_NORM_FWD, cs, [&] {
        return p->dtype == GDR_BF16 ? norm_fwd_bf16(a, s, vec, quant, res, cs) : norm_fwd_fp16(a, s, vec, quant, res, cs);
    });
}

gdr_status gdr_norm_bwd_workspace_size(const gdr_norm_problem *p, size_t *bytes) {
    gdr_status st = check_norm(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    // (covers both forms, whose blocks take different numbers of rows)
    size_t parts = 0;
    for (bool rag : {false, true}) {
        const NormShape s = norm_shape(p->D, rag);
        const size_t n = p->rows ? (size_t)norm_blocks(p->rows, s, true, rag) : 0;
        parts = n > parts ? n : parts;
    }
    *bytes = round_up(parts * p->D * sizeof(float), 256);
    return GDR_OK;
}

gdr_status gdr_norm_bwd(const gdr_norm_problem *p, const void *h, const void *weight, const void *dy,
                        const void *dresidual, void *dx, float *dresidual_in, void *dweight, void *workspace,
                        size_t workspace_bytes, void *stream) {
    size_t need = 0;
    gdr_status st = gdr_norm_bwd_workspace_size(p, &need);
    if (st != GDR_OK) return st;
    if (!weight || !dweight || (p->rows && (!h || !dy || !dx))) return GDR_ERR_NULL;
    const bool f32 = p->residual_dtype == GDR_FP32;
    if (dresidual_in && !f32) return GDR_ERR_DTYPE;
    bool vec = p->D % 8 == 0 && p->x_ld % 8 == 0;
    if (!norm_ptr(h, f32 ? 4 : 2, 16, &vec) || !norm_ptr(weight, esize(p->weight_dtype), 16, &vec) ||
        !norm_ptr(dy, 2, 16, &vec) || !norm_ptr(dresidual, f32 ? 4 : 2, 16, &vec) || !norm_ptr(dx, 2, 16, &vec) ||
        !norm_ptr(dresidual_in, 4, 16, &vec) || !norm_ptr(dweight, esize(p->weight_dtype), 4, &vec))
        return GDR_ERR_ALIGN;
    if (need && (!workspace || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    if (need && !aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->rows == 0) return cuda_status(cudaMemsetAsync(dweight, 0, (size_t)p->D * esize(p->weight_dtype), cs));
    NormArgs a = {};
    a.x = h, a.w = weight, a.dy = dy, a.res = dresidual, a.dx = dx, a.dres = dresidual_in;
    a.dw_part = static_cast<float *>(workspace);
    a.rows = p->rows, a.x_ld = p->x_ld, a.D = p->D, a.eps = p->eps;
    a.w_f32 = p->weight_dtype == GDR_FP32;
    const NormShape s = norm_shape(p->D, !vec);
    a.tpr = s.tpr;
    const int blocks = norm_blocks(p->rows, s, true, !vec);
    st = timed(K_NORM_BWD, cs, [&] {
        return p->dtype == GDR_BF16 ? norm_bwd_bf16(a, s, vec, f32, blocks, cs) : norm_bwd_fp16(a, s, vec, f32, blocks, cs);
    });
    if (st != GDR_OK) return st;
    return timed(K_REDUCE, cs, [&] {
        const RowSums out = {dweight, p->D};
        return launch_reduce_rows(a.dw_part, blocks, p->D, &out, 1, p->dtype == GDR_BF16, a.w_f32, cs);
    });
}

}  // extern "C"
