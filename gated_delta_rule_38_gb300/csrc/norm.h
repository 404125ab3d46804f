// What the norm's entry points and its kernels share.
#pragma once

#include <cuda_runtime.h>

#include "host.h"

namespace gdr {
namespace norm {

enum { RES_NONE = 0, RES_HALF = 1, RES_F32 = 2 };

struct NormArgs {
    const void *x, *w, *res;
    void *y, *res_out;
    float *scale;
    const void *dy;            // backward
    void *dx, *dres;           // backward: dres only for an fp32 residual stream
    float *dw_part;            // backward: [blocks][D]
    long long rows, x_ld;
    int D, tpr, group, nscale;  // group: 0 = one scale a row
    bool w_f32;
    float eps;
};

// Threads a row: with whole vectors the power of two that covers D with 16 elements a thread (32 for rows over 8,192);
// ragged the multiple of 32 (rows of up to 128 threads share a block of at most 256).
constexpr int kNormThreads = 512;
struct NormShape {
    int tpr, nv, threads, rpb;
};
constexpr NormShape norm_shape(int D, bool rag) {
    NormShape s = {};
    s.nv = D <= 16 * kNormThreads ? 2 : 4;
    if (rag) {
        s.tpr = (D + s.nv * 8 * 32 - 1) / (s.nv * 8 * 32) * 32;
        s.rpb = s.tpr <= 128 ? 256 / s.tpr : 1;
        s.threads = s.tpr * s.rpb;
    } else {
        s.tpr = 8;
        while (s.tpr * s.nv * 8 < D) s.tpr *= 2;
        s.threads = s.tpr < 256 ? 256 : s.tpr;
        s.rpb = s.threads / s.tpr;
    }
    return s;
}

// Every width's threads cover it, fit a block and have a row: a shape without one would walk no rows and never end.
constexpr bool norm_shapes_hold(int from, int to, bool rag) {
    for (int D = from; D <= to; ++D) {
        const NormShape s = norm_shape(D, rag);
        if (s.rpb < 1 || s.threads != s.tpr * s.rpb || s.threads > kNormThreads || s.tpr * s.nv * 8 < D || (rag && s.tpr % 32)) return false;
    }
    return true;
}
static_assert(norm_shapes_hold(1, GDR_NORM_MAX_D, false) && norm_shapes_hold(1, GDR_NORM_MAX_D, true), "norm shapes");

// Blocks: at most as many as are resident at once; each walks rows, with its weights at hand and its next row's loads
// in flight.
inline int norm_blocks(long long rows, const NormShape &s, bool bwd, bool rag) {
    const long long need = (rows + s.rpb - 1) / s.rpb;
    long long per = s.threads <= 256 ? (bwd ? 2 : 3) : 1;
    if (rag) per = s.threads <= 128 ? 4 : s.threads <= 192 ? 3 : s.threads <= 288 ? 2 : 1;
    const long long most = (long long)kSMs * per;
    return (int)(need < most ? need : most);
}

cudaError_t norm_fwd_bf16(const NormArgs &a, const NormShape &s, bool vec, bool quant, int res, cudaStream_t st);
cudaError_t norm_fwd_fp16(const NormArgs &a, const NormShape &s, bool vec, bool quant, int res, cudaStream_t st);
cudaError_t norm_bwd_bf16(const NormArgs &a, const NormShape &s, bool vec, bool f32, int blocks, cudaStream_t st);
cudaError_t norm_bwd_fp16(const NormArgs &a, const NormShape &s, bool vec, bool f32, int blocks, cudaStream_t st);

}  // namespace norm
}  // namespace gdr
