// What the gated norm's and the block norm's entry points share with their kernels.
#pragma once

#include <cuda_runtime.h>

#include "norm.h"

namespace gdr {
namespace rownorm {

enum { ACT_NONE = 0, ACT_RAW = 1, ACT_SIGMOID = 2, ACT_SILU = 3 };

// A tensor of rows: row r at (r / heads) ld + (r mod heads) D elements.
struct RowIn {
    const void *p;
    long long ld;
    int heads;
    int elem;  // bytes an element, 2 or 4 (p null: not given)
};

constexpr int kMaxIn = 5;
struct RowArgs {
    RowIn in[kMaxIn];
    const void *w, *pw;           // [D]; pw nullable
    void *y, *res_out;            // forward
    void *dx, *dgate, *dres;      // backward
    float *part;                  // [blocks][D or 2 D]: dw, then dpw
    long long rows;
    int D, tpr, rpb, stages, act;
    int place, period;            // bytes of a stage; rows after which the first element lies as far into a vector again
    bool wide;                    // fp32 outputs begin on 32-byte boundaries
    bool w_f32;
    float eps, rscale;
};

// The inputs' places in RowArgs::in.
enum { IN_X = 0, IN_GATE = 1, IN_DY = 2, IN_H = 3, IN_DRES = 4, IN_RES = IN_H };

struct RowForm {
    norm::NormShape s;
    bool shift, f32, gate;  // rows that begin inside a vector; an fp32 residual stream; a gate
    int blocks;
    size_t smem;
};

cudaError_t gated_fwd_bf16(const RowArgs &a, const RowForm &f, cudaStream_t st);
cudaError_t gated_fwd_fp16(const RowArgs &a, const RowForm &f, cudaStream_t st);
cudaError_t gated_bwd_bf16(const RowArgs &a, const RowForm &f, cudaStream_t st);
cudaError_t gated_bwd_fp16(const RowArgs &a, const RowForm &f, cudaStream_t st);
cudaError_t block_fwd_bf16(const RowArgs &a, const RowForm &f, cudaStream_t st);
cudaError_t block_fwd_fp16(const RowArgs &a, const RowForm &f, cudaStream_t st);
cudaError_t block_bwd_bf16(const RowArgs &a, const RowForm &f, cudaStream_t st);
cudaError_t block_bwd_fp16(const RowArgs &a, const RowForm &f, cudaStream_t st);

}  // namespace rownorm
}  // namespace gdr
