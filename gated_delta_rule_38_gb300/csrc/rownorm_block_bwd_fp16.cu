// The block norm's backward kernels in fp16.
#include "rownorm.cuh"

namespace gdr {
namespace rownorm {
namespace {
using T = __half;
}
cudaError_t block_bwd_fp16(const RowArgs &a, const RowForm &f, cudaStream_t st) {
    if (f.f32 && f.gate) GDR_ROW_FORMS(block_bwd_kernel, , true, true);
    if (f.f32) GDR_ROW_FORMS(block_bwd_kernel, , true, false);
    if (f.gate) GDR_ROW_FORMS(block_bwd_kernel, , false, true);
    GDR_ROW_FORMS(block_bwd_kernel, , false, false);
}

}  // namespace rownorm
}  // namespace gdr
