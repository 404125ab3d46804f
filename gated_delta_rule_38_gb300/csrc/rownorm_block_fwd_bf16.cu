// The block norm's forward kernels in bf16.
#include "rownorm.cuh"

namespace gdr {
namespace rownorm {
namespace {
using T = __nv_bfloat16;
}
cudaError_t block_fwd_bf16(const RowArgs &a, const RowForm &f, cudaStream_t st) {
    if (f.f32 && f.gate) GDR_ROW_FORMS(block_fwd_kernel, , true, true);
    if (f.f32) GDR_ROW_FORMS(block_fwd_kernel, , true, false);
    if (f.gate) GDR_ROW_FORMS(block_fwd_kernel, , false, true);
    GDR_ROW_FORMS(block_fwd_kernel, , false, false);
}

}  // namespace rownorm
}  // namespace gdr
