// The gated norm's kernels in bf16.
#include "rownorm.cuh"

namespace gdr {
namespace rownorm {
namespace {
using T = __nv_bfloat16;
}
cudaError_t gated_fwd_bf16(const RowArgs &a, const RowForm &f, cudaStream_t st) { GDR_ROW_FORMS(gated_fwd_kernel, ); }
cudaError_t gated_bwd_bf16(const RowArgs &a, const RowForm &f, cudaStream_t st) { GDR_ROW_FORMS(gated_bwd_kernel, ); }

}  // namespace rownorm
}  // namespace gdr
