// The gated norm's kernels in fp16.
#include "rownorm.cuh"

namespace gdr {
namespace rownorm {
namespace {
using T = __half;
}
cudaError_t gated_fwd_fp16(const RowArgs &a, const RowForm &f, cudaStream_t st) { GDR_ROW_FORMS(gated_fwd_kernel, ); }
cudaError_t gated_bwd_fp16(const RowArgs &a, const RowForm &f, cudaStream_t st) { GDR_ROW_FORMS(gated_bwd_kernel, ); }

}  // namespace rownorm
}  // namespace gdr
