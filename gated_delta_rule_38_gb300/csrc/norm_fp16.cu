// The norm's kernels for fp16 data (one translation unit a type: they compile side by side).
#include "norm.cuh"

namespace gdr {
namespace norm {

cudaError_t norm_fwd_fp16(const NormArgs &a, const NormShape &s, bool vec, bool quant, int res, cudaStream_t st) {
    return norm_fwd_t<__half>(a, s, vec, quant, res, st);
}
cudaError_t norm_bwd_fp16(const NormArgs &a, const NormShape &s, bool vec, bool f32, int blocks, cudaStream_t st) {
    return norm_bwd_t<__half>(a, s, vec, f32, blocks, st);
}

}  // namespace norm
}  // namespace gdr
