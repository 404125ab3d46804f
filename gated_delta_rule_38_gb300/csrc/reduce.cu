// Sums of partial rows: the second step of every parameter gradient.  Kernels that sum over tokens leave one partial
// row a block; these are added in a fixed order, so that the same call gives the same bits.
#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"

namespace gdr {
namespace {

struct ReduceArgs {
    const float *part;
    long long parts, stride;
    int cols;            // of all outputs
    RowSums out[3];
};

// 32 columns a block; its eight warps take every eighth row, four loads in flight each.  (304 rows of 4096: 8 us with the launch,
// which sixteen loads in flight do not shorten.)
template <typename T>
__global__ void __launch_bounds__(256) reduce_rows_kernel(const ReduceArgs a, bool out_f32) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int c = blockIdx.x * 32 + lane;
    float x = 0.f;
    if (c < a.cols) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        long long i = warp;
        for (; i + 24 < a.parts; i += 32) {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] += a.part[(i + 8 * k) * a.stride + c];
        }
        for (; i < a.parts; i += 8) p[0] += a.part[i * a.stride + c];
        x = (p[0] + p[1]) + (p[2] + p[3]);
    }
    s[warp][lane] = x;
    __syncthreads();
    if (warp != 0 || c >= a.cols) return;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) y += s[k][lane];
#pragma unroll
    for (int o = 0; o < 3; ++o) {
        if (c >= 0 && c < a.out[o].cols) {
            if (out_f32)
                static_cast<float *>(a.out[o].to)[c] = y;
            else
                static_cast<T *>(a.out[o].to)[c] = Elt<T>::from_f(y);
        }
        c -= a.out[o].cols;
    }
}

}  // namespace

cudaError_t launch_reduce_rows(const float *part, long long parts, long long stride, const RowSums *out, int outs,
                               bool bf16, bool out_f32, cudaStream_t s) {
    ReduceArgs a = {};
    a.part = part, a.parts = parts, a.stride = stride;
    for (int i = 0; i < outs; ++i) {
        a.out[i] = out[i];
        a.cols += out[i].cols;
    }
    const dim3 grid((unsigned)((a.cols + 31) / 32));
    if (bf16) return launch_plain(reduce_rows_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, a, out_f32);
    return launch_plain(reduce_rows_kernel<__half>, grid, dim3(256), 0, s, a, out_f32);
}

}  // namespace gdr
