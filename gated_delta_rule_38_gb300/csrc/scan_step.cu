// Selective scan for single tokens: the T tokens of every row applied one by one to its cached fp32 state, in place.
//
//   h <- exp(delta A) h + delta x B,   y = (C . h + D x) silu(z)      (delta = softplus(dt + bias) or dt + bias)
//
// Bound by HBM: 8 bytes of state a (row, channel, state) against ten of token data a (row, channel).  A channel's N
// states lie in NL = 1 .. 16 lanes side by side, four in each (one 16-byte access where N allows it), so a warp moves
// contiguous state; the sum over the states is a butterfly over those lanes.
#include "scan.cuh"

namespace gdr {
namespace scan {
namespace {

template <typename T, int NL>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanArgs a) {
    const long long ch = (long long)blockIdx.x * (256 / NL) + threadIdx.x / NL;  // channel of all rows
    const int n0 = (threadIdx.x % NL) * 4;
    const bool live = ch < (long long)a.B * a.D;
    const long long b = live ? ch / a.D : 0;
    const int d = live ? (int)(ch - b * a.D) : 0, g = d / a.Dg;
    float h[4], A2[4];
    const float *st = a.state_in + ch * a.N + n0, *ap = a.A + (long long)d * a.N + n0;
    const bool wide = a.st_vec && n0 < a.N;
    if (live && wide) {
        const float4 f = *reinterpret_cast<const float4 *>(st), e = *reinterpret_cast<const float4 *>(ap);
        h[0] = f.x, h[1] = f.y, h[2] = f.z, h[3] = f.w;
        A2[0] = e.x, A2[1] = e.y, A2[2] = e.z, A2[3] = e.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = (live && n0 + i < a.N) ? st[i] : 0.f;
            A2[i] = (live && n0 + i < a.N) ? ap[i] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] *= LOG2E;
    const float bias = (live && a.bias) ? a.bias[d] : 0.f, skip = (live && a.skip) ? a.skip[d] : 0.f;
    for (int t = 0; t < a.T; ++t) {
        const long long row = b * a.T + t;
        float x = 0.f, dl = 0.f, z = 0.f, B[4], C[4];
        if (live) {
            x = Elt<T>::to_f(static_cast<const T *>(a.x)[row * a.x_ld + d]);
            dl = Elt<T>::to_f(static_cast<const T *>(a.dt)[row * a.dt_ld + d]) + bias;
            if (a.z) z = Elt<T>::to_f(static_cast<const T *>(a.z)[row * a.z_ld + d]);
        }
        const T *pb = static_cast<const T *>(a.Bm) + row * a.b_ld + (long long)g * a.N + n0;
        const T *pc = static_cast<const T *>(a.Cm) + row * a.c_ld + (long long)g * a.N + n0;
        if (live && wide && a.vec_bc) {
            const uint2 ub = *reinterpret_cast<const uint2 *>(pb), uc = *reinterpret_cast<const uint2 *>(pc);
            const float2 b0 = Elt<T>::unpack(ub.x), b1 = Elt<T>::unpack(ub.y), c0 = Elt<T>::unpack(uc.x), c1 = Elt<T>::unpack(uc.y);
            B[0] = b0.x, B[1] = b0.y, B[2] = b1.x, B[3] = b1.y;
            C[0] = c0.x, C[1] = c0.y, C[2] = c1.x, C[3] = c1.y;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                B[i] = (live && n0 + i < a.N) ? Elt<T>::to_f(pb[i]) : 0.f;
                C[i] = (live && n0 + i < a.N) ? Elt<T>::to_f(pc[i]) : 0.f;
            }
        }
        if (a.softplus) dl = softplus(dl);
        const float u = dl * x;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = fmaf(ex2(A2[i] * dl), h[i], u * B[i]);
            y = fmaf(C[i], h[i], y);
        }
#pragma unroll
        for (int o = NL / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (live && n0 == 0) {
            y = fmaf(skip, x, y);
            if (a.z) y *= z * sigmoid(z);
            static_cast<T *>(a.y)[row * a.D + d] = Elt<T>::from_f(y);
        }
    }
    if (!live) return;
    float *out = a.state_out + ch * a.N + n0;
    if (wide) {
        *reinterpret_cast<float4 *>(out) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 + i < a.N) out[i] = h[i];
    }
}

template <typename T>
cudaError_t launch_t(const ScanArgs &a, int L, cudaStream_t s) {
    const long long per = 256 / L, blocks = ((long long)a.B * a.D + per - 1) / per;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(256);
    switch (L) {
        case 1: return launch_plain(scan_step_kernel<T, 1>, grid, block, 0, s, a);
        case 2: return launch_plain(scan_step_kernel<T, 2>, grid, block, 0, s, a);
        case 4: return launch_plain(scan_step_kernel<T, 4>, grid, block, 0, s, a);
        case 8: return launch_plain(scan_step_kernel<T, 8>, grid, block, 0, s, a);
        default: return launch_plain(scan_step_kernel<T, 16>, grid, block, 0, s, a);
    }
}

}  // namespace

cudaError_t launch_scan_step(const ScanArgs &a, int L, bool bf16, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(a, L, s) : launch_t<__half>(a, L, s);
}

}  // namespace scan
}  // namespace gdr
