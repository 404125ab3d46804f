// Selective scan for single tokens: the T tokens of every row applied one by one to its cached fp32 state, in place.
//
//   h <- exp(delta A) h + delta x B,   y = (C . h + D x) silu(z)      (delta = softplus(dt + bias) or dt + bias)
//
// Bound by HBM: 8 bytes of state a (row, channel, state) against ten of token data a (row, channel).  A channel's N
// states lie in NL = 1 .. 16 lanes side by side, four in each (one 16-byte access where N allows it), so a warp moves
// contiguous state.  A thread takes RB rows of the batch, so that several states are in flight and A, the bias and D
// are read once; the scalar work of a row (softplus, the gate) is done by one of the channel's lanes and handed round.
// The sum over the states is a butterfly over the lanes.
#include "scan.cuh"

namespace gdr {
namespace scan {
namespace {

template <typename T, int NL, int RB>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanArgs a) {
    constexpr int OWN = RB > NL ? RB / NL : 1;  // rows whose scalars a lane computes (lanes past RB repeat them)
    const int nl = threadIdx.x % NL, n0 = nl * 4, lead = (threadIdx.x & 31) - nl;
    const unsigned ch = blockIdx.x * (256 / NL) + threadIdx.x / NL;  // (group of rows, channel)
    const int rows = (a.B + RB - 1) / RB;
    const int rg = (int)(ch / (unsigned)a.D), d = (int)(ch - (unsigned)rg * a.D), g = d / a.Dg, b0 = rg * RB;
    const bool live = rg < rows;
    const bool wide = a.st_vec && n0 < a.N;
    float h[RB][4], A2[4];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const bool in = live && b0 + r < a.B;
        const float *st = a.state_in + ((long long)(b0 + r) * a.D + d) * a.N + n0;
        if (in && wide) {
            const float4 f = *reinterpret_cast<const float4 *>(st);
            h[r][0] = f.x, h[r][1] = f.y, h[r][2] = f.z, h[r][3] = f.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[r][i] = (in && n0 + i < a.N) ? st[i] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] = (live && n0 + i < a.N) ? a.A[(long long)d * a.N + n0 + i] * LOG2E : 0.f;
    const float bias = (live && a.bias) ? a.bias[d] : 0.f, skip = (live && a.skip) ? a.skip[d] : 0.f;
    for (int t = 0; t < a.T; ++t) {
        // the scalars of this lane's rows
        float dl[OWN], u[OWN], base[OWN], gate[OWN];
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            const int r = RB >= NL ? nl * OWN + o : nl % RB;
            float x = 0.f, v = 0.f, z = 0.f;
            if (live && b0 + r < a.B) {
                const long long row = (long long)(b0 + r) * a.T + t;
                x = Elt<T>::to_f(static_cast<const T *>(a.x)[row * a.x_ld + d]);
                v = Elt<T>::to_f(static_cast<const T *>(a.dt)[row * a.dt_ld + d]);
                if (a.z) z = Elt<T>::to_f(static_cast<const T *>(a.z)[row * a.z_ld + d]);
            }
            v += bias;
            dl[o] = a.softplus ? softplus(v) : v;
            u[o] = dl[o] * x;
            base[o] = skip * x;
            gate[o] = a.z ? z * sigmoid(z) : 1.f;
        }
        float y[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int from = lead + (RB >= NL ? r / OWN : r), o = RB >= NL ? r % OWN : 0;
            const float dr = __shfl_sync(0xffffffffu, dl[o], from), ur = __shfl_sync(0xffffffffu, u[o], from);
            float B[4], C[4];
            const bool in = live && b0 + r < a.B;
            const long long row = (long long)(b0 + r) * a.T + t;
            const T *pb = static_cast<const T *>(a.Bm) + row * a.b_ld + (long long)g * a.N + n0;
            const T *pc = static_cast<const T *>(a.Cm) + row * a.c_ld + (long long)g * a.N + n0;
            if (in && a.vec_bc && n0 < a.N) {
                const uint2 ub = *reinterpret_cast<const uint2 *>(pb), uc = *reinterpret_cast<const uint2 *>(pc);
                unpack2(widen2<T>(ub.x), B[0], B[1]);
                unpack2(widen2<T>(ub.y), B[2], B[3]);
                unpack2(widen2<T>(uc.x), C[0], C[1]);
                unpack2(widen2<T>(uc.y), C[2], C[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    B[i] = (in && n0 + i < a.N) ? Elt<T>::to_f(pb[i]) : 0.f;
                    C[i] = (in && n0 + i < a.N) ? Elt<T>::to_f(pc[i]) : 0.f;
                }
            }
            y[r] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[r][i] = fmaf(ex2(A2[i] * dr), h[r][i], ur * B[i]);
                y[r] = fmaf(C[i], h[r][i], y[r]);
            }
#pragma unroll
            for (int o2 = NL / 2; o2 > 0; o2 >>= 1) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o2);
        }
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
            const int r = RB >= NL ? nl * OWN + o : nl % RB;
            float v = y[0];
#pragma unroll
            for (int k = 1; k < RB; ++k) v = k == r ? y[k] : v;
            if (live && nl < RB && b0 + r < a.B)
                static_cast<T *>(a.y)[((long long)(b0 + r) * a.T + t) * a.D + d] = Elt<T>::from_f((base[o] + v) * gate[o]);
        }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        if (!(live && b0 + r < a.B)) continue;
        float *out = a.state_out + ((long long)(b0 + r) * a.D + d) * a.N + n0;
        if (wide) {
            *reinterpret_cast<float4 *>(out) = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n0 + i < a.N) out[i] = h[r][i];
        }
    }
}

template <typename T, int RB>
cudaError_t launch_rb(const ScanArgs &a, int L, cudaStream_t s) {
    const long long per = 256 / L, chans = (long long)((a.B + RB - 1) / RB) * a.D, blocks = (chans + per - 1) / per;
    if (chans + per > 0xffffffffLL || blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(256);
    switch (L) {
        case 1: return launch_plain(scan_step_kernel<T, 1, RB>, grid, block, 0, s, a);
        case 2: return launch_plain(scan_step_kernel<T, 2, RB>, grid, block, 0, s, a);
        case 4: return launch_plain(scan_step_kernel<T, 4, RB>, grid, block, 0, s, a);
        case 8: return launch_plain(scan_step_kernel<T, 8, RB>, grid, block, 0, s, a);
        default: return launch_plain(scan_step_kernel<T, 16, RB>, grid, block, 0, s, a);
    }
}
// Four rows a thread once that still leaves every SM its threads.
template <typename T>
cudaError_t launch_t(const ScanArgs &a, int L, cudaStream_t s) {
    if ((long long)a.B * a.D * L >= 4LL * kSMs * 1024) return launch_rb<T, 4>(a, L, s);
    return launch_rb<T, 1>(a, L, s);
}

}  // namespace

cudaError_t launch_scan_step(const ScanArgs &a, int L, bool bf16, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(a, L, s) : launch_t<__half>(a, L, s);
}

}  // namespace scan
}  // namespace gdr
