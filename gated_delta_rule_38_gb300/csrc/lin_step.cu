// Linear attention with one decay a head, a few tokens at a time on the cached fp32 states [B,H,K,V], in place:
//   S <- lambda S + k v^T,  o = scale S^T q
//
// One block of 128 threads a (row, head, 64 columns of v): 16 lanes of four columns side by side, eight groups of rows,
// at most 16 rows a thread, all in registers, so that a block's 32 KB are on their way at once.  Bound by HBM: 8 K V bytes
// of state in and out a (row, head); 256 rows x 32 heads, 1.08 GB: 158 us, 6.85 TB/s.  Sums of o: over a thread's rows, then
// the two halves of a warp, then the four warps, always in this order.
#include "common.cuh"
#include "f32x2.cuh"
#include "lin.h"

namespace gdr {
namespace lin {
namespace {

constexpr int ST_T = 128, CW = 64, RG = 8, RPT = LD / RG;  // threads, columns a block, row groups, rows a thread

template <typename T, bool FULL>
__global__ void __launch_bounds__(ST_T, 4) lin_step_kernel(const StepArgs a) {
    __shared__ float sq[LD], sk[LD];
    __shared__ __align__(16) float so[4][CW];
    const int halves = FULL ? LD / CW : (a.V + CW - 1) / CW;
    const unsigned item = blockIdx.x / (unsigned)halves;
    const int half = (int)(blockIdx.x % (unsigned)halves), b = (int)(item / (unsigned)a.H), j = (int)(item % (unsigned)a.H);
    const int hk = j / (a.H / a.Hk), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = FULL ? LD : a.K, V = FULL ? LD : a.V;
    const int c = half * CW + (tid & 15) * 4, rg = tid >> 4;  // columns c .. c + 3, rows rg + 8 i
    const bool in = FULL || c < V;
    float *S = a.state + ((long long)b * a.H + j) * K * V + c;
    f2 s[2 * RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
        ulonglong2 x = make_ulonglong2(0ull, 0ull);
        if (in && (FULL || r < K)) x = *reinterpret_cast<const ulonglong2 *>(S + (long long)r * V);
        s[2 * i] = x.x, s[2 * i + 1] = x.y;
    }
    const float g = a.decay[j] < -120.f ? -120.f : a.decay[j];
    // lambda as the sum of two numbers: rounded once, it would be off by up to 2^-25 in the same direction at every token (a
    // memory of 1e4 tokens: states 2.6e-4 off).  From exp(g) - 1, good to its own last bits, while that is the smaller one.
    const float below = expm1f(g), whole = g > -0.5f ? 1.f + below : expf(g);
    const f2 lam = both(whole), rest = both(g > -0.5f ? below - (whole - 1.f) : 0.f);
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    for (int t = 0; t < a.T; ++t) {
        const long long at = (long long)b * a.T + t;
        if (FULL || tid < K) {
            sq[tid] = Elt<T>::to_f(q[at * a.q_ld + hk * K + tid]);
            sk[tid] = Elt<T>::to_f(k[at * a.k_ld + hk * K + tid]);
        }
        f2 v0 = 0ull, v1 = 0ull, o0 = 0ull, o1 = 0ull;
        if (in) {
            const T *p = v + at * a.v_ld + j * V + c;
            v0 = pack2(Elt<T>::to_f(p[0]), Elt<T>::to_f(p[1]));
            v1 = pack2(Elt<T>::to_f(p[2]), Elt<T>::to_f(p[3]));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = rg + RG * i;
            if (FULL || r < K) {
                const f2 kr = both(sk[r]), qr = both(sq[r]);
                s[2 * i] = fma2(lam, s[2 * i], fma2(rest, s[2 * i], mul2(kr, v0)));
                s[2 * i + 1] = fma2(lam, s[2 * i + 1], fma2(rest, s[2 * i + 1], mul2(kr, v1)));
                o0 = fma2(qr, s[2 * i], o0);
                o1 = fma2(qr, s[2 * i + 1], o1);
            }
        }
        float o[4];
        unpack2(o0, o[0], o[1]);
        unpack2(o1, o[2], o[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], 16);
        if (lane < 16) *reinterpret_cast<float4 *>(&so[warp][lane * 4]) = make_float4(o[0], o[1], o[2], o[3]);
        __syncthreads();
        if (tid < CW && half * CW + tid < V)
            static_cast<T *>(a.o)[(at * a.H + j) * V + half * CW + tid] =
                Elt<T>::from_f(a.scale * ((so[0][tid] + so[1][tid]) + (so[2][tid] + so[3][tid])));
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + RG * i;
        if (in && (FULL || r < K)) *reinterpret_cast<ulonglong2 *>(S + (long long)r * V) = make_ulonglong2(s[2 * i], s[2 * i + 1]);
    }
}

template <typename T>
cudaError_t step_t(const StepArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)((long long)a.B * a.H * ((a.V + CW - 1) / CW)));
    if (a.K == LD && a.V == LD) return launch_plain(lin_step_kernel<T, true>, grid, dim3(ST_T), 0, s, a);
    return launch_plain(lin_step_kernel<T, false>, grid, dim3(ST_T), 0, s, a);
}

// One thread eight columns.  (5311 tokens, 8 heads on 4, 64 columns: 3.6 us for 13.6 MB, which L2 still holds.)
template <typename T>
__global__ void __launch_bounds__(256) lin_group_sum_kernel(const float *part, T *out, long long n, int group, int D) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // vector of eight of out
    if (i >= n) return;
    const int per = D / 8;
    const long long head = i / per;
    const float *p = part + head * group * D + (i - head * per) * 8;
    f2 x[4] = {0ull, 0ull, 0ull, 0ull};
    for (int g = 0; g < group; ++g) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(p + (long long)g * D), w = *reinterpret_cast<const ulonglong2 *>(p + (long long)g * D + 4);
        x[0] = add2(x[0], u.x), x[1] = add2(x[1], u.y), x[2] = add2(x[2], w.x), x[3] = add2(x[3], w.y);
    }
    *reinterpret_cast<uint4 *>(out + i * 8) = make_uint4(narrow2<T>(x[0]), narrow2<T>(x[1]), narrow2<T>(x[2]), narrow2<T>(x[3]));
}

}  // namespace

cudaError_t launch_lin_step(const StepArgs &a, bool bf16, cudaStream_t s) {
    return bf16 ? step_t<__nv_bfloat16>(a, s) : step_t<__half>(a, s);
}

cudaError_t launch_lin_group_sum(const float *part, void *out, long long rows, int heads, int group, int D, bool bf16,
                                 cudaStream_t s) {
    const long long n = rows * (heads / group) * (D / 8);
    if (n == 0) return cudaSuccess;
    const dim3 grid((unsigned)((n + 255) / 256));
    if (bf16) return launch_plain(lin_group_sum_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, part, static_cast<__nv_bfloat16 *>(out), n, group, D);
    return launch_plain(lin_group_sum_kernel<__half>, grid, dim3(256), 0, s, part, static_cast<__half *>(out), n, group, D);
}

}  // namespace lin
}  // namespace gdr
