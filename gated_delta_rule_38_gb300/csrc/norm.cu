// Root-mean-square norm of rows, with the residual's addition in front of it and an 8-bit output with scales
// behind it, and its backward pass.
//
//   h = x + residual;  r = 1 / sqrt(mean_c h_c^2 + eps);  y_c = h_c r w_c
//   8-bit: s = max(max_c |y_c|, 1e-30) / 448 over a row or over each 128 columns,  q_c = e4m3(y_c / s)
//   backward at the stored h:  dh_c = r (w_c dy_c - h_c r^2 mean_c(w_c dy_c h_c)) + dresidual_c,
//                              dw_c = sum over rows of dy_c h_c r
//
// Each element is read and written once: a row lives in the registers of its threads (fp32) between the two
// passes over it that the formulas need, so the kernels are bound by HBM.  A row is spread over TPR threads
// (a power of two, 8 to 512) of EPT elements each; rows narrower than a block share it.  All sums are fp32.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "host.h"
#include "launch.h"

namespace gdr {
namespace {

constexpr int kNormThreads = 512;  // largest block: 128 registers a thread

enum { RES_NONE = 0, RES_HALF = 1, RES_F32 = 2 };

struct NormArgs {
    const void *x, *w, *res;
    void *y, *res_out;
    float *scale;
    const void *dy;            // backward
    void *dx, *dres;           // backward: dres only for an fp32 residual stream
    float *dw_part;            // backward: [blocks * rows per block][D]
    long long rows, x_ld;
    int D, tpr, res_kind, group, nscale;  // group: 0 = one scale a row
    bool w_f32;
    float eps;
};

// VEC consecutive elements of T at p as fp32 (one 16-byte load for VEC = 8).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *o) {
    if (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Elt<T>::unpack(r[i]);
            o[2 * i] = f.x, o[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = Elt<T>::to_f(p[i]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *v) {
    if (VEC == 8) {
        uint4 u;
        u.x = Elt<T>::pack(v[0], v[1]), u.y = Elt<T>::pack(v[2], v[3]);
        u.z = Elt<T>::pack(v[4], v[5]), u.w = Elt<T>::pack(v[6], v[7]);
        *reinterpret_cast<uint4 *>(p) = u;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = Elt<T>::from_f(v[i]);
    }
}
template <int VEC>
__device__ __forceinline__ void load_vec_f32(const float *p, float *o) {
    if (VEC == 8) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = p[i];
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec_f32(float *p, const float *v) {
    if (VEC == 8) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = v[i];
    }
}

// Where a thread's elements lie in its row.  VEC = 8: vector v of thread t at column 8 (v TPR + t).  VEC = 1
// (TPR >= 32): a warp takes 128 consecutive columns in four steps of its lanes, so that every load is contiguous
// over the lanes and every group of 128 columns stays inside one warp.
template <int VEC>
struct Cols {
    int tpr, t;
    __device__ __forceinline__ Cols(int tpr_, int t_) : tpr(tpr_), t(t_) {}
    __device__ __forceinline__ int operator()(int v) const {
        if (VEC == 8) return (v * tpr + t) * 8;
        return (v >> 2) * (tpr * 4) + (t >> 5) * 128 + (v & 3) * 32 + (t & 31);
    }
};

__device__ __forceinline__ float lanes_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// Maximum of non-negative floats (and NaN, which wins) by their bits.
__device__ __forceinline__ uint32_t lanes_max(uint32_t x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <typename T, int VEC, int NV, bool QUANT>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(const NormArgs a) {
    constexpr int EPT = VEC * NV;
    __shared__ float s_sum[2][32];
    __shared__ uint32_t s_max[2][32];
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x & (tpr - 1);
    const int rpb = blockDim.x / tpr, lanes = min(tpr, 32), wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cols<VEC> col(tpr, t);
    const float inv_d = 1.0f / (float)a.D;
    int parity = 0;
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < a.rows; r0 += (long long)gridDim.x * rpb, parity ^= 1) {
        const long long row = r0 + slot;
        const bool live = row < a.rows;
        const T *x = static_cast<const T *>(a.x) + row * a.x_ld;
        float h[EPT];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = col(v);
            if (live && c < a.D) {
                load_vec<T, VEC>(x + c, h + v * VEC);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[v * VEC + i] = 0.f;
            }
        }
        if (a.res_kind != RES_NONE) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = col(v);
                if (!(live && c < a.D)) continue;
                float e[VEC];
                if (a.res_kind == RES_F32)
                    load_vec_f32<VEC>(static_cast<const float *>(a.res) + row * a.D + c, e);
                else
                    load_vec<T, VEC>(static_cast<const T *>(a.res) + row * a.D + c, e);
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[v * VEC + i] += e[i];
                if (a.res_kind == RES_F32)
                    store_vec_f32<VEC>(static_cast<float *>(a.res_out) + row * a.D + c, h + v * VEC);
                else
                    store_vec<T, VEC>(static_cast<T *>(a.res_out) + row * a.D + c, h + v * VEC);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) ss = fmaf(h[i], h[i], ss);
        ss = lanes_sum(ss, lanes);
        if (tpr > 32) {
            if (lane == 0) s_sum[parity][warp] = ss;
            __syncthreads();
            ss = 0.f;
            for (int i = 0; i < wpr; ++i) ss += s_sum[parity][slot * wpr + i];
        }
        const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = col(v);
            if (c >= a.D) continue;
            float w[VEC];
            if (a.w_f32)
                load_vec_f32<VEC>(static_cast<const float *>(a.w) + c, w);
            else
                load_vec<T, VEC>(static_cast<const T *>(a.w) + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[v * VEC + i] *= r * w[i];
        }
        if constexpr (!QUANT) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = col(v);
                if (live && c < a.D) store_vec<T, VEC>(static_cast<T *>(a.y) + row * a.D + c, h + v * VEC);
            }
        } else {
            // largest magnitude of each vector, then of its scale's columns
            uint32_t m[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                m[v] = 0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) m[v] = max(m[v], abs_bits(h[v * VEC + i]));
            }
            if (a.group == 0) {
                uint32_t mm = 0;
#pragma unroll
                for (int v = 0; v < NV; ++v) mm = max(mm, m[v]);
                mm = lanes_max(mm, lanes);
                if (tpr > 32) {
                    if (lane == 0) s_max[parity][warp] = mm;
                    __syncthreads();
                    mm = 0;
                    for (int i = 0; i < wpr; ++i) mm = max(mm, s_max[parity][slot * wpr + i]);
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) m[v] = mm;
            } else if (VEC == 8) {
                // 16 lanes of 8 columns are a group; a row of 8 lanes has at most 128 columns, all one group
                if (tpr < 16) {
                    uint32_t mm = 0;
#pragma unroll
                    for (int v = 0; v < NV; ++v) mm = max(mm, m[v]);
                    mm = lanes_max(mm, 8);
#pragma unroll
                    for (int v = 0; v < NV; ++v) m[v] = mm;
                } else {
#pragma unroll
                    for (int v = 0; v < NV; ++v) m[v] = lanes_max(m[v], 16);
                }
            } else {
                // four steps of a warp are a group
#pragma unroll
                for (int q = 0; q + 3 < NV; q += 4) {
                    const uint32_t mm = max(max(m[q], m[q + 1]), max(m[q + 2], m[q + 3]));
                    m[q] = m[q + 1] = m[q + 2] = m[q + 3] = lanes_max(mm, 32);
                }
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = col(v);
                if (!(live && c < a.D)) continue;
                const float mx = __uint_as_float(m[v]);
                const float sc = (mx < 1e-30f ? 1e-30f : mx) / 448.0f;  // (a NaN stays)
                const float is = 1.0f / sc;
                unsigned char *q = static_cast<unsigned char *>(a.y) + row * a.D + c;
                if (VEC == 8) {
                    uint32_t u[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float *e = h + v * VEC + 4 * i;
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(e[0] * is, e[1] * is), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(e[2] * is, e[3] * is), __NV_SATFINITE, __NV_E4M3);
                        u[i] = lo | (hi << 16);
                    }
                    *reinterpret_cast<uint2 *>(q) = make_uint2(u[0], u[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) q[i] = __nv_cvt_float_to_fp8(h[v * VEC + i] * is, __NV_SATFINITE, __NV_E4M3);
                }
                if (a.group == 0 ? c == 0 : (c & 127) == 0) a.scale[row * a.nscale + (a.group ? c >> 7 : 0)] = sc;
            }
        }
    }
}

// Each block walks rows and keeps its threads' share of dw in registers; the per-block sums are added by
// reduce_rows_kernel in a fixed order.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(const NormArgs a) {
    constexpr int EPT = VEC * NV;
    __shared__ float2 s_sum[2][32];
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x & (tpr - 1);
    const int rpb = blockDim.x / tpr, lanes = min(tpr, 32), wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cols<VEC> col(tpr, t);
    const float inv_d = 1.0f / (float)a.D;
    float dw[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) dw[i] = 0.f;
    int parity = 0;
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < a.rows; r0 += (long long)gridDim.x * rpb, parity ^= 1) {
        const long long row = r0 + slot;
        const bool live = row < a.rows;
        float h[EPT], g[EPT];  // g: dy, then w dy
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = col(v);
            if (live && c < a.D) {
                if (a.res_kind == RES_F32)
                    load_vec_f32<VEC>(static_cast<const float *>(a.x) + row * a.x_ld + c, h + v * VEC);
                else
                    load_vec<T, VEC>(static_cast<const T *>(a.x) + row * a.x_ld + c, h + v * VEC);
                load_vec<T, VEC>(static_cast<const T *>(a.dy) + row * a.D + c, g + v * VEC);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[v * VEC + i] = g[v * VEC + i] = 0.f;
            }
        }
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = col(v);
            if (c >= a.D) continue;
            float w[VEC];
            if (a.w_f32)
                load_vec_f32<VEC>(static_cast<const float *>(a.w) + c, w);
            else
                load_vec<T, VEC>(static_cast<const T *>(a.w) + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                ss = fmaf(h[k], h[k], ss);
                sd = fmaf(g[k] * w[i], h[k], sd);
            }
        }
        ss = lanes_sum(ss, lanes);
        sd = lanes_sum(sd, lanes);
        if (tpr > 32) {
            if (lane == 0) s_sum[parity][warp] = make_float2(ss, sd);
            __syncthreads();
            ss = sd = 0.f;
            for (int i = 0; i < wpr; ++i) {
                const float2 f = s_sum[parity][slot * wpr + i];
                ss += f.x, sd += f.y;
            }
        }
        const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
        const float k2 = r * r * (sd * inv_d);
        const float one = a.eps * r * r;  // 1 - h^2 r^2 at D = 1, where the two terms below cancel but for it
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = col(v);
            if (!(live && c < a.D)) continue;
            float w[VEC], d[VEC], e[VEC];
            if (a.w_f32)
                load_vec_f32<VEC>(static_cast<const float *>(a.w) + c, w);
            else
                load_vec<T, VEC>(static_cast<const T *>(a.w) + c, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = v * VEC + i;
                dw[k] = fmaf(g[k], h[k] * r, dw[k]);
                d[i] = r * (a.D == 1 ? g[k] * w[i] * one : g[k] * w[i] - h[k] * k2);
            }
            if (a.res) {  // the gradient that reaches the summed stream from later layers
                if (a.res_kind == RES_F32)
                    load_vec_f32<VEC>(static_cast<const float *>(a.res) + row * a.D + c, e);
                else
                    load_vec<T, VEC>(static_cast<const T *>(a.res) + row * a.D + c, e);
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[i] += e[i];
            }
            store_vec<T, VEC>(static_cast<T *>(a.dx) + row * a.D + c, d);
            if (a.dres) store_vec_f32<VEC>(static_cast<float *>(a.dres) + row * a.D + c, d);
        }
    }
    float *part = a.dw_part + ((long long)blockIdx.x * rpb + slot) * a.D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = col(v);
        if (c < a.D) store_vec_f32<VEC>(part + c, dw + v * VEC);
    }
}

// out[c] = sum over `parts` rows of part[.][c]: 32 columns a block, its eight warps take every eighth row.
template <typename T>
__global__ void __launch_bounds__(256) reduce_rows_kernel(const float *part, long long parts, long long stride, int cols,
                                                          void *out, bool out_f32) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float x = 0.f;
    if (c < cols) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        long long i = warp;
        for (; i + 24 < parts; i += 32) {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] += part[(i + 8 * k) * stride + c];
        }
        for (; i < parts; i += 8) p[0] += part[i * stride + c];
        x = (p[0] + p[1]) + (p[2] + p[3]);
    }
    s[warp][lane] = x;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) y += s[k][lane];
        if (out_f32)
            static_cast<float *>(out)[c] = y;
        else
            static_cast<T *>(out)[c] = Elt<T>::from_f(y);
    }
}

// Threads a row: the power of two that covers D with 16 elements a thread (32 for rows over 8,192).
struct NormShape {
    int tpr, ept, threads, rpb;
};
NormShape norm_shape(int D, bool vec) {
    NormShape s;
    s.ept = D <= 16 * kNormThreads ? 16 : 32;
    s.tpr = vec ? 8 : 32;
    while (s.tpr * s.ept < D) s.tpr *= 2;
    s.threads = s.tpr < 256 ? 256 : s.tpr;
    s.rpb = s.threads / s.tpr;
    return s;
}

// Blocks of the backward: as many as are resident at once, so that dw is summed over few partial rows.
int norm_bwd_blocks(long long rows, const NormShape &s) {
    const long long need = (rows + s.rpb - 1) / s.rpb;
    const long long most = (long long)kSMs * (1024 / s.threads);
    return (int)(need < most ? need : most);
}

template <typename T, bool QUANT>
cudaError_t norm_fwd_t(const NormArgs &a, const NormShape &s, bool vec, cudaStream_t st) {
    const long long need = (a.rows + s.rpb - 1) / s.rpb;
    const dim3 grid((unsigned)(need < 0x7fffffff ? need : 0x7fffffff)), block(s.threads);
    if (vec) {
        if (s.ept == 16) return launch_plain(norm_fwd_kernel<T, 8, 2, QUANT>, grid, block, 0, st, a);
        return launch_plain(norm_fwd_kernel<T, 8, 4, QUANT>, grid, block, 0, st, a);
    }
    if (s.ept == 16) return launch_plain(norm_fwd_kernel<T, 1, 16, QUANT>, grid, block, 0, st, a);
    return launch_plain(norm_fwd_kernel<T, 1, 32, QUANT>, grid, block, 0, st, a);
}

template <typename T>
cudaError_t norm_bwd_t(const NormArgs &a, const NormShape &s, bool vec, int blocks, cudaStream_t st) {
    const dim3 grid(blocks), block(s.threads);
    if (vec) {
        if (s.ept == 16) return launch_plain(norm_bwd_kernel<T, 8, 2>, grid, block, 0, st, a);
        return launch_plain(norm_bwd_kernel<T, 8, 4>, grid, block, 0, st, a);
    }
    if (s.ept == 16) return launch_plain(norm_bwd_kernel<T, 1, 16>, grid, block, 0, st, a);
    return launch_plain(norm_bwd_kernel<T, 1, 32>, grid, block, 0, st, a);
}

gdr_status check_norm(const gdr_norm_problem *p) {
    if (!p) return GDR_ERR_NULL;
    if (p->rows < 0 || p->D < 1 || p->D > GDR_NORM_MAX_D || p->x_ld < p->D) return GDR_ERR_SHAPE;
    if (p->scale_group != 0 && p->scale_group != 128) return GDR_ERR_SHAPE;
    if (!is_half(p->dtype)) return GDR_ERR_DTYPE;
    if (p->weight_dtype != p->dtype && p->weight_dtype != GDR_FP32) return GDR_ERR_DTYPE;
    if (p->residual_dtype != p->dtype && p->residual_dtype != GDR_FP32) return GDR_ERR_DTYPE;
    if (p->y_dtype != p->dtype && p->y_dtype != GDR_E4M3) return GDR_ERR_DTYPE;
    return GDR_OK;
}

// Every pointer that is given is aligned to its elements; `vec` is cleared unless all allow 16-byte accesses.
bool norm_ptr(const void *p, size_t elem, size_t vec_bytes, bool *vec) {
    if (!p) return true;
    if (!aligned_to(p, elem)) return false;
    if (!aligned_to(p, vec_bytes)) *vec = false;
    return true;
}

}  // namespace

cudaError_t launch_reduce_rows(const float *part, long long parts, long long stride, int cols, void *out, bool bf16,
                               bool out_f32, cudaStream_t s) {
    const dim3 grid((unsigned)((cols + 31) / 32));
    if (bf16)
        return launch_plain(reduce_rows_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, part, parts, stride, cols, out,
                            out_f32);
    return launch_plain(reduce_rows_kernel<__half>, grid, dim3(256), 0, s, part, parts, stride, cols, out, out_f32);
}

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_norm_fwd(const gdr_norm_problem *p, const void *x, const void *weight, const void *residual, void *y,
                        void *residual_out, float *scale, void *stream) {
    gdr_status st = check_norm(p);
    if (st != GDR_OK) return st;
    const bool quant = p->y_dtype == GDR_E4M3;
    if (p->rows == 0) return GDR_OK;
    if (!x || !weight || !y || (quant && !scale) || ((residual != nullptr) != (residual_out != nullptr)))
        return GDR_ERR_NULL;
    bool vec = p->D % 8 == 0 && p->x_ld % 8 == 0;
    const size_t rs = esize(p->residual_dtype);
    if (!norm_ptr(x, 2, 16, &vec) || !norm_ptr(weight, esize(p->weight_dtype), 16, &vec) ||
        !norm_ptr(residual, rs, 16, &vec) || !norm_ptr(residual_out, rs, 16, &vec) ||
        !norm_ptr(y, quant ? 1 : 2, quant ? 8 : 16, &vec) || !norm_ptr(scale, 4, 4, &vec))
        return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    NormArgs a = {};
    a.x = x, a.w = weight, a.res = residual, a.y = y, a.res_out = residual_out, a.scale = scale;
    a.rows = p->rows, a.x_ld = p->x_ld, a.D = p->D, a.eps = p->eps;
    a.group = p->scale_group;
    a.nscale = p->scale_group ? (p->D + 127) / 128 : 1;
    a.w_f32 = p->weight_dtype == GDR_FP32;
    a.res_kind = !residual ? RES_NONE : p->residual_dtype == GDR_FP32 ? RES_F32 : RES_HALF;
    const NormShape s = norm_shape(p->D, vec);
    a.tpr = s.tpr;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return timed(K_NORM_FWD, cs, [&] {
        if (p->dtype == GDR_BF16)
            return quant ? norm_fwd_t<__nv_bfloat16, true>(a, s, vec, cs) : norm_fwd_t<__nv_bfloat16, false>(a, s, vec, cs);
        return quant ? norm_fwd_t<__half, true>(a, s, vec, cs) : norm_fwd_t<__half, false>(a, s, vec, cs);
    });
}

gdr_status gdr_norm_bwd_workspace_size(const gdr_norm_problem *p, size_t *bytes) {
    gdr_status st = check_norm(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    // (the wide path packs more of a narrow row's partial sums into a block: its size covers both)
    const NormShape s = norm_shape(p->D, true);
    const int blocks = p->rows ? norm_bwd_blocks(p->rows, s) : 0;
    *bytes = round_up((size_t)blocks * s.rpb * p->D * sizeof(float), 256);
    return GDR_OK;
}

gdr_status gdr_norm_bwd(const gdr_norm_problem *p, const void *h, const void *weight, const void *dy,
                        const void *dresidual, void *dx, float *dresidual_in, void *dweight, void *workspace,
                        size_t workspace_bytes, void *stream) {
    size_t need = 0;
    gdr_status st = gdr_norm_bwd_workspace_size(p, &need);
    if (st != GDR_OK) return st;
    if (!weight || !dweight || (p->rows && (!h || !dy || !dx))) return GDR_ERR_NULL;
    const bool f32 = p->residual_dtype == GDR_FP32;
    if (dresidual_in && !f32) return GDR_ERR_DTYPE;
    bool vec = p->D % 8 == 0 && p->x_ld % 8 == 0;
    if (!norm_ptr(h, f32 ? 4 : 2, 16, &vec) || !norm_ptr(weight, esize(p->weight_dtype), 16, &vec) ||
        !norm_ptr(dy, 2, 16, &vec) || !norm_ptr(dresidual, f32 ? 4 : 2, 16, &vec) || !norm_ptr(dx, 2, 16, &vec) ||
        !norm_ptr(dresidual_in, 4, 16, &vec) || !norm_ptr(dweight, esize(p->weight_dtype), 4, &vec))
        return GDR_ERR_ALIGN;
    if (need && (!workspace || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    if (need && !aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->rows == 0) return cuda_status(cudaMemsetAsync(dweight, 0, (size_t)p->D * esize(p->weight_dtype), cs));
    NormArgs a = {};
    a.x = h, a.w = weight, a.dy = dy, a.res = dresidual, a.dx = dx, a.dres = dresidual_in;
    a.dw_part = static_cast<float *>(workspace);
    a.rows = p->rows, a.x_ld = p->x_ld, a.D = p->D, a.eps = p->eps;
    a.w_f32 = p->weight_dtype == GDR_FP32;
    a.res_kind = f32 ? RES_F32 : RES_HALF;
    const NormShape s = norm_shape(p->D, vec);
    a.tpr = s.tpr;
    const int blocks = norm_bwd_blocks(p->rows, s);
    st = timed(K_NORM_BWD, cs, [&] {
        return p->dtype == GDR_BF16 ? norm_bwd_t<__nv_bfloat16>(a, s, vec, blocks, cs)
                                    : norm_bwd_t<__half>(a, s, vec, blocks, cs);
    });
    if (st != GDR_OK) return st;
    return timed(K_REDUCE, cs, [&] {
        return launch_reduce_rows(a.dw_part, (long long)blocks * s.rpb, p->D, p->D, dweight, p->dtype == GDR_BF16,
                                  a.w_f32, cs);
    });
}

}  // extern "C"
