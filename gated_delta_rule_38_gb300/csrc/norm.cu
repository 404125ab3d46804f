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
#include "f32x2.cuh"
#include "host.h"
#include "launch.h"

namespace gdr {
namespace {

enum { RES_NONE = 0, RES_HALF = 1, RES_F32 = 2 };

struct NormArgs {
    const void *x, *w, *res;
    void *y, *res_out;
    float *scale;
    const void *dy;            // backward
    void *dx, *dres;           // backward: dres only for an fp32 residual stream
    float *dw_part;            // backward: [blocks * rows per block][D]
    long long rows, x_ld;
    int D, tpr, group, nscale;  // group: 0 = one scale a row
    bool w_f32;
    float eps;
};

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

// A thread's elements of one row as they lie in memory (16-bit or fp32), so that the next row can be on its way
// while this one is worked on; zeros past the row's end.
template <int VEC, int NV, bool F32>
struct RawRow {
    static constexpr int W = F32 ? VEC * NV : VEC * NV / 2;  // words
    uint32_t w[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const void *base, long long at, const Cols<VEC> &col, int D) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = col(v);
            if constexpr (VEC == 8) {
                constexpr int Q = F32 ? 2 : 1;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (c < D) {
                        const uint4 *p = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at + c)
                                             : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at + c);
                        u = p[q];
                    }
                    uint32_t *o = w + (v * Q + q) * 4;
                    o[0] = u.x, o[1] = u.y, o[2] = u.z, o[3] = u.w;
                }
            } else if constexpr (F32) {
                w[v] = c < D ? static_cast<const uint32_t *>(base)[at + c] : 0;
            } else {
                const uint32_t e = c < D ? static_cast<const uint16_t *>(base)[at + c] : 0;
                if (v & 1) w[v / 2] |= e << 16; else w[v / 2] = e;
            }
        }
    }
    // pairs of consecutive elements
    template <typename T>
    __device__ __forceinline__ f2 pair(int i) const {
        if constexpr (F32) return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return widen2<T>(w[i]);
    }
};

// The same elements back to memory.
template <typename T, int VEC, int NV, bool F32>
__device__ __forceinline__ void store_row(void *base, long long at, const Cols<VEC> &col, int D, const f2 *h) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = col(v);
        if (c >= D) continue;
        if constexpr (VEC == 8) {
            const f2 *e = h + v * 4;
            if constexpr (F32) {
                ulonglong2 *p = reinterpret_cast<ulonglong2 *>(static_cast<float *>(base) + at + c);
                p[0] = make_ulonglong2(e[0], e[1]);
                p[1] = make_ulonglong2(e[2], e[3]);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at + c) =
                    make_uint4(narrow2<T>(e[0]), narrow2<T>(e[1]), narrow2<T>(e[2]), narrow2<T>(e[3]));
            }
        } else {
            float lo, hi;
            unpack2(h[v / 2], lo, hi);
            const float x = v & 1 ? hi : lo;
            if constexpr (F32) static_cast<float *>(base)[at + c] = x;
            else static_cast<T *>(base)[at + c] = Elt<T>::from_f(x);
        }
    }
}

// The thread's weights as fp32 pairs (zeros past the row's end).
template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_weight(const NormArgs &a, const Cols<VEC> &col, f2 *w) {
    if (a.w_f32) {
        RawRow<VEC, NV, true> r;
        r.load(a.w, 0, col, a.D);
#pragma unroll
        for (int i = 0; i < VEC * NV / 2; ++i) w[i] = r.template pair<T>(i);
    } else {
        RawRow<VEC, NV, false> r;
        r.load(a.w, 0, col, a.D);
#pragma unroll
        for (int i = 0; i < VEC * NV / 2; ++i) w[i] = r.template pair<T>(i);
    }
}

__device__ __forceinline__ float lanes_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// Maximum of magnitudes; a NaN wins.  (Over lanes by the bits, which order non-negative floats, NaN last.)
__device__ __forceinline__ float max_abs(float m, float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
    return r;
}
__device__ __forceinline__ float lanes_max(float m, int lanes) {
    uint32_t x = __float_as_uint(m);
    for (int o = lanes >> 1; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return __uint_as_float(x);
}

// Registers: 16 elements a thread leave room for three blocks of 256 an SM (two in the backward) with the weights and
// the next row's loads held in registers.  Rows over 8,192 take 32 elements a thread and hold neither.
template <int EPT, int BT>
struct Bounds {
    static constexpr bool hold = EPT <= 16;
    static constexpr int fwd = BT == 256 ? 3 : 1, bwd = BT == 256 ? 2 : 1;
};

template <typename T, int VEC, int NV, int BT, bool QUANT, int RES>
__global__ void __launch_bounds__(BT, Bounds<VEC * NV, BT>::fwd) norm_fwd_kernel(const NormArgs a) {
    constexpr int P = VEC * NV / 2;  // pairs a thread
    constexpr bool HOLD = Bounds<VEC * NV, BT>::hold;
    __shared__ float s_sum[2][16];
    __shared__ float s_max[2][16];
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x & (tpr - 1);
    const int rpb = blockDim.x / tpr, lanes = min(tpr, 32), wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cols<VEC> col(tpr, t);
    const float inv_d = 1.0f / (float)a.D;
    const long long step = (long long)gridDim.x * rpb;
    RawRow<VEC, NV, false> rx;
    RawRow<VEC, NV, RES == RES_F32> rr;
    auto fetch = [&](long long row) {
        if (row < a.rows) {
            rx.load(a.x, row * a.x_ld, col, a.D);
            if (RES != RES_NONE) rr.load(a.res, row * a.D, col, a.D);
        } else {
            rx.zero();
            rr.zero();
        }
    };
    long long row = (long long)blockIdx.x * rpb + slot;
    f2 w[P];
    if (HOLD) {
        fetch(row);
        load_weight<T, VEC, NV>(a, col, w);
    }
    int parity = 0;
    // (all threads of a block run the same number of rounds: its last slot's rows may lie past the end)
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < a.rows; r0 += step, row += step, parity ^= 1) {
        const bool live = row < a.rows;
        f2 h[P], ss2 = 0ull;
        if (!HOLD) fetch(row);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            h[i] = rx.template pair<T>(i);
            if (RES != RES_NONE) h[i] = add2(h[i], rr.template pair<T>(i));
            ss2 = fma2(h[i], h[i], ss2);
        }
        if (HOLD) fetch(row + step);
        if (RES != RES_NONE && live) store_row<T, VEC, NV, RES == RES_F32>(a.res_out, row * a.D, col, a.D, h);
        float ss = lanes_sum(sum2(ss2), lanes);
        if (tpr > 32) {
            if (lane == 0) s_sum[parity][warp] = ss;
            __syncthreads();
            ss = 0.f;
            for (int i = 0; i < wpr; ++i) ss += s_sum[parity][slot * wpr + i];
        }
        const f2 r = both(rsqrtf(fmaf(ss, inv_d, a.eps)));
        if (!HOLD) load_weight<T, VEC, NV>(a, col, w);
#pragma unroll
        for (int i = 0; i < P; ++i) h[i] = mul2(mul2(h[i], r), w[i]);
        if constexpr (!QUANT) {
            if (live) store_row<T, VEC, NV, false>(a.y, row * a.D, col, a.D, h);
        } else {
            float y[2 * P], m[NV];  // largest magnitude of each vector, then of its scale's columns
#pragma unroll
            for (int i = 0; i < P; ++i) unpack2(h[i], y[2 * i], y[2 * i + 1]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                m[v] = 0.f;
#pragma unroll
                for (int i = 0; i < VEC; ++i) m[v] = max_abs(m[v], y[v * VEC + i]);
            }
            if (a.group == 0) {
                float mm = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) mm = max_abs(mm, m[v]);
                mm = lanes_max(mm, lanes);
                if (tpr > 32) {
                    if (lane == 0) s_max[parity][warp] = mm;
                    __syncthreads();
                    mm = 0.f;
                    for (int i = 0; i < wpr; ++i) mm = max_abs(mm, s_max[parity][slot * wpr + i]);
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) m[v] = mm;
            } else if (VEC == 8) {
                // 16 lanes of 8 columns are a group; a row of 8 lanes has at most 128 columns, all one group
                if (tpr < 16) {
                    float mm = 0.f;
#pragma unroll
                    for (int v = 0; v < NV; ++v) mm = max_abs(mm, m[v]);
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
                    const float mm = max_abs(max_abs(m[q], m[q + 1]), max_abs(m[q + 2], m[q + 3]));
                    m[q] = m[q + 1] = m[q + 2] = m[q + 3] = lanes_max(mm, 32);
                }
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = col(v);
                if (!(live && c < a.D)) continue;
                const float sc = (m[v] < 1e-30f ? 1e-30f : m[v]) * (1.0f / 448.0f);  // (a NaN stays)
                const float is = 1.0f / sc;
                const float *e = y + v * VEC;
                unsigned char *q = static_cast<unsigned char *>(a.y) + row * a.D + c;
                if constexpr (VEC == 8) {
                    uint32_t u[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(e[4 * i] * is, e[4 * i + 1] * is), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(e[4 * i + 2] * is, e[4 * i + 3] * is), __NV_SATFINITE, __NV_E4M3);
                        u[i] = lo | (hi << 16);
                    }
                    *reinterpret_cast<uint2 *>(q) = make_uint2(u[0], u[1]);
                } else {
                    q[0] = __nv_cvt_float_to_fp8(e[0] * is, __NV_SATFINITE, __NV_E4M3);
                }
                if (a.group == 0 ? c == 0 : (c & 127) == 0) a.scale[row * a.nscale + (a.group ? c >> 7 : 0)] = sc;
            }
        }
    }
}

// Each block walks rows and keeps its threads' share of dw in registers; the per-block sums are added by
// reduce_rows_kernel in a fixed order.
template <typename T, int VEC, int NV, int BT, bool F32>
__global__ void __launch_bounds__(BT, Bounds<VEC * NV, BT>::bwd) norm_bwd_kernel(const NormArgs a) {
    constexpr int P = VEC * NV / 2;
    constexpr bool HOLD = Bounds<VEC * NV, BT>::hold;
    __shared__ float2 s_sum[2][16];
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x & (tpr - 1);
    const int rpb = blockDim.x / tpr, lanes = min(tpr, 32), wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cols<VEC> col(tpr, t);
    const float inv_d = 1.0f / (float)a.D;
    const long long step = (long long)gridDim.x * rpb;
    RawRow<VEC, NV, F32> rh, re;  // h; the gradient that reaches the summed stream from later layers
    RawRow<VEC, NV, false> rg;    // dy
    auto fetch = [&](long long row) {
        if (row < a.rows) {
            rh.load(a.x, row * a.x_ld, col, a.D);
            rg.load(a.dy, row * a.D, col, a.D);
            if (HOLD && a.res) re.load(a.res, row * a.D, col, a.D);
        } else {
            rh.zero();
            rg.zero();
            re.zero();
        }
    };
    long long row = (long long)blockIdx.x * rpb + slot;
    re.zero();
    f2 w[P], dw[P];
    if (HOLD) {
        fetch(row);
        load_weight<T, VEC, NV>(a, col, w);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) dw[i] = 0ull;
    int parity = 0;
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < a.rows; r0 += step, row += step, parity ^= 1) {
        const bool live = row < a.rows;
        f2 h[P], g[P], e[P], ss2 = 0ull, sd2 = 0ull;
        if (!HOLD) {
            fetch(row);
            load_weight<T, VEC, NV>(a, col, w);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            h[i] = rh.template pair<T>(i);
            g[i] = rg.template pair<T>(i);
            if (HOLD) e[i] = re.template pair<T>(i);
            ss2 = fma2(h[i], h[i], ss2);
            sd2 = fma2(mul2(g[i], w[i]), h[i], sd2);
        }
        if (HOLD) fetch(row + step);
        float ss = lanes_sum(sum2(ss2), lanes), sd = lanes_sum(sum2(sd2), lanes);
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
        const f2 r2 = both(r), k2 = both(-(r * r * r) * (sd * inv_d));
        if (!HOLD) {
            // (the weights again, and the later layers' gradient, now that dy's registers are to be freed)
            load_weight<T, VEC, NV>(a, col, w);
            if (a.res && live) re.load(a.res, row * a.D, col, a.D);
        }
        // at D = 1 the two terms of dh cancel but for 1 - h^2 r^2 = eps r^2
        const f2 one = both(a.D == 1 ? a.eps * r * r * r : r);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            dw[i] = fma2(g[i], mul2(h[i], r2), dw[i]);
            const f2 own = mul2(mul2(g[i], w[i]), one);
            if (!HOLD) e[i] = re.template pair<T>(i);
            h[i] = add2(e[i], a.D == 1 ? own : fma2(h[i], k2, own));
        }
        if (live) {
            store_row<T, VEC, NV, false>(a.dx, row * a.D, col, a.D, h);
            if (F32 && a.dres) store_row<T, VEC, NV, true>(a.dres, row * a.D, col, a.D, h);
        }
    }
    store_row<T, VEC, NV, true>(a.dw_part, ((long long)blockIdx.x * rpb + slot) * a.D, col, a.D, dw);
}

// Threads a row: the power of two that covers D with 16 elements a thread (32 for rows over 8,192).
struct NormShape {
    int tpr, ept, threads, rpb;
};
NormShape norm_shape(int D, bool vec) {
    NormShape s;
    s.ept = D <= 8192 ? 16 : 32;
    s.tpr = vec ? 8 : 32;
    while (s.tpr * s.ept < D) s.tpr *= 2;
    s.threads = s.tpr < 256 ? 256 : s.tpr;
    s.rpb = s.threads / s.tpr;
    return s;
}

// Blocks: at most as many as are resident at once; each walks rows, with its weights in registers and its next
// row's loads in flight.
int norm_blocks(long long rows, const NormShape &s, bool bwd) {
    const long long need = (rows + s.rpb - 1) / s.rpb;
    const long long most = (long long)kSMs * (s.threads == 256 ? (bwd ? 2 : 3) : 1);
    return (int)(need < most ? need : most);
}

template <typename T, int VEC, int EPT, int BT>
cudaError_t norm_fwd_v(const NormArgs &a, bool quant, int res, dim3 grid, cudaStream_t st) {
    constexpr int NV = EPT / VEC;
    const dim3 block(BT);
    if (quant) {
        if (res == RES_NONE) return launch_plain(norm_fwd_kernel<T, VEC, NV, BT, true, RES_NONE>, grid, block, 0, st, a);
        if (res == RES_HALF) return launch_plain(norm_fwd_kernel<T, VEC, NV, BT, true, RES_HALF>, grid, block, 0, st, a);
        return launch_plain(norm_fwd_kernel<T, VEC, NV, BT, true, RES_F32>, grid, block, 0, st, a);
    }
    if (res == RES_NONE) return launch_plain(norm_fwd_kernel<T, VEC, NV, BT, false, RES_NONE>, grid, block, 0, st, a);
    if (res == RES_HALF) return launch_plain(norm_fwd_kernel<T, VEC, NV, BT, false, RES_HALF>, grid, block, 0, st, a);
    return launch_plain(norm_fwd_kernel<T, VEC, NV, BT, false, RES_F32>, grid, block, 0, st, a);
}
template <typename T, int VEC>
cudaError_t norm_fwd_t(const NormArgs &a, const NormShape &s, bool quant, int res, cudaStream_t st) {
    const dim3 grid(norm_blocks(a.rows, s, false));
    if (s.ept == 32) return norm_fwd_v<T, VEC, 32, 512>(a, quant, res, grid, st);
    return s.threads == 256 ? norm_fwd_v<T, VEC, 16, 256>(a, quant, res, grid, st)
                            : norm_fwd_v<T, VEC, 16, 512>(a, quant, res, grid, st);
}
template <typename T, int VEC, int EPT, int BT>
cudaError_t norm_bwd_v(const NormArgs &a, bool f32, int blocks, cudaStream_t st) {
    if (f32) return launch_plain(norm_bwd_kernel<T, VEC, EPT / VEC, BT, true>, dim3(blocks), dim3(BT), 0, st, a);
    return launch_plain(norm_bwd_kernel<T, VEC, EPT / VEC, BT, false>, dim3(blocks), dim3(BT), 0, st, a);
}
template <typename T, int VEC>
cudaError_t norm_bwd_t(const NormArgs &a, const NormShape &s, bool f32, int blocks, cudaStream_t st) {
    if (s.ept == 32) return norm_bwd_v<T, VEC, 32, 512>(a, f32, blocks, st);
    return s.threads == 256 ? norm_bwd_v<T, VEC, 16, 256>(a, f32, blocks, st) : norm_bwd_v<T, VEC, 16, 512>(a, f32, blocks, st);
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
    const int res = !residual ? RES_NONE : p->residual_dtype == GDR_FP32 ? RES_F32 : RES_HALF;
    const NormShape s = norm_shape(p->D, vec);
    a.tpr = s.tpr;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return timed(K_NORM_FWD, cs, [&] {
        if (p->dtype == GDR_BF16)
            return vec ? norm_fwd_t<__nv_bfloat16, 8>(a, s, quant, res, cs) : norm_fwd_t<__nv_bfloat16, 1>(a, s, quant, res, cs);
        return vec ? norm_fwd_t<__half, 8>(a, s, quant, res, cs) : norm_fwd_t<__half, 1>(a, s, quant, res, cs);
    });
}

gdr_status gdr_norm_bwd_workspace_size(const gdr_norm_problem *p, size_t *bytes) {
    gdr_status st = check_norm(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    // (the wide path packs more of a narrow row's partial sums into a block: its size covers both)
    const NormShape s = norm_shape(p->D, true);
    const int blocks = p->rows ? norm_blocks(p->rows, s, true) : 0;
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
    const NormShape s = norm_shape(p->D, vec);
    a.tpr = s.tpr;
    const int blocks = norm_blocks(p->rows, s, true);
    st = timed(K_NORM_BWD, cs, [&] {
        if (p->dtype == GDR_BF16)
            return vec ? norm_bwd_t<__nv_bfloat16, 8>(a, s, f32, blocks, cs) : norm_bwd_t<__nv_bfloat16, 1>(a, s, f32, blocks, cs);
        return vec ? norm_bwd_t<__half, 8>(a, s, f32, blocks, cs) : norm_bwd_t<__half, 1>(a, s, f32, blocks, cs);
    });
    if (st != GDR_OK) return st;
    return timed(K_REDUCE, cs, [&] {
        const RowSums out = {dweight, p->D};
        return launch_reduce_rows(a.dw_part, (long long)blocks * s.rpb, p->D, &out, 1, p->dtype == GDR_BF16, a.w_f32, cs);
    });
}

}  // extern "C"
