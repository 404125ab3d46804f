// Root-mean-square norm of rows, with the residual's addition in front of it and an 8-bit output with scales
// behind it, and its backward pass.
//
//   h = x + residual;  r = 1 / sqrt(mean_c h_c^2 + eps);  y_c = h_c r w_c
//   8-bit: s = max(max_c |y_c|, 1e-30) / 448 over a row or over each 128 columns,  q_c = e4m3(y_c / s)
//   backward at the stored h:  dh_c = r (w_c dy_c - h_c r^2 mean_c(w_c dy_c h_c)) + dresidual_c,
//                              dw_c = sum over rows of dy_c h_c r
//
// Each element is read and written once: between the two passes over a row that the formulas need it lives in the
// registers of its threads (forward, fp32) or in shared memory (backward), so the kernels are bound by HBM.  A row is spread over TPR threads
// (a power of two, 8 to 512) of EPT elements each; rows narrower than a block share it.  All sums are fp32.
//
// Two forms.  Where every row starts on a 16-byte boundary a thread owns whole vectors of 8 columns.  Otherwise
// (ragged) a block brings rows into shared memory as the aligned 16-byte pieces that hold them, asynchronously and a
// row ahead, and a thread owns every TPR-th column, so that lanes side by side read and write side by side.  (7203 x 4381 with
// a residual: 82 us; 150 with vectors cut at the multiples of 8 elements and weights in shared memory, 167 with single elements.)
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "host.h"
#include "launch.h"
#include "norm.h"

namespace gdr {
namespace norm {
namespace {

// A thread's elements of one row as they lie in memory (16-bit or fp32), so that the next row can be on its way
// while this one is worked on: vector v of thread t at column 8 (v TPR + t); zeros past the row's end.
template <int NV, bool F32>
struct RawRow {
    static constexpr int PW = F32 ? 8 : 4;  // words a vector
    uint32_t w[PW * NV];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < PW * NV; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const void *base, long long row_at, int tpr, int t, int D) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * tpr + t) * 8;
#pragma unroll
            for (int k = 0; k < PW / 4; ++k) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (c < D) {
                    const uint4 *q = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + row_at + c)
                                         : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + row_at + c);
                    u = q[k];
                }
                uint32_t *o = w + v * PW + 4 * k;
                o[0] = u.x, o[1] = u.y, o[2] = u.z, o[3] = u.w;
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

// The same elements to memory.
template <typename T, int NV, bool F32>
__device__ __forceinline__ void store_row(void *base, long long row_at, int tpr, int t, int D, const f2 *h) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * tpr + t) * 8;
        if (c >= D) continue;
        const f2 *e = h + v * 4;
        if constexpr (F32) {
            ulonglong2 *q = reinterpret_cast<ulonglong2 *>(static_cast<float *>(base) + row_at + c);
            q[0] = make_ulonglong2(e[0], e[1]);
            q[1] = make_ulonglong2(e[2], e[3]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + row_at + c) =
                make_uint4(narrow2<T>(e[0]), narrow2<T>(e[1]), narrow2<T>(e[2]), narrow2<T>(e[3]));
        }
    }
}

// The thread's weights as fp32 pairs.
template <typename T, int NV>
__device__ __forceinline__ void load_weight(const NormArgs &a, int t, f2 *w) {
    if (a.w_f32) {
        RawRow<NV, true> r;
        r.load(a.w, 0, a.tpr, t, a.D);
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) w[i] = r.template pair<T>(i);
    } else {
        RawRow<NV, false> r;
        r.load(a.w, 0, a.tpr, t, a.D);
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) w[i] = r.template pair<T>(i);
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
// The scale of columns whose largest magnitude is m.  (A NaN stays.)
__device__ __forceinline__ float scale_of(float m) { return (m < 1e-30f ? 1e-30f : m) / 448.0f; }

// y / scale to the nearest fp32 number from one reciprocal a scale: the quotient's estimate y (1 / scale) is off by an ulp or
// two, its remainder is exact in one fused operation, and the remainder times the reciprocal corrects it (Markstein, IBM
// Journal of Research and Development 34, 1990).  Small rows are taken 2^64 times as large, so that no remainder
// underflows; an infinite scale has no remainder and makes what is finite 0.  (Equal to the division in 6e10 pairs tried, most
// of them beside ties of the 8-bit type, where the estimate alone falls on the other side.  8192 x 4096 from an fp32 stream:
// 66 us as with the estimate, 70 with a division an element; ragged 7203 x 4381: 126 us, 117 and 138.)
struct Quotient {
    float up, rs, neg;
    __device__ __forceinline__ Quotient() {}
    __device__ __forceinline__ explicit Quotient(float scale) {
        up = scale < 1e-25f ? 0x1p64f : 1.f;
        const float s = scale * up;
        rs = 1.0f / s;
        neg = s < __int_as_float(0x7f800000) ? -s : 0.f;
    }
    __device__ __forceinline__ float of(float y) const {
        y *= up;
        const float q = y * rs;
        return fmaf(fmaf(q, neg, y), rs, q);
    }
    __device__ __forceinline__ float2 of(f2 y) const {
        y = mul2(y, both(up));
        f2 q = mul2(y, both(rs));
        q = fma2(fma2(q, both(neg), y), both(rs), q);
        float2 r;
        unpack2(q, r.x, r.y);
        return r;
    }
};

// Registers: 16 elements a thread leave room for three blocks of 256 an SM with the weights and the next row's loads held
// in registers.  Rows over 8,192 take 32 elements a thread and hold neither.
template <int NV, int BT>
struct Bounds {
    static constexpr bool hold = NV <= 2;
    static constexpr int fwd = BT == 256 ? 3 : 1;
};

// 8192 x 4096 bf16, cold caches: 48 us with a bf16 residual (268 MB, 5.6 TB/s, 83 % of a copy's rate); with an fp32 residual
// and e4m3 output 66 us (369 MB, 5.6 TB/s).
template <typename T, int NV, int BT, bool QUANT, int RES>
__global__ void __launch_bounds__(BT, Bounds<NV, BT>::fwd) norm_fwd_kernel(const NormArgs a) {
    constexpr int P = 4 * NV;  // pairs a thread
    constexpr bool HOLD = Bounds<NV, BT>::hold;
    __shared__ float s_sum[2][16];
    __shared__ float s_max[2][16];
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x & (tpr - 1), D = a.D;
    const int rpb = blockDim.x / tpr, lanes = min(tpr, 32), wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_d = 1.0f / (float)D;
    const long long step = (long long)gridDim.x * rpb;
    RawRow<NV, false> rx;
    RawRow<NV, RES == RES_F32> rr;
    auto fetch = [&](long long row) {
        if (row < a.rows) {
            rx.load(a.x, row * a.x_ld, tpr, t, D);
            if (RES != RES_NONE) rr.load(a.res, row * D, tpr, t, D);
        } else {
            rx.zero();
            rr.zero();
        }
    };
    long long row = (long long)blockIdx.x * rpb + slot;
    f2 w[P];
    if (HOLD) {
        fetch(row);
        load_weight<T, NV>(a, t, w);
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
        if (RES != RES_NONE && live) store_row<T, NV, RES == RES_F32>(a.res_out, row * D, tpr, t, D, h);
        float ss = lanes_sum(sum2(ss2), lanes);
        if (tpr > 32) {
            if (lane == 0) s_sum[parity][warp] = ss;
            __syncthreads();
            ss = 0.f;
            for (int i = 0; i < wpr; ++i) ss += s_sum[parity][slot * wpr + i];
        }
        const f2 r = both(rsqrtf(fmaf(ss, inv_d, a.eps)));
        if (!HOLD) load_weight<T, NV>(a, t, w);
#pragma unroll
        for (int i = 0; i < P; ++i) h[i] = mul2(mul2(h[i], r), w[i]);
        if constexpr (!QUANT) {
            if (live) store_row<T, NV, false>(a.y, row * D, tpr, t, D, h);
        } else {
            float y[2 * P], m[NV];  // largest magnitude of each vector, then of its scale's columns
#pragma unroll
            for (int i = 0; i < P; ++i) unpack2(h[i], y[2 * i], y[2 * i + 1]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                m[v] = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m[v] = max_abs(m[v], y[v * 8 + i]);
            }
            if (a.group == 0 || tpr < 16) {  // (a row of 8 lanes has at most 128 columns, all one group)
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
            } else {  // 16 lanes of 8 columns are a group
#pragma unroll
                for (int v = 0; v < NV; ++v) m[v] = lanes_max(m[v], 16);
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * tpr + t) * 8;
                if (!(live && c < D)) continue;
                const float scale = scale_of(m[v]);
                const Quotient quot(scale);
                const f2 *e = h + v * 4;
                uint32_t u[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(quot.of(e[2 * i]), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(quot.of(e[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
                    u[i] = lo | (hi << 16);
                }
                *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(a.y) + row * D + c) = make_uint2(u[0], u[1]);
                if (a.group == 0 ? c == 0 : (c & 127) == 0) a.scale[row * a.nscale + (a.group ? c >> 7 : 0)] = scale;
            }
        }
    }
}

// dh of a pair: r w g + h k2 (k2 = -r^3 mean(w g h), taken from the mean's side: r^3 alone leaves fp32's range at rows of
// 1e13 or, with a small eps, 1e-13), where at D = 1 the two terms cancel but for
// 1 - h^2 r^2 = eps r^2 (`one` is then eps r^3 and k2 unused).
__device__ __forceinline__ f2 dh_pair(f2 g, f2 w, f2 h, f2 one, f2 k2, bool d1) {
    const f2 own = mul2(mul2(g, w), one);
    return d1 ? own : fma2(h, k2, own);
}

// The block's share of dw from those of its row slots [rpb][D], in order.
__device__ __forceinline__ void sum_slots(const NormArgs &a, const float *slots, int rpb) {
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
        float v = 0.f;
        for (int i = 0; i < rpb; ++i) v += slots[i * a.D + c];
        a.dw_part[(long long)blockIdx.x * a.D + c] = v;
    }
}

// A thread's elements of one row of h, of dy and of the gradient that reaches the summed stream from later layers, in
// places of shared memory that only it uses: vector k of a stage lies at [stage][k][thread].
template <int NV, int BT, bool F32>
struct BwdRows {
    static constexpr int VH = F32 ? 2 : 1;                       // 16-byte vectors of 8 elements of h
    static constexpr int H = 0, G = NV * VH, E = G + NV;         // where each begins
    static constexpr int stages = NV <= 2 || !F32 ? 2 : 1;
    uint4 *mine;
    int per;                                                     // vectors a stage
    __device__ __forceinline__ BwdRows(void *smem, bool later) : mine(static_cast<uint4 *>(smem) + threadIdx.x), per(later ? E + NV * VH : E) {}
    static size_t bytes(bool later) { return (size_t)stages * (later ? E + NV * VH : E) * BT * sizeof(uint4); }
    __device__ __forceinline__ uint4 *at(int stage, int k) const { return mine + (stage * per + k) * BT; }
    // `in`: the row exists; else zeros, as past the row's end.
    template <int V>
    __device__ __forceinline__ void copy(int stage, int k0, const void *base, long long row_at, int tpr, int t, int D, bool in) const {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * tpr + t) * 8;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                uint4 *to = at(stage, k0 + v * V + k);
                const char *from = static_cast<const char *>(base) + (row_at + c) * (2 * V) + 16 * k;
                if (in && c < D)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(to)), "l"(from) : "memory");
                else
                    *to = make_uint4(0, 0, 0, 0);
            }
        }
    }
    // the four pairs of vector v
    template <typename T, int V>
    __device__ __forceinline__ void get(int stage, int k0, int v, f2 *o) const {
        const uint4 u = *at(stage, k0 + v * V);
        if constexpr (V == 1) {
            o[0] = widen2<T>(u.x), o[1] = widen2<T>(u.y), o[2] = widen2<T>(u.z), o[3] = widen2<T>(u.w);
        } else {
            const uint4 x = *at(stage, k0 + v * V + 1);
            o[0] = pack2(__uint_as_float(u.x), __uint_as_float(u.y)), o[1] = pack2(__uint_as_float(u.z), __uint_as_float(u.w));
            o[2] = pack2(__uint_as_float(x.x), __uint_as_float(x.y)), o[3] = pack2(__uint_as_float(x.z), __uint_as_float(x.w));
        }
    }
};

// Each block walks rows and keeps its threads' share of dw in registers; the per-block sums are added by
// reduce_rows_kernel in a fixed order.  The next row comes by asynchronous copies while this one is worked on, and both
// passes over a row read it from shared memory, so that no registers hold rows.  With a later gradient, bf16, cold caches:
// 8192 x 4096 46 us for 268 MB, 5.8 TB/s, at two blocks an SM (three, at 80 registers, take 4 us more), and 8 us of reduction;
// 2048 x 16384 58 us with the reduction for 268 MB (103 with rows in registers, loaded twice).
template <typename T, int NV, int BT, bool F32>
__global__ void __launch_bounds__(BT, BT > 256 ? 1 : 2) norm_bwd_kernel(const NormArgs a) {
    using R = BwdRows<NV, BT, F32>;
    constexpr int P = 4 * NV, VH = R::VH, AHEAD = R::stages - 1;
    __shared__ float2 s_sum[2][16];
    extern __shared__ __align__(16) float s_dyn[];   // the rows; then, with several rows a block, their shares of dw
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x & (tpr - 1), D = a.D;
    const int rpb = blockDim.x / tpr, lanes = min(tpr, 32), wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_d = 1.0f / (float)D;
    const long long step = (long long)gridDim.x * rpb;
    const R rows(s_dyn, a.res != nullptr);
    auto fetch = [&](long long row, int stage) {
        const bool in = row < a.rows;
        rows.template copy<VH>(stage, R::H, a.x, row * a.x_ld, tpr, t, D, in);
        rows.template copy<1>(stage, R::G, a.dy, row * D, tpr, t, D, in);
        if (a.res) rows.template copy<VH>(stage, R::E, a.res, row * D, tpr, t, D, in);
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    long long row = (long long)blockIdx.x * rpb + slot;
    fetch(row, 0);
    f2 w[P], dw[P];
    load_weight<T, NV>(a, t, w);
#pragma unroll
    for (int i = 0; i < P; ++i) dw[i] = 0ull;
    int parity = 0;
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < a.rows; r0 += step, row += step, parity ^= 1) {
        const bool live = row < a.rows;
        const int stage = AHEAD ? parity : 0;
        if (AHEAD) fetch(row + step, stage ^ 1);
        asm volatile("cp.async.wait_group %0;\n" ::"n"(AHEAD) : "memory");
        f2 ss2 = 0ull, sd2 = 0ull;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            f2 h[4], g[4];
            rows.template get<T, VH>(stage, R::H, v, h);
            rows.template get<T, 1>(stage, R::G, v, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ss2 = fma2(h[i], h[i], ss2);
                sd2 = fma2(mul2(g[i], w[v * 4 + i]), h[i], sd2);
            }
        }
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
        const float r = live ? rsqrtf(fmaf(ss, inv_d, a.eps)) : 0.f;  // (no row: with eps = 0 the factor would be infinite)
        const f2 r2 = both(r), k2 = both(-(r * (sd * inv_d)) * r * r), one = both(D == 1 ? a.eps * r * r * r : r);
        f2 out[P];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            f2 h[4], g[4], e[4] = {0ull, 0ull, 0ull, 0ull};
            rows.template get<T, VH>(stage, R::H, v, h);
            rows.template get<T, 1>(stage, R::G, v, g);
            if (a.res) rows.template get<T, VH>(stage, R::E, v, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dw[v * 4 + i] = fma2(g[i], mul2(h[i], r2), dw[v * 4 + i]);
                out[v * 4 + i] = add2(e[i], dh_pair(g[i], w[v * 4 + i], h[i], one, k2, D == 1));
            }
        }
        if (!AHEAD) fetch(row + step, 0);
        if (live) {
            store_row<T, NV, false>(a.dx, row * D, tpr, t, D, out);
            if (F32 && a.dres) store_row<T, NV, true>(a.dres, row * D, tpr, t, D, out);
        }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    if (rpb == 1) {
        store_row<T, NV, true>(a.dw_part, (long long)blockIdx.x * D, tpr, t, D, dw);
    } else {
        __syncthreads();  // (the rows are read no more)
        store_row<T, NV, true>(s_dyn, slot * D, tpr, t, D, dw);
        __syncthreads();
        sum_slots(a, s_dyn, rpb);
    }
}

// ---------------------------------------------------------------- ragged rows

// Rows of one tensor on their way into shared memory: `bytes` each from row_at(row), as the aligned 16-byte pieces that
// hold them, cut off at the tensor's ends; row r's data then begins skew(r) bytes into its place.
struct RagRows {
    const char *base, *hi;
    long long ld;  // bytes between rows
    int bytes;
    __device__ __forceinline__ RagRows(const void *p, long long ld_, long long rows, int D, int elem)
        : base(static_cast<const char *>(p)), hi(base + (rows - 1) * ld_ * elem + (long long)D * elem), ld(ld_ * elem), bytes(D * elem) {}
    __device__ __forceinline__ int skew(long long row) const { return (int)(reinterpret_cast<uintptr_t>(base + row * ld) & 15); }
    __device__ __forceinline__ void copy(char *to, long long row, int t, int tpr, int elem) const {
        const uintptr_t at = reinterpret_cast<uintptr_t>(base + row * ld);
        const int sk = (int)(at & 15), pieces = (sk + bytes + 15) / 16;
        for (int k = t; k < pieces; k += tpr) {
            const char *src = reinterpret_cast<const char *>(at - sk) + k * 16;
            if (src >= base) {
                const long long left = hi - src;
                const int n = left < 16 ? (int)left : 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(to + k * 16)), "l"(src), "r"(n) : "memory");
            } else {  // the piece begins before the tensor
                for (int i = sk; i < 16 && i - sk < bytes; i += 2)
                    *reinterpret_cast<uint16_t *>(to + i) = *reinterpret_cast<const uint16_t *>(src + i);
            }
        }
    }
};
// Bytes of a row's place.
__host__ __device__ constexpr int rag_place(int D, int elem) { return (D * elem + 14 + 15) / 16 * 16; }

template <typename T, bool F32>
__device__ __forceinline__ float rag_get(const char *row, int c) {
    if (F32) return *reinterpret_cast<const float *>(row + 4 * c);
    return Elt<T>::to_f(*reinterpret_cast<const T *>(row + 2 * c));
}
template <typename T, bool F32>
__device__ __forceinline__ void rag_put(void *to, long long at, float v) {
    if (F32) static_cast<float *>(to)[at] = v;
    else static_cast<T *>(to)[at] = Elt<T>::from_f(v);
}
__device__ __forceinline__ void rag_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void rag_arrive() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(LEFT) : "memory");
    __syncthreads();
}

// Registers: 16 columns a thread in blocks of up to 288 threads leave two blocks an SM, up to 512 one.
template <int EPT, int BT>
struct RagBounds {
    static constexpr int blocks = BT <= 288 ? 2 : 1;
};

template <typename T, int EPT, int BT, bool QUANT, int RES>
__global__ void __launch_bounds__(BT, RagBounds<EPT, BT>::blocks) norm_fwd_ragged_kernel(const NormArgs a, int rpb, int stages) {
    constexpr bool RF = RES == RES_F32;
    __shared__ float s_sum[2][16];
    extern __shared__ __align__(16) char s_rows[];  // [stages][rpb](x, residual), then the maxima of each 32 columns
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x - slot * tpr, D = a.D, wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int px = rag_place(D, 2), pr = RES == RES_NONE ? 0 : rag_place(D, RF ? 4 : 2), place = px + pr;
    const RagRows X(a.x, a.x_ld, a.rows, D, 2), R(RES == RES_NONE ? a.x : a.res, D, a.rows, D, RF ? 4 : 2);
    const float inv_d = 1.0f / (float)D;
    const long long step = (long long)gridDim.x * rpb;
    const int chunks = wpr * EPT;                    // of 32 columns a row
    float *s_chunk = reinterpret_cast<float *>(s_rows + (size_t)stages * rpb * place) + slot * chunks;
    auto fetch = [&](long long row, int stage) {
        if (row < a.rows) {
            char *to = s_rows + (size_t)(stage * rpb + slot) * place;
            X.copy(to, row, t, tpr, 2);
            if (RES != RES_NONE) R.copy(to + px, row, t, tpr, RF ? 4 : 2);
        }
        rag_commit();
    };
    long long row = (long long)blockIdx.x * rpb + slot;
    if (stages == 2) fetch(row, 0);
    float w[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) w[j] = t + j * tpr < D ? load_gate<T>(a.w, t + j * tpr, a.w_f32) : 0.f;
    int parity = 0;
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < a.rows; r0 += step, row += step, parity ^= 1) {
        const int stage = stages == 2 ? parity : 0;
        if (stages == 2) {
            fetch(row + step, stage ^ 1);
            rag_arrive<1>();
        } else {
            __syncthreads();  // (the place has been read)
            fetch(row, 0);
            rag_arrive<0>();
        }
        const bool live = row < a.rows;
        const char *at = s_rows + (size_t)(stage * rpb + slot) * place;
        const char *x = at + X.skew(row), *e = at + px + R.skew(row);
        float h[EPT], ss = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = t + j * tpr;
            h[j] = 0.f;
            if (live && c < D) {
                h[j] = rag_get<T, false>(x, c);
                if (RES != RES_NONE) {
                    h[j] += rag_get<T, RF>(e, c);
                    rag_put<T, RF>(a.res_out, row * D + c, h[j]);
                }
            }
            ss = fmaf(h[j], h[j], ss);
        }
        ss = lanes_sum(ss, 32);
        if (tpr > 32) {
            if (lane == 0) s_sum[parity][warp] = ss;
            __syncthreads();
            ss = 0.f;
            for (int i = 0; i < wpr; ++i) ss += s_sum[parity][slot * wpr + i];
        }
        const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            h[j] *= r * w[j];
            if (!QUANT && live && t + j * tpr < D) rag_put<T, false>(a.y, row * D + t + j * tpr, h[j]);
        }
        if constexpr (QUANT) {
            // magnitudes of each 32 columns, then of the scale's
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h[j]) & 0x7fffffffu);
                if (lane == 0) s_chunk[j * wpr + (t >> 5)] = __uint_as_float(m);
            }
            __syncthreads();
            // one thread a scale: the largest of its columns' maxima, which the scale's quotient then replaces
            const int used = (D + 31) / 32;
            Quotient own[2];
            if (a.group) {
                for (int i = 0, q = t; q < a.nscale; ++i, q += tpr) {
                    float m = s_chunk[4 * q];
#pragma unroll
                    for (int k = 1; k < 4; ++k)
                        if (4 * q + k < used) m = max_abs(m, s_chunk[4 * q + k]);
                    const float scale = scale_of(m);
                    own[i & 1] = Quotient(scale);
                    if (live) a.scale[row * a.nscale + q] = scale;
                }
            } else {
                float m = 0.f;
                for (int i = lane; i < used; i += 32) m = max_abs(m, s_chunk[i]);
                const float scale = scale_of(lanes_max(m, 32));
                own[0] = Quotient(scale);
                if (live && t == 0) a.scale[row] = scale;
            }
            if (a.group) {
                __syncthreads();
                for (int i = 0, q = t; q < a.nscale; ++i, q += tpr) *reinterpret_cast<Quotient *>(s_chunk + 4 * q) = own[i & 1];
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                const int c = t + j * tpr;
                if (!(live && c < D)) continue;
                const float q = a.group ? reinterpret_cast<const Quotient *>(s_chunk + (c >> 7) * 4)->of(h[j]) : own[0].of(h[j]);
                static_cast<unsigned char *>(a.y)[row * D + c] = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
            }
            __syncthreads();  // (the maxima have been read)
        }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}

template <typename T, int EPT, int BT, bool F32>
__global__ void __launch_bounds__(BT, RagBounds<EPT, BT>::blocks) norm_bwd_ragged_kernel(const NormArgs a, int rpb, int stages) {
    __shared__ float2 s_sum[2][16];
    extern __shared__ __align__(16) char s_rows[];  // [stages][rpb](h, dy, dresidual)
    const int tpr = a.tpr, slot = threadIdx.x / tpr, t = threadIdx.x - slot * tpr, D = a.D, wpr = tpr >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int HE = F32 ? 4 : 2;
    const int ph = rag_place(D, HE), pg = rag_place(D, 2), place = ph + pg + (a.res ? ph : 0);
    const RagRows H(a.x, a.x_ld, a.rows, D, HE), G(a.dy, D, a.rows, D, 2), E(a.res ? a.res : a.dy, D, a.rows, D, HE);
    const float inv_d = 1.0f / (float)D;
    const long long step = (long long)gridDim.x * rpb;
    auto fetch = [&](long long row, int stage) {
        if (row < a.rows) {
            char *to = s_rows + (size_t)(stage * rpb + slot) * place;
            H.copy(to, row, t, tpr, HE);
            G.copy(to + ph, row, t, tpr, 2);
            if (a.res) E.copy(to + ph + pg, row, t, tpr, HE);
        }
        rag_commit();
    };
    long long row = (long long)blockIdx.x * rpb + slot;
    if (stages == 2) fetch(row, 0);
    float w[EPT], dw[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        w[j] = t + j * tpr < D ? load_gate<T>(a.w, t + j * tpr, a.w_f32) : 0.f;
        dw[j] = 0.f;
    }
    int parity = 0;
    for (long long r0 = (long long)blockIdx.x * rpb; r0 < a.rows; r0 += step, row += step, parity ^= 1) {
        const int stage = stages == 2 ? parity : 0;
        if (stages == 2) {
            // (the other stage was read up to the barrier below, or, with rows of one warp, by this warp)
            if (tpr == 32) __syncthreads();
            fetch(row + step, stage ^ 1);
            rag_arrive<1>();
        } else {
            __syncthreads();
            fetch(row, 0);
            rag_arrive<0>();
        }
        const bool live = row < a.rows;
        const char *at = s_rows + (size_t)(stage * rpb + slot) * place;
        const char *h = at + H.skew(row), *g = at + ph + G.skew(row), *e = at + ph + pg + E.skew(row);
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = t + j * tpr;
            if (live && c < D) {
                const float hv = rag_get<T, F32>(h, c), gv = rag_get<T, false>(g, c);
                ss = fmaf(hv, hv, ss);
                sd = fmaf(gv * w[j], hv, sd);
            }
        }
        ss = lanes_sum(ss, 32);
        sd = lanes_sum(sd, 32);
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
        const float k2 = -(r * (sd * inv_d)) * r * r, one = D == 1 ? a.eps * r * r * r : r;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = t + j * tpr;
            if (!(live && c < D)) continue;
            const float hv = rag_get<T, F32>(h, c), gv = rag_get<T, false>(g, c);
            dw[j] = fmaf(gv, hv * r, dw[j]);
            float d = gv * w[j] * one;
            if (D != 1) d = fmaf(hv, k2, d);
            if (a.res) d += rag_get<T, F32>(e, c);
            rag_put<T, false>(a.dx, row * D + c, d);
            if (F32 && a.dres) static_cast<float *>(a.dres)[row * D + c] = d;
        }
        if (stages == 2 && tpr > 32) __syncthreads();  // (this stage is the next copies' place)
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();
    float *slots = reinterpret_cast<float *>(s_rows);  // (a row's place holds at least 4 bytes a column)
#pragma unroll
    for (int j = 0; j < EPT; ++j)
        if (t + j * tpr < D) slots[slot * D + t + j * tpr] = dw[j];
    __syncthreads();
    sum_slots(a, slots, rpb);
}

template <typename T, int NV, int BT>
cudaError_t norm_fwd_v(const NormArgs &a, int blocks, bool quant, int res, cudaStream_t st) {
    const dim3 g(blocks), b(BT);
    if (quant) {
        if (res == RES_NONE) return launch_plain(norm_fwd_kernel<T, NV, BT, true, RES_NONE>, g, b, 0, st, a);
        if (res == RES_HALF) return launch_plain(norm_fwd_kernel<T, NV, BT, true, RES_HALF>, g, b, 0, st, a);
        return launch_plain(norm_fwd_kernel<T, NV, BT, true, RES_F32>, g, b, 0, st, a);
    }
    if (res == RES_NONE) return launch_plain(norm_fwd_kernel<T, NV, BT, false, RES_NONE>, g, b, 0, st, a);
    if (res == RES_HALF) return launch_plain(norm_fwd_kernel<T, NV, BT, false, RES_HALF>, g, b, 0, st, a);
    return launch_plain(norm_fwd_kernel<T, NV, BT, false, RES_F32>, g, b, 0, st, a);
}

// Two rows' places where they fit beside another block's, else one.
template <typename K>
cudaError_t launch_ragged(K k, const NormArgs &a, const NormShape &s, int blocks, size_t place, size_t extra, cudaStream_t st) {
    const size_t one = (size_t)s.rpb * place;
    const int stages = 2 * one + extra <= 100 * 1024 ? 2 : 1;
    const size_t smem = stages * one + extra;
    const cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
    return launch_plain(k, dim3(blocks), dim3(s.threads), smem, st, a, s.rpb, stages);
}
template <typename T, int EPT, int BT>
cudaError_t norm_fwd_r(const NormArgs &a, const NormShape &s, int n, bool quant, int res, cudaStream_t st) {
    const size_t place = rag_place(a.D, 2) + (res == RES_NONE ? 0 : rag_place(a.D, res == RES_F32 ? 4 : 2));
    const size_t extra = quant ? (size_t)s.threads / 32 * EPT * sizeof(float) : 0;
    if (quant) {
        if (res == RES_NONE) return launch_ragged(norm_fwd_ragged_kernel<T, EPT, BT, true, RES_NONE>, a, s, n, place, extra, st);
        if (res == RES_HALF) return launch_ragged(norm_fwd_ragged_kernel<T, EPT, BT, true, RES_HALF>, a, s, n, place, extra, st);
        return launch_ragged(norm_fwd_ragged_kernel<T, EPT, BT, true, RES_F32>, a, s, n, place, extra, st);
    }
    if (res == RES_NONE) return launch_ragged(norm_fwd_ragged_kernel<T, EPT, BT, false, RES_NONE>, a, s, n, place, extra, st);
    if (res == RES_HALF) return launch_ragged(norm_fwd_ragged_kernel<T, EPT, BT, false, RES_HALF>, a, s, n, place, extra, st);
    return launch_ragged(norm_fwd_ragged_kernel<T, EPT, BT, false, RES_F32>, a, s, n, place, extra, st);
}
template <typename T>
cudaError_t norm_fwd_t(const NormArgs &a, const NormShape &s, bool vec, bool quant, int res, cudaStream_t st) {
    const int n = norm_blocks(a.rows, s, false, !vec);
    if (vec) {
        if (s.nv == 4) return norm_fwd_v<T, 4, 512>(a, n, quant, res, st);
        return s.threads == 256 ? norm_fwd_v<T, 2, 256>(a, n, quant, res, st) : norm_fwd_v<T, 2, 512>(a, n, quant, res, st);
    }
    if (a.D <= 128) return norm_fwd_r<T, 4, 288>(a, s, n, quant, res, st);
    if (s.nv == 4) return norm_fwd_r<T, 32, 512>(a, s, n, quant, res, st);
    return s.threads <= 288 ? norm_fwd_r<T, 16, 288>(a, s, n, quant, res, st) : norm_fwd_r<T, 16, 512>(a, s, n, quant, res, st);
}
template <typename K>
cudaError_t launch_wide(K k, int blocks, int threads, size_t smem, const NormArgs &a, cudaStream_t st) {
    const cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
    return launch_plain(k, dim3(blocks), dim3(threads), smem, st, a);
}
template <typename T, int NV, int BT>
cudaError_t norm_bwd_v(const NormArgs &a, int blocks, bool f32, cudaStream_t st) {
    // (the shares of dw, at most 4 bytes a column of a thread, fit in the rows' place)
    if (f32) return launch_wide(norm_bwd_kernel<T, NV, BT, true>, blocks, BT, BwdRows<NV, BT, true>::bytes(a.res), a, st);
    return launch_wide(norm_bwd_kernel<T, NV, BT, false>, blocks, BT, BwdRows<NV, BT, false>::bytes(a.res), a, st);
}
template <typename T, int EPT, int BT>
cudaError_t norm_bwd_r(const NormArgs &a, const NormShape &s, int n, bool f32, cudaStream_t st) {
    const size_t ph = rag_place(a.D, f32 ? 4 : 2), place = ph + rag_place(a.D, 2) + (a.res ? ph : 0);
    if (f32) return launch_ragged(norm_bwd_ragged_kernel<T, EPT, BT, true>, a, s, n, place, 0, st);
    return launch_ragged(norm_bwd_ragged_kernel<T, EPT, BT, false>, a, s, n, place, 0, st);
}
template <typename T>
cudaError_t norm_bwd_t(const NormArgs &a, const NormShape &s, bool vec, bool f32, int n, cudaStream_t st) {
    if (vec) {
        if (s.nv == 4) return norm_bwd_v<T, 4, 512>(a, n, f32, st);
        return s.threads == 256 ? norm_bwd_v<T, 2, 256>(a, n, f32, st) : norm_bwd_v<T, 2, 512>(a, n, f32, st);
    }
    if (a.D <= 128) return norm_bwd_r<T, 4, 288>(a, s, n, f32, st);
    if (s.nv == 4) return norm_bwd_r<T, 32, 512>(a, s, n, f32, st);
    return s.threads <= 288 ? norm_bwd_r<T, 16, 288>(a, s, n, f32, st) : norm_bwd_r<T, 16, 512>(a, s, n, f32, st);
}

}  // namespace
}  // namespace norm
}  // namespace gdr
