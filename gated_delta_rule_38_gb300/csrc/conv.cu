// Short causal convolution of every channel with its own W taps (2 <= W <= 4), optionally through SiLU, over dense
// rows or packed sequences, from cached inputs, and its backward pass.
//
//   pre_t = b + sum_{j<W} w_{W-1-j} x_{t-j};   y_t = pre_t  or  pre_t sigmoid(pre_t)
//   backward: dpre_t = dy_t (sig + pre sig (1 - sig));  dx_s = sum_j w_{W-1-j} dpre_{s+j} (same sequence only);
//             dw_{W-1-j} = sum_t dpre_t x_{t-j};  db = sum_t dpre_t
// Inputs before a sequence's first token are its W - 1 cached ones (state [N, W-1, D]) or zeros; their gradients
// come out as if they were tokens of it.
//
// A thread walks TT tokens of VEC channels with the last W - 1 inputs (backward: also the W - 1 open sums of dx) in
// registers, so every element is read and written once but for W - 1 tokens of overlap between neighbouring walks:
// the kernels are bound by HBM.  A block is 32 lanes along the channels (one contiguous row segment a warp) by 8
// walks.  All sums are fp32.
#include <cuda_runtime.h>

#include "common.cuh"
#include "host.h"
#include "launch.h"
#include "seqwalk.cuh"

namespace gdr {
namespace {

constexpr int WALKS = 8;  // walks (warps) of a block

struct ConvArgs {
    const void *x, *w, *bias, *state_in;
    void *y, *state_out;
    const void *dy, *dstate_out;   // backward: gradients of y and of the final states
    void *dx, *dstate_in;
    float *dw_part, *db_part;      // backward: [blocks along the tokens][D * W] and [..][D]
    const int32_t *cu;
    unsigned *err;
    long long x_ld;
    int B, T, D, N;
    int tt, tiles, cblocks;        // tokens a walk; walks a row; blocks along the channels
    bool w_f32, silu;
};

// N consecutive parameters of type T or fp32 as fp32.
template <typename T, int N>
__device__ __forceinline__ void load_params(const void *p, long long at, bool f32, float *o) {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = load_gate<T>(p, at + i, f32);
}

template <typename T, int VEC>
__device__ __forceinline__ void load_x(const T *p, float *o) {
    if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Elt<T>::unpack(r[i]);
            o[2 * i] = f.x, o[2 * i + 1] = f.y;
        }
    } else if constexpr (VEC == 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        const float2 f = Elt<T>::unpack(u.x), g = Elt<T>::unpack(u.y);
        o[0] = f.x, o[1] = f.y, o[2] = g.x, o[3] = g.y;
    } else {
        o[0] = Elt<T>::to_f(p[0]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_x(T *p, const float *v) {
    if constexpr (VEC == 8) {
        uint4 u;
        u.x = Elt<T>::pack(v[0], v[1]), u.y = Elt<T>::pack(v[2], v[3]);
        u.z = Elt<T>::pack(v[4], v[5]), u.w = Elt<T>::pack(v[6], v[7]);
        *reinterpret_cast<uint4 *>(p) = u;
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(Elt<T>::pack(v[0], v[1]), Elt<T>::pack(v[2], v[3]));
    } else {
        p[0] = Elt<T>::from_f(v[0]);
    }
}

__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// The cached inputs of sequence n (zeros without them): xs[j-1] = input j tokens before its first.
template <typename T, int VEC, int W>
__device__ __forceinline__ void cached_inputs(const ConvArgs &a, long long n, int c, float (*xs)[VEC]) {
#pragma unroll
    for (int j = 1; j < W; ++j) {
        if (a.state_in) {
            load_x<T, VEC>(static_cast<const T *>(a.state_in) + (n * (W - 1) + (W - 1 - j)) * a.D + c, xs[j - 1]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) xs[j - 1][i] = 0.f;
        }
    }
}

// The W - 1 inputs before token t0 of a sequence that starts at `start` (both tokens of the row at `row`).
template <typename T, int VEC, int W>
__device__ __forceinline__ void inputs_before(const ConvArgs &a, const T *row, int t0, int start, long long n, int c,
                                              float (*xs)[VEC]) {
    if (t0 - start < W - 1) cached_inputs<T, VEC, W>(a, n, c, xs);
    float past[W - 1][VEC];
#pragma unroll
    for (int j = 1; j < W; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) past[j - 1][i] = xs[j - 1][i];
#pragma unroll
    for (int j = 1; j < W; ++j) {
        if (t0 - j >= start) {
            load_x<T, VEC>(row + (long long)(t0 - j) * a.x_ld + c, xs[j - 1]);
        } else {
            // j - (t0 - start) tokens before the start: one of the cached inputs
#pragma unroll
            for (int k = 1; k < W; ++k)
                if (k == j - (t0 - start))
#pragma unroll
                    for (int i = 0; i < VEC; ++i) xs[j - 1][i] = past[k - 1][i];
        }
    }
}

// Block -> channel of this lane and (row, first token) of this warp's walk; false past either end.
template <int VEC>
__device__ __forceinline__ bool my_walk(const ConvArgs &a, int &c, int &b, int &t0, long long &tblock) {
    tblock = blockIdx.x / (unsigned)a.cblocks;
    c = ((int)(blockIdx.x - tblock * a.cblocks) * 32 + (int)threadIdx.x) * VEC;
    const long long walk = tblock * WALKS + threadIdx.y;
    b = (int)(walk / a.tiles);
    t0 = (int)(walk - (long long)b * a.tiles) * a.tt;
    return c < a.D && b < a.B;
}

template <typename T, int VEC, int W, bool PACKED>
__global__ void __launch_bounds__(32 * WALKS) conv_fwd_kernel(const ConvArgs a) {
    constexpr int U = 8;  // tokens in flight
    if (PACKED && blockIdx.x == 0 && threadIdx.y == 0) check_cu(a.cu, a.N, a.T, a.err);
    int c, b, t0;
    long long tblock;
    if (!my_walk<VEC>(a, c, b, t0, tblock)) return;
    const int t1 = min(a.T, t0 + a.tt);
    const T *row = static_cast<const T *>(a.x) + (long long)b * a.T * a.x_ld;
    T *out = static_cast<T *>(a.y) + (long long)b * a.T * a.D + c;

    float wp[VEC * W], bias[VEC], xs[W - 1][VEC];
    load_params<T, VEC * W>(a.w, (long long)c * W, a.w_f32, wp);
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = 0.f;
    if (a.bias) load_params<T, VEC>(a.bias, c, a.w_f32, bias);

    SeqWalk sw;
    if (PACKED) sw.find(a.cu, a.N, t0);
    long long seq = PACKED ? sw.cur() : b;
    if (!PACKED) {
        inputs_before<T, VEC, W>(a, row, t0, 0, seq, c, xs);
    } else if (sw.bound != t0) {
        inputs_before<T, VEC, W>(a, row, t0, max(0, a.cu[seq]), seq, c, xs);
    } else {
        cached_inputs<T, VEC, W>(a, seq, c, xs);  // (replaced at the first token)
    }
    auto write_state = [&](long long n, const float(*s)[VEC]) {
        if (!a.state_out) return;
#pragma unroll
        for (int j = 1; j < W; ++j)
            store_x<T, VEC>(static_cast<T *>(a.state_out) + (n * (W - 1) + (W - 1 - j)) * a.D + c, s[j - 1]);
    };
    auto empty = [&](long long n) {
        float e[W - 1][VEC];
        cached_inputs<T, VEC, W>(a, n, c, e);
        write_state(n, e);
    };

    for (int t = t0; t < t1; t += U) {
        float x[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1) load_x<T, VEC>(row + (long long)(t + u) * a.x_ld + c, x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            if (PACKED && t + u == sw.bound) {
                if (sw.step(t + u, empty)) {
                    seq = sw.cur();
                    cached_inputs<T, VEC, W>(a, seq, c, xs);
                }
            }
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float pre = fmaf(wp[i * W + W - 1], x[u][i], bias[i]);
#pragma unroll
                for (int j = 1; j < W; ++j) pre = fmaf(wp[i * W + W - 1 - j], xs[j - 1][i], pre);
                y[i] = a.silu ? pre * sigmoid_fast(pre) : pre;
            }
            store_x<T, VEC>(out + (long long)(t + u) * a.D, y);
#pragma unroll
            for (int j = W - 1; j > 1; --j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) xs[j - 1][i] = xs[j - 2][i];
#pragma unroll
            for (int i = 0; i < VEC; ++i) xs[0][i] = x[u][i];
            if (PACKED && t + u + 1 == sw.bound) write_state(seq, xs);
        }
    }
    if (!PACKED && t1 == a.T) write_state(seq, xs);
    if (PACKED && t1 == a.T && sw.bound == a.T) sw.step(a.T, empty);
}

template <typename T, int VEC, int W, bool PACKED>
__global__ void __launch_bounds__(32 * WALKS) conv_bwd_kernel(const ConvArgs a) {
    constexpr int U = 4;
    constexpr int NP = VEC * (W + 1);
    __shared__ float s_part[WALKS][NP][32];
    if (PACKED && blockIdx.x == 0 && threadIdx.y == 0) check_cu(a.cu, a.N, a.T, a.err);
    int c, b, t0;
    long long tblock;
    const bool live = my_walk<VEC>(a, c, b, t0, tblock);
    float wp[VEC * W], dw[VEC * W], db[VEC];
#pragma unroll
    for (int i = 0; i < VEC * W; ++i) dw[i] = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) db[i] = 0.f;
    if (live) {
        const int t1 = min(a.T, t0 + a.tt);
        const T *row = static_cast<const T *>(a.x) + (long long)b * a.T * a.x_ld;
        const T *dy = static_cast<const T *>(a.dy) + (long long)b * a.T * a.D + c;
        T *dx = static_cast<T *>(a.dx) + (long long)b * a.T * a.D + c;
        float bias[VEC], xs[W - 1][VEC], acc[W - 1][VEC];  // acc[j-1]: the open sum of dx, j tokens back
        load_params<T, VEC * W>(a.w, (long long)c * W, a.w_f32, wp);
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = 0.f;
        if (a.bias) load_params<T, VEC>(a.bias, c, a.w_f32, bias);
#pragma unroll
        for (int j = 1; j < W; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[j - 1][i] = 0.f;

        SeqWalk sw;
        if (PACKED) sw.find(a.cu, a.N, t0);
        long long seq = PACKED ? sw.cur() : b;
        int start = 0;
        if (PACKED && sw.bound != t0) start = max(0, a.cu[seq]);
        if (!PACKED || sw.bound != t0)
            inputs_before<T, VEC, W>(a, row, t0, start, seq, c, xs);
        else
            cached_inputs<T, VEC, W>(a, seq, c, xs);  // (replaced at the first token)
        // A finished sum: of an input of this walk, or of a cached input of a sequence that starts in it.
        auto emit = [&](int s, const float *v) {
            if (s >= start) {
                if (s >= t0 && s < t1) store_x<T, VEC>(dx + (long long)s * a.D, v);
            } else if (start >= t0 && a.dstate_in && W - 1 + s - start >= 0) {
                store_x<T, VEC>(static_cast<T *>(a.dstate_in) + (seq * (W - 1) + (W - 1 + s - start)) * a.D + c, v);
            }
        };
        // The last W - 1 sums of a sequence that ends at token e: also the final state's gradient.
        auto flush = [&](int e) {
#pragma unroll
            for (int j = W - 1; j >= 1; --j) {
                if (a.dstate_out) {
                    float d[VEC];
                    load_x<T, VEC>(static_cast<const T *>(a.dstate_out) + (seq * (W - 1) + (W - 1 - j)) * a.D + c, d);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[j - 1][i] += d[i];
                }
                emit(e - j, acc[j - 1]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[j - 1][i] = 0.f;
            }
        };
        auto empty = [&](long long n) {
            if (!a.dstate_in) return;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                float d[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[i] = 0.f;
                if (a.dstate_out) load_x<T, VEC>(static_cast<const T *>(a.dstate_out) + (n * (W - 1) + j) * a.D + c, d);
                store_x<T, VEC>(static_cast<T *>(a.dstate_in) + (n * (W - 1) + j) * a.D + c, d);
            }
        };

        const int tend = min(a.T, t1 + W - 1);  // the sums of the last W - 1 inputs close past the walk's end
        bool open = true;                       // a sequence of this walk is still to be flushed
        for (int t = t0; open && t < tend; t += U) {
            float x[U][VEC], g[U][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < tend) {
                    load_x<T, VEC>(row + (long long)(t + u) * a.x_ld + c, x[u]);
                    load_x<T, VEC>(dy + (long long)(t + u) * a.D, g[u]);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!open || t + u >= tend) break;
                if (PACKED && t + u == sw.bound) {
                    if (t + u > t0) flush(t + u);
                    if (t + u >= t1) {
                        open = false;
                        break;
                    }
                    if (sw.step(t + u, empty)) {
                        seq = sw.cur();
                        start = t + u;
                        cached_inputs<T, VEC, W>(a, seq, c, xs);
                    }
                }
                const bool mine = t + u < t1;
                float done[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float d = g[u][i];
                    if (a.silu) {
                        float pre = fmaf(wp[i * W + W - 1], x[u][i], bias[i]);
#pragma unroll
                        for (int j = 1; j < W; ++j) pre = fmaf(wp[i * W + W - 1 - j], xs[j - 1][i], pre);
                        const float s = sigmoid_fast(pre);
                        d *= fmaf(pre * s, 1.f - s, s);
                    }
                    done[i] = fmaf(wp[i * W], d, acc[W - 2][i]);
#pragma unroll
                    for (int j = W - 2; j >= 1; --j) acc[j][i] = fmaf(wp[i * W + W - 1 - j], d, acc[j - 1][i]);
                    acc[0][i] = wp[i * W + W - 1] * d;
                    const float dm = mine ? d : 0.f;
                    dw[i * W + W - 1] = fmaf(dm, x[u][i], dw[i * W + W - 1]);
#pragma unroll
                    for (int j = 1; j < W; ++j)
                        dw[i * W + W - 1 - j] = fmaf(dm, xs[j - 1][i], dw[i * W + W - 1 - j]);
                    db[i] += dm;
#pragma unroll
                    for (int j = W - 1; j > 1; --j) xs[j - 1][i] = xs[j - 2][i];
                    xs[0][i] = x[u][i];
                }
                emit(t + u - (W - 1), done);
            }
        }
        if (open && tend == a.T && (!PACKED || sw.bound == a.T)) flush(a.T);
        if (PACKED && t1 == a.T && sw.bound == a.T) sw.step(a.T, empty);
    }
    // the block's share of dw and db: its walks added in order
#pragma unroll
    for (int i = 0; i < VEC * W; ++i) s_part[threadIdx.y][i][threadIdx.x] = dw[i];
#pragma unroll
    for (int i = 0; i < VEC; ++i) s_part[threadIdx.y][VEC * W + i][threadIdx.x] = db[i];
    __syncthreads();
    if (c >= a.D) return;
    for (int i = threadIdx.y; i < NP; i += WALKS) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < WALKS; ++k) s += s_part[k][i][threadIdx.x];
        if (i < VEC * W)
            a.dw_part[tblock * a.D * W + (long long)c * W + i] = s;
        else if (a.db_part)
            a.db_part[tblock * a.D + c + i - VEC * W] = s;
    }
}

// Tokens a walk: long walks repeat fewer overlapping reads, short ones fill the chip; the longest of 64, 32, 16 and
// 8 that still gives two blocks an SM.
int conv_tt(const gdr_conv_problem *p, int vec) {
    const long long cb = (p->D + 32 * vec - 1) / (32 * vec);
    int tt = 64;
    for (; tt > 8; tt /= 2) {
        const long long walks = (long long)p->B * ((p->T + tt - 1) / tt);
        if ((walks + WALKS - 1) / WALKS * cb >= 2 * kSMs) break;
    }
    return tt;
}

struct ConvGrid {
    int tt, tiles, cblocks;
    long long tblocks;
};
ConvGrid conv_grid(const gdr_conv_problem *p, int vec, int tt) {
    ConvGrid g;
    g.tt = tt;
    g.tiles = (p->T + g.tt - 1) / g.tt;
    g.cblocks = (p->D + 32 * vec - 1) / (32 * vec);
    g.tblocks = ((long long)p->B * g.tiles + WALKS - 1) / WALKS;
    return g;
}

gdr_status check_conv(const gdr_conv_problem *p) {
    if (!p) return GDR_ERR_NULL;
    if (p->B < 1 || p->T < 0 || p->D < 1 || p->D > (1 << 28) || p->T > (1 << 30) || p->W < 2 || p->W > 4 || p->x_ld < p->D) return GDR_ERR_SHAPE;
    if (p->cu_seqlens && (p->B != 1 || p->num_seqs < 1)) return GDR_ERR_SHAPE;
    if (!is_half(p->dtype)) return GDR_ERR_DTYPE;
    if (p->weight_dtype != p->dtype && p->weight_dtype != GDR_FP32) return GDR_ERR_DTYPE;
    if (p->flags & ~(unsigned)GDR_CONV_SILU) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Blocks of a launch fit the grid's x dimension.
bool grid_fits(const ConvGrid &g) { return g.tblocks * g.cblocks <= 0x7fffffffLL; }

template <typename T, int VEC, bool PACKED>
cudaError_t conv_fwd_w(const ConvArgs &a, int W, const ConvGrid &g, cudaStream_t s) {
    const dim3 grid((unsigned)(g.tblocks * g.cblocks)), block(32, WALKS);
    if (W == 2) return launch_plain(conv_fwd_kernel<T, VEC, 2, PACKED>, grid, block, 0, s, a);
    if (W == 3) return launch_plain(conv_fwd_kernel<T, VEC, 3, PACKED>, grid, block, 0, s, a);
    return launch_plain(conv_fwd_kernel<T, VEC, 4, PACKED>, grid, block, 0, s, a);
}
template <typename T>
cudaError_t conv_fwd_t(const ConvArgs &a, int W, bool vec, const ConvGrid &g, cudaStream_t s) {
    if (vec) return a.cu ? conv_fwd_w<T, 8, true>(a, W, g, s) : conv_fwd_w<T, 8, false>(a, W, g, s);
    return a.cu ? conv_fwd_w<T, 1, true>(a, W, g, s) : conv_fwd_w<T, 1, false>(a, W, g, s);
}
template <typename T, int VEC, bool PACKED>
cudaError_t conv_bwd_w(const ConvArgs &a, int W, const ConvGrid &g, cudaStream_t s) {
    const dim3 grid((unsigned)(g.tblocks * g.cblocks)), block(32, WALKS);
    if (W == 2) return launch_plain(conv_bwd_kernel<T, VEC, 2, PACKED>, grid, block, 0, s, a);
    if (W == 3) return launch_plain(conv_bwd_kernel<T, VEC, 3, PACKED>, grid, block, 0, s, a);
    return launch_plain(conv_bwd_kernel<T, VEC, 4, PACKED>, grid, block, 0, s, a);
}
template <typename T>
cudaError_t conv_bwd_t(const ConvArgs &a, int W, bool vec, const ConvGrid &g, cudaStream_t s) {
    if (vec) return a.cu ? conv_bwd_w<T, 4, true>(a, W, g, s) : conv_bwd_w<T, 4, false>(a, W, g, s);
    return a.cu ? conv_bwd_w<T, 1, true>(a, W, g, s) : conv_bwd_w<T, 1, false>(a, W, g, s);
}

ConvArgs conv_args(const gdr_conv_problem *p, const ConvGrid &g, unsigned *err) {
    ConvArgs a = {};
    a.cu = p->cu_seqlens;
    a.err = err;
    a.x_ld = p->x_ld;
    a.B = p->B, a.T = p->T, a.D = p->D;
    a.N = p->cu_seqlens ? p->num_seqs : p->B;
    a.tt = g.tt, a.tiles = g.tiles, a.cblocks = g.cblocks;
    a.w_f32 = p->weight_dtype == GDR_FP32;
    a.silu = (p->flags & GDR_CONV_SILU) != 0;
    return a;
}

size_t conv_state_bytes(const gdr_conv_problem *p) {
    return (size_t)(p->cu_seqlens ? p->num_seqs : p->B) * (p->W - 1) * p->D * 2;
}

// Without tokens the states pass through: dst = src, or zeros.
gdr_status conv_no_tokens(const gdr_conv_problem *p, const void *src, void *dst, cudaStream_t s) {
    if (!dst || dst == src) return GDR_OK;
    const size_t n = conv_state_bytes(p);
    return cuda_status(src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dst, 0, n, s));
}

gdr_status conv_fwd_core(const gdr_conv_problem *p, const void *x, const void *weight, const void *bias,
                         const void *state_in, void *y, void *state_out, int tt, void *stream) {
    if (!weight || (p->T > 0 && (!x || !y))) return GDR_ERR_NULL;
    const size_t ws = esize(p->weight_dtype);
    for (const void *q : {x, state_in, (const void *)y, (const void *)state_out})
        if (!aligned_to(q, 2)) return GDR_ERR_ALIGN;
    if (!aligned_to(weight, ws) || !aligned_to(bias, ws)) return GDR_ERR_ALIGN;
    const bool vec = p->D % 8 == 0 && p->x_ld % 8 == 0 && aligned16(x) && aligned16(y) && aligned16(state_in) &&
                     aligned16(state_out);
    const ConvGrid g = conv_grid(p, vec ? 8 : 1, tt ? tt : conv_tt(p, vec ? 8 : 1));
    if (!grid_fits(g)) return GDR_ERR_SHAPE;
    unsigned *err = nullptr;
    gdr_status st = device_state(&err);
    if (st != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->T == 0) return conv_no_tokens(p, state_in, state_out, cs);
    ConvArgs a = conv_args(p, g, err);
    a.x = x, a.w = weight, a.bias = bias, a.state_in = state_in, a.y = y, a.state_out = state_out;
    return timed(K_CONV_FWD, cs, [&] {
        return p->dtype == GDR_BF16 ? conv_fwd_t<__nv_bfloat16>(a, p->W, vec, g, cs) : conv_fwd_t<__half>(a, p->W, vec, g, cs);
    });
}

}  // namespace
}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_conv_fwd(const gdr_conv_problem *p, const void *x, const void *weight, const void *bias,
                        const void *state_in, void *y, void *state_out, void *stream) {
    gdr_status st = check_conv(p);
    if (st != GDR_OK) return st;
    // (a sequence's first and last tokens belong to different threads)
    if (state_out && state_out == state_in) return GDR_ERR_UNSUPPORTED;
    return conv_fwd_core(p, x, weight, bias, state_in, y, state_out, 0, stream);
}

gdr_status gdr_conv_step(const gdr_conv_problem *p, const void *x, const void *weight, const void *bias, void *state,
                         void *y, void *stream) {
    gdr_status st = check_conv(p);
    if (st != GDR_OK) return st;
    if (p->cu_seqlens) return GDR_ERR_UNSUPPORTED;
    if (!state) return GDR_ERR_NULL;
    // one walk a row: the thread that reads a channel's cached inputs is the one that replaces them
    return conv_fwd_core(p, x, weight, bias, state, y, state, p->T > 0 ? p->T : 1, stream);
}

gdr_status gdr_conv_bwd_workspace_size(const gdr_conv_problem *p, size_t *bytes) {
    gdr_status st = check_conv(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    // (covers the wide and the narrow path, whose walks differ)
    size_t most = 0;
    if (p->T > 0)
        for (int vec : {1, 4}) {
            const ConvGrid g = conv_grid(p, vec, conv_tt(p, vec));
            const size_t n = round_up((size_t)g.tblocks * p->D * p->W * sizeof(float), 256) +
                             round_up((size_t)g.tblocks * p->D * sizeof(float), 256);
            most = n > most ? n : most;
        }
    *bytes = most;
    return GDR_OK;
}

gdr_status gdr_conv_bwd(const gdr_conv_problem *p, const void *x, const void *weight, const void *bias, const void *dy,
                        const void *state_in, const void *dstate_out, void *dx, void *dweight, void *dbias,
                        void *dstate_in, void *workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0;
    gdr_status st = gdr_conv_bwd_workspace_size(p, &need);
    if (st != GDR_OK) return st;
    if (!weight || !dweight || (dbias && !bias) || (p->T > 0 && (!x || !dy || !dx))) return GDR_ERR_NULL;
    const size_t ws = esize(p->weight_dtype);
    for (const void *q : {x, dy, state_in, dstate_out, (const void *)dx, (const void *)dstate_in})
        if (!aligned_to(q, 2)) return GDR_ERR_ALIGN;
    for (const void *q : {weight, bias, (const void *)dweight, (const void *)dbias})
        if (!aligned_to(q, ws)) return GDR_ERR_ALIGN;
    if (need && (!workspace || workspace_bytes < need)) return GDR_ERR_WORKSPACE;
    if (need && !aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    bool vec = p->D % 4 == 0 && p->x_ld % 4 == 0;
    for (const void *q : {x, dy, state_in, dstate_out, (const void *)dx, (const void *)dstate_in})
        vec = vec && aligned_to(q, 8);
    const ConvGrid g = conv_grid(p, vec ? 4 : 1, conv_tt(p, vec ? 4 : 1));
    if (!grid_fits(g)) return GDR_ERR_SHAPE;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->T == 0) {
        cudaError_t e = cudaMemsetAsync(dweight, 0, (size_t)p->D * p->W * ws, cs);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)p->D * ws, cs);
        if (e != cudaSuccess) return cuda_status(e);
        return conv_no_tokens(p, dstate_out, dstate_in, cs);
    }
    ConvArgs a = conv_args(p, g, err);
    a.x = x, a.w = weight, a.bias = bias, a.state_in = state_in, a.dy = dy, a.dstate_out = dstate_out;
    a.dx = dx, a.dstate_in = dstate_in;
    a.dw_part = static_cast<float *>(workspace);
    if (dbias)
        a.db_part = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                              round_up((size_t)g.tblocks * p->D * p->W * sizeof(float), 256));
    const bool bf = p->dtype == GDR_BF16;
    st = timed(K_CONV_BWD, cs, [&] {
        return bf ? conv_bwd_t<__nv_bfloat16>(a, p->W, vec, g, cs) : conv_bwd_t<__half>(a, p->W, vec, g, cs);
    });
    if (st != GDR_OK) return st;
    st = timed(K_REDUCE, cs, [&] {
        return launch_reduce_rows(a.dw_part, g.tblocks, (long long)p->D * p->W, p->D * p->W, dweight, bf, a.w_f32, cs);
    });
    if (st != GDR_OK || !dbias) return st;
    return timed(K_REDUCE, cs, [&] { return launch_reduce_rows(a.db_part, g.tblocks, p->D, p->D, dbias, bf, a.w_f32, cs); });
}

}  // extern "C"
