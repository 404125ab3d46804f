// What the selective scan's kernels share: the problem, the lane layout, the staging of a token tile and the
// two-element fp32 arithmetic.
//
// Lane layout.  Every thread owns 4 channels x 4 states (in registers, fp32), L lanes side by side hold one channel's
// N <= 4 L states (padded with states whose B and C are zero), and the 32 / L lane groups of a warp take consecutive
// channels.  Pairs of channels go through the two-element instructions.  Shared memory gives 128 bytes a clock to the lanes
// together, however many of them read the same address, so what a lane reads a token is kept small: 16 bytes of delta
// and of the input, and 8 bytes of B and of C in their own 16-bit type (with B and C staged as duplicated fp32 pairs
// the forward's 41 wavefronts a warp and token took 72 % of its time).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "host.h"
#include "launch.h"
#include "seqwalk.cuh"

namespace gdr {
namespace scan {

constexpr int SAVE = 16;       // tokens between saved states; segments are multiples of it

struct ScanArgs {
    const void *x, *dt, *z, *Bm, *Cm;
    const float *A, *skip, *bias, *state_in;
    void *y;
    float *state_out, *saved;
    float *seg, *segdt;    // workspace: [B][nseg][NP][DP] states at the segments' ends, [B][nseg][DP] sums of delta
    int32_t *cut;          // workspace, packed: [nseg] whether a sequence starts (backward: ends) in the segment
    // backward
    const void *dy;
    const float *dstate_out;
    void *dx, *ddt, *dz, *dB, *dC;
    float *dstate_in, *dbc_part;
    float *param_part;     // [B nseg][dA | dD | ddt_bias]: rows of param_ld floats, the latter two at dD_at, dbias_at
    long long param_ld, dD_at, dbias_at;
    const int32_t *cu;
    unsigned *err;
    long long x_ld, dt_ld, z_ld, b_ld, c_ld;
    int B, T, D, N, G, Dg, nseq;
    int gblocks;           // channel blocks a group
    int gpad, DP;          // padded channels a group, and of all groups
    int nseg, seglen;
    bool softplus, vec, vec_bc, st_vec;
    // vec, vec_bc: the token tensors, B and C, take the 16-byte accesses; otherwise their rows are copied as pieces
};

struct F2x2 {
    f2 lo, hi;
};
__device__ __forceinline__ F2x2 lds_f2x2(const float *p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    return F2x2{v.x, v.y};
}

// Four 16-bit elements (a thread's states of B or C), each as the pair (v, v).
template <typename T>
__device__ __forceinline__ void lds_dup4(const uint16_t *p, f2 *o) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    float v[4];
    unpack2(widen2<T>(u.x), v[0], v[1]);
    unpack2(widen2<T>(u.y), v[2], v[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack2(v[i], v[i]);
}

// ---------------------------------------------------------------- pairs of scalars

// log(1 + e^x) = max(x, 0) + log1p(t), t = e^-|x| in (0, 1], with log1p(t) = t P(t).  P is the polynomial of degree 8
// that minimises the largest relative error on [0, 1] (3.0e-8; found by the exchange algorithm of Remez), so small
// steps keep their relative precision, which a logarithm of 1 + t would lose.
__device__ __forceinline__ f2 softplus2(f2 x) {
    float a, b;
    unpack2(x, a, b);
    const f2 t = ex2x2(mul2(pack2(-fabsf(a), -fabsf(b)), both(LOG2E)));
    f2 p = both(0.0052326941f);
    p = fma2(p, t, both(-0.0295052398f));
    p = fma2(p, t, both(0.0782259554f));
    p = fma2(p, t, both(-0.1366324574f));
    p = fma2(p, t, both(0.1910600662f));
    p = fma2(p, t, both(-0.2484298199f));
    p = fma2(p, t, both(0.3331909776f));
    p = fma2(p, t, both(-0.4999949336f));
    p = fma2(p, t, both(0.9999999404f));
    return fma2(p, t, pack2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
__device__ __forceinline__ float softplus(float x) {
    float a, b;
    unpack2(softplus2(pack2(x, x)), a, b);
    return a;
}

// ---------------------------------------------------------------- geometry

// Block -> channels.  Blocks never cross a group, whose B and C they stage.
template <int CB>
struct Chans {
    int g, first, count, pad;  // group; first channel; channels of this block; first padded channel
    __device__ __forceinline__ Chans(const ScanArgs &a, int block) {
        g = block / a.gblocks;
        const int in = (block - g * a.gblocks) * CB;
        first = g * a.Dg + in;
        count = min(CB, a.Dg - in);
        pad = g * a.gpad + in;
    }
};

// ---------------------------------------------------------------- tiles

// Eight 16-bit elements as four fp32 pairs, and back.
template <typename T>
__device__ __forceinline__ void widen8(uint4 u, f2 *o) {
    o[0] = widen2<T>(u.x), o[1] = widen2<T>(u.y), o[2] = widen2<T>(u.z), o[3] = widen2<T>(u.w);
}
template <typename T>
__device__ __forceinline__ uint4 narrow8(const f2 *v) {
    return make_uint4(narrow2<T>(v[0]), narrow2<T>(v[1]), narrow2<T>(v[2]), narrow2<T>(v[3]));
}
__device__ __forceinline__ void put8(float *p, const f2 *v) {
    reinterpret_cast<ulonglong2 *>(p)[0] = make_ulonglong2(v[0], v[1]);
    reinterpret_cast<ulonglong2 *>(p)[1] = make_ulonglong2(v[2], v[3]);
}
__device__ __forceinline__ void get8(const float *p, f2 *v) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0], b = reinterpret_cast<const ulonglong2 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// Asynchronous 16-byte copies, in groups (common.cuh's, as barriers for the compiler too: the copied places are read and
// written by plain accesses around them).
__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(LEFT) : "memory");
}

// Eight elements into shared memory: an asynchronous copy, or zeros where they do not exist.
__device__ __forceinline__ void copy8(uint16_t *to, const uint16_t *from, bool exist) {
    if (exist)
        copy16(to, from);
    else
        *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
}

// Rows of a tensor that allows no 16-byte accesses (odd widths or strides, views at any element).  Threads copy the
// aligned 16-byte pieces that hold `width` elements of each row, cut off at the tensor's ends, so that the copies are
// asynchronous all the same; element e of row j then lies at to[j rs + skew + e], rs >= width + 7.
struct Rows {
    const uint16_t *base;
    long long ld, first, rows;   // row stride; first element of interest in a row; rows of the tensor
    int cols;                    // elements of a row
    __device__ __forceinline__ const uint16_t *at(long long row) const { return base + row * ld + first; }
    __device__ __forceinline__ int skew(long long row) const { return (int)((reinterpret_cast<uintptr_t>(at(row)) & 15) >> 1); }
};
template <int NT, int PIECES>
__device__ __forceinline__ void copy_rows(uint16_t *to, int rs, const Rows &r, long long row, int rows, int width) {
    const char *lo = reinterpret_cast<const char *>(r.base);
    const char *hi = reinterpret_cast<const char *>(r.base + (r.rows - 1) * r.ld + r.cols);
    for (int i = threadIdx.x; i < rows * PIECES; i += NT) {
        const int j = i / PIECES, k = i % PIECES;
        const uintptr_t at = reinterpret_cast<uintptr_t>(r.at(row + j));
        const int skew = (int)(at & 15);
        if (k * 16 >= skew + 2 * width) continue;
        const char *src = reinterpret_cast<const char *>(at - skew) + k * 16;
        uint16_t *dst = to + j * rs + k * 8;
        if (src >= lo) {
            const long long left = hi - src;
            const int n = left < 16 ? (int)left : 16;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
        } else {  // the piece begins before the tensor
            for (int e = skew / 2; e < 8 && e - skew / 2 < width; ++e) dst[e] = reinterpret_cast<const uint16_t *>(src)[e];
        }
    }
}

// Packed batches: the sequence that token t starts (first) and the one that it ends (last), -1 for neither.
__device__ __forceinline__ void edges(const ScanArgs &a, int t, int t_end, int &first, int &last) {
    first = last = -1;
    if (t >= t_end) return;
    int lo = 0, hi = a.nseq - 1;  // the first n with cu[n + 1] > t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    if (a.cu[lo] == t) first = lo;
    if (a.cu[lo + 1] == t + 1) last = lo;
}

// For every token of a tile at once (the first lanes of a block's first warp): first[], last[], and whether any is set.
template <int TOKENS>
__device__ __forceinline__ void tile_edges(const ScanArgs &a, int base, int t_end, int *first, int *last, int *any) {
    if (threadIdx.x >= TOKENS) return;
    edges(a, base + threadIdx.x, t_end, first[threadIdx.x], last[threadIdx.x]);
    const int some = __any_sync(0xffffffffu >> (32 - TOKENS), first[threadIdx.x] >= 0 || last[threadIdx.x] >= 0);
    if (threadIdx.x == 0) *any = some;
}

// A compile-time flag to pass to a generic lambda: tiles that no sequence starts or ends in run without the tests.
template <bool V>
struct Flag {
    static constexpr bool value = V;
};

// ---------------------------------------------------------------- a thread's 4 channels x 4 states

// h[n][p]: state n of channels (2p, 2p + 1).
typedef f2 State[4][2];

__device__ __forceinline__ void zero(State h) {
#pragma unroll
    for (int n = 0; n < 4; ++n) h[n][0] = h[n][1] = 0ull;
}
// A as the exponent of 2 that a unit step takes.  Held finite: A = -inf, or one whose product overflows, forgets at every
// step, but a step of zero (a tile's places past the last token are such) changes nothing.
__device__ __forceinline__ float rate2(float A) {
    const float v = A * LOG2E;
    return v < -3.4e38f ? -3.4e38f : v;  // (a NaN stays)
}

// From or to a [.., D, N] fp32 array at channel `ch` (of `nc` that exist from there) and state `n0`.
__device__ __forceinline__ void load_rows(const ScanArgs &a, const float *p, int nc, int n0, State h) {
    float v[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float *q = p + (long long)c * a.N + n0;
        if (c < nc && a.st_vec && n0 < a.N) {
            const float4 f = *reinterpret_cast<const float4 *>(q);
            v[c][0] = f.x, v[c][1] = f.y, v[c][2] = f.z, v[c][3] = f.w;
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n) v[c][n] = (c < nc && n0 + n < a.N) ? q[n] : 0.f;
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        h[n][0] = pack2(v[0][n], v[1][n]);
        h[n][1] = pack2(v[2][n], v[3][n]);
    }
}
__device__ __forceinline__ void load_rates(const ScanArgs &a, int c, int nc, int n0, State r) {  // of the channels from c
    load_rows(a, a.A + (long long)c * a.N, nc, n0, r);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float lo, hi;
            unpack2(r[n][p], lo, hi);
            r[n][p] = pack2(rate2(lo), rate2(hi));
        }
}
__device__ __forceinline__ void store_rows(const ScanArgs &a, float *p, int nc, int n0, const State h) {
    float v[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        unpack2(h[n][0], v[0][n], v[1][n]);
        unpack2(h[n][1], v[2][n], v[3][n]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c >= nc) continue;
        float *q = p + (long long)c * a.N + n0;
        if (a.st_vec && n0 < a.N) {
            *reinterpret_cast<float4 *>(q) = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n0 + n < a.N) q[n] = v[c][n];
        }
    }
}
// From or to a padded workspace array [.., NP, DP]: p at (state n0, this thread's first padded channel).
__device__ __forceinline__ void load_padded(const float *p, long long DP, State h) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const F2x2 v = lds_f2x2(p + n * DP);
        h[n][0] = v.lo, h[n][1] = v.hi;
    }
}
__device__ __forceinline__ void store_padded(float *p, long long DP, const State h) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        ulonglong2 v;
        v.x = h[n][0], v.y = h[n][1];
        *reinterpret_cast<ulonglong2 *>(p + n * DP) = v;
    }
}

// Sums the four channels' values over the L lanes that share them.  Each of the first two steps halves the channels
// a lane keeps; the lane ends with R = max(1, 4 / L) channels from `at` (the lanes whose remaining index bits are
// not zero end with copies).
template <int L>
struct LaneSum {
    static constexpr int R = L >= 4 ? 1 : 4 / L;
    static __device__ __forceinline__ int at(int nl) {
        if constexpr (L == 1) return 0;
        else if constexpr (L == 2) return 2 * nl;
        else return nl / (L / 4);
    }
    static __device__ __forceinline__ bool keeper(int nl) {
        if constexpr (L <= 4) return true;
        else return nl % (L / 4) == 0;
    }
    static __device__ __forceinline__ void run(f2 lo, f2 hi, int nl, float *out) {
        if constexpr (L == 1) {
            unpack2(lo, out[0], out[1]);
            unpack2(hi, out[2], out[3]);
        } else {
            const bool up = (nl & (L / 2)) != 0;
            const f2 keep = up ? hi : lo, send = up ? lo : hi;
            const f2 s = add2(keep, __shfl_xor_sync(0xffffffffu, send, L / 2));
            if constexpr (L == 2) {
                unpack2(s, out[0], out[1]);
            } else {
                float a, b;
                unpack2(s, a, b);
                const bool odd = (nl & (L / 4)) != 0;
                float v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, L / 4);
#pragma unroll
                for (int o = L / 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                out[0] = v;
            }
        }
    }
};

}  // namespace scan
}  // namespace gdr
