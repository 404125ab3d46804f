// What the selective scan's kernels share: the problem, the lane layout, the staging of a token tile and the
// two-element fp32 arithmetic.
//
// Lane layout.  Every thread owns 4 channels x 4 states (in registers, fp32), L lanes side by side hold one channel's
// N <= 4 L states (padded with states whose B and C are zero), and the 32 / L lane groups of a warp take consecutive
// channels.  Pairs of channels go through the two-element instructions: a channel's step delta and input are then
// natural pairs, and B and C are staged twice (B_n, B_n) so that they are pairs too.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "host.h"
#include "launch.h"
#include "seqwalk.cuh"

namespace gdr {
namespace scan {

constexpr int SAVE = 16;       // tokens between saved states; segments are multiples of it
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

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
    float *dstate_in, *dA_part, *dD_part, *dbias_part, *dbc_part;
    const int32_t *cu;
    unsigned *err;
    long long x_ld, dt_ld, z_ld, b_ld, c_ld;
    int B, T, D, N, G, Dg, nseq;
    int gblocks;           // channel blocks a group
    int gpad, DP;          // padded channels a group, and of all groups
    int nseg, seglen;
    bool softplus, vec, vec_bc, st_vec;
};

// ---------------------------------------------------------------- two fp32 at a time

typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 exp2x2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return a + b;
}
struct F2x2 {
    f2 lo, hi;
};
__device__ __forceinline__ F2x2 lds_f2x2(const float *p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    return F2x2{v.x, v.y};
}

// ---------------------------------------------------------------- scalar functions

// log(1 + e^x) = max(x, 0) + log1p(t) with t = e^-|x|, and log1p(t) = 2 atanh(t / (2 + t)) by atanh's series in
// s = t / (2 + t) <= 1/3: the terms left out are below 2e-9 of the sum, so small steps keep their relative precision.
__device__ __forceinline__ float softplus(float x) {
    const float t = ex2(-fabsf(x) * LOG2E);
    const float s = __fdividef(t, 2.f + t), q = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * s, p, fmaxf(x, 0.f));
}
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + ex2(-x * LOG2E)); }

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

// Eight 16-bit elements from p; `n` of them exist.
__device__ __forceinline__ uint4 load8(const uint16_t *p, int n, bool vec) {
    if (vec && n >= 8) return *reinterpret_cast<const uint4 *>(p);
    uint32_t r[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) r[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store8(uint16_t *p, uint4 u, int n, bool vec) {
    if (vec && n >= 8) {
        *reinterpret_cast<uint4 *>(p) = u;
        return;
    }
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
}
template <typename T>
__device__ __forceinline__ void widen8(uint4 u, float *o) {
    const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Elt<T>::unpack(r[i]);
        o[2 * i] = f.x, o[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 narrow8(const float *v) {
    return make_uint4(Elt<T>::pack(v[0], v[1]), Elt<T>::pack(v[2], v[3]), Elt<T>::pack(v[4], v[5]), Elt<T>::pack(v[6], v[7]));
}
__device__ __forceinline__ void put8(float *p, const float *v) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void get8(const float *p, float *v) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
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

// ---------------------------------------------------------------- a thread's 4 channels x 4 states

// h[n][p]: state n of channels (2p, 2p + 1).
typedef f2 State[4][2];

__device__ __forceinline__ void zero(State h) {
#pragma unroll
    for (int n = 0; n < 4; ++n) h[n][0] = h[n][1] = 0ull;
}
// From or to a [.., D, N] fp32 array at channel `ch` (of `nc` that exist from there) and state `n0`.
__device__ __forceinline__ void load_rows(const ScanArgs &a, const float *p, int nc, int n0, State h, float mul = 1.f) {
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
        h[n][0] = pack2(v[0][n] * mul, v[1][n] * mul);
        h[n][1] = pack2(v[2][n] * mul, v[3][n] * mul);
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
