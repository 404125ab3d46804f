// The norm of a mixer's output with its gate, and the norms behind and before a block fused with its gate and residual
// scale:
//
//   gated:  y = x r w act(g),  r = 1 / sqrt(mean x^2 + eps)
//     dn = dy w act(g);  dx = r dn - x r^3 mean(dn x);  dg = dy x r w act'(g);  dw = sum over rows of dy x r act(g)
//   block:  n = x r1 (or x);  b = n pw;  h = res + s b act(g);  y = h r2 w
//     dh = r2 w dy - h r2^3 mean(w dy h) + dres;  db = s dh act(g);  dg = s dh b act'(g);  dn = db pw
//     dx = r1 dn - x r1^3 mean(dn x);  dpw = sum of db n;  dw = sum of dy h r2
//   at the stored h; act is the number itself, its sigmoid or g sigmoid(g), or 1 without a gate.
//
// Every element is read and written once, so all four are bound by HBM.  A block walks rows; a row is spread over TPR
// threads of 8 NG elements each, and the next row's elements come into shared memory by asynchronous copies while this
// one is worked on (all passes over a row read it there).  All sums are fp32; sums over rows leave one partial row a
// block, which a second kernel adds in a fixed order.
//
// A thread owns vectors of 8 columns, aligned to 16 bytes, and copies what it reads itself (fp32: its warp does).  Where
// rows do not begin on such a boundary (SHIFT: a width that is no multiple of 8, contiguous tensors) the vectors are those of
// the tensor, not of the row: row r's first element lies r D mod 8 elements into its first vector.  A block walks rows of one
// remainder only, so that its threads keep their columns, their weights and their sums; the vectors at a row's ends are
// masked.  (5311 x 4099, gated norm's backward: 167 us with a column of 2 bytes at a time, 90 so.)
#pragma once

#include "norm.cuh"
#include "rowclip.h"
#include "rownorm.h"

namespace gdr {
namespace rownorm {
namespace {

using namespace norm;

// Access to the rows of the tensors in MASK (bits of IN_*; the gradient from later layers, last, may be missing at run
// time).  Elements come in groups of 8: group g of thread t holds columns 8 (g TPR + t) - shift and on.  Everything about
// places that can be known when compiling is: worked out at run time it took more instructions than the arithmetic (block
// norm's backward, 8192 x 4096: 188 us then, 120 so).
template <typename T, int NG, int BT, bool SHIFT, bool F32, unsigned MASK>
struct Rows {
    static constexpr int elem(int i) { return (i == IN_H || i == IN_DRES) && F32 ? 4 : 2; }
    static constexpr bool has(int i) { return MASK >> i & 1; }
    const RowArgs &a;
    char *smem;
    int t, slot, shift;     // thread of the row, row slot of the block, elements before a row in its first vector
    bool edge;              // some but not all of a vector's columns lie in the row
    uint32_t own;           // the columns of this thread that lie in the row, a bit each (whole vectors: a bit a group)
    __device__ __forceinline__ Rows(const RowArgs &a_, void *s) : a(a_), smem(static_cast<char *>(s)) {
        slot = threadIdx.x / a.tpr;
        t = threadIdx.x - slot * a.tpr;
        shift = SHIFT ? (int)((blockIdx.x % (unsigned)a.period) * (unsigned)a.D & 7u) : 0;
        own = 0;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (!SHIFT) own |= (uint32_t)(column(g) < a.D) << g;
#pragma unroll
            for (int e = 0; SHIFT && e < 8; ++e) own |= (uint32_t)(column(g) + e >= 0 && column(g) + e < a.D) << (8 * g + e);
        }
        edge = false;
#pragma unroll
        for (int g = 0; SHIFT && g < NG; ++g) edge = edge || (any(g) && !whole(g));
    }
    __device__ __forceinline__ int column(int g) const { return (g * a.tpr + t) * 8 - (SHIFT ? shift : 0); }
    __device__ __forceinline__ bool any(int g) const { return SHIFT ? own >> (8 * g) & 0xffu : own >> g & 1; }
    __device__ __forceinline__ bool whole(int g) const { return !SHIFT || (own >> (8 * g) & 0xffu) == 0xffu; }
    __device__ __forceinline__ bool has_column(int g, int e) const { return SHIFT ? own >> (8 * g + e) & 1 : own >> g & 1; }
    // the block's rows: of one remainder modulo the period
    __device__ __forceinline__ long long first() const {
        if (!SHIFT) return (long long)blockIdx.x * a.rpb + slot;
        return (long long)(blockIdx.x / (unsigned)a.period * (unsigned)a.rpb + slot) * a.period + blockIdx.x % (unsigned)a.period;
    }
    __device__ __forceinline__ int apart() const { return SHIFT ? a.period : 1; }
    __device__ __forceinline__ long long step() const { return (long long)gridDim.x * a.rpb; }
    // where an input's rows begin in a stage: NG groups of all threads
    static constexpr int bytes_before(int i) {  // of a thread
        int o = 0;
        for (int k = 0; k < i; ++k)
            if (has(k)) o += NG * 8 * elem(k);
        return o;
    }
    __device__ __forceinline__ int threads() const { return (int)blockDim.x; }
    __device__ __forceinline__ int off(int i) const { return bytes_before(i) * threads(); }
    __device__ __forceinline__ const char *at(int i, long long row) const {
        const RowIn &in = a.in[i];
        long long e = row * in.ld - shift;
        if (in.heads > 1) {
            const long long token = a.rows <= 0x7fffffff ? (long long)((unsigned)row / (unsigned)in.heads) : row / in.heads;
            e = token * in.ld + (row - token * in.heads) * a.D;
        }
        return static_cast<const char *>(in.p) + e * elem(i);
    }
    template <int I>
    __device__ __forceinline__ void fetch_one(long long row, int stage) const {
        if constexpr (has(I)) {
            if (I == IN_DRES && !a.in[I].p) return;
            constexpr bool W = elem(I) == 4;
            const bool in = row < a.rows;
            // fp32: two instructions a group, each over a whole run of the warp's (or, with fewer, the row's) lanes
            const int lanes = min(a.tpr, 32), l = t & (lanes - 1);
            const char *src = at(I, row) + (W ? (t - l) * 32 + l * 16 : t * 16);
            const uint32_t to = smem_u32(smem) + stage * a.place + off(I) + (W ? (threadIdx.x - l) * 32 + l * 16 : threadIdx.x * 16);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int h = 0; h < (W ? 2 : 1); ++h) {
                    const char *from = src + g * a.tpr * 8 * elem(I) + (W ? h * lanes * 16 : 0);
                    const uint32_t d = to + g * threads() * 8 * elem(I) + (W ? h * lanes * 16 : 0);
                    // (no bytes, zeros: for what lies behind the row's end or the last row; nothing behind the tensor's end)
                    const int c = (g * a.tpr + t - l) * 8 + h * lanes * 4 + l * 4 - shift;
                    int n = in && (W ? c < a.D && c + 4 > 0 : any(g)) ? 16 : 0;
                    if (SHIFT && n) n = bytes_to_copy(row, a.rows, static_cast<const char *>(a.in[I].p) + a.rows * a.D * elem(I) - from);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d), "l"(from), "r"(n) : "memory");
                }
            }
        }
    }
    __device__ __forceinline__ void fetch(long long row, int stage) const {
        fetch_one<0>(row, stage);
        fetch_one<1>(row, stage);
        fetch_one<2>(row, stage);
        fetch_one<3>(row, stage);
        fetch_one<4>(row, stage);
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    template <int I>
    __device__ __forceinline__ void get(int stage, long long, int g, f2 *o) const {
        constexpr bool W = elem(I) == 4;
        const char *s = smem + stage * a.place + off(I) + (g * threads() + threadIdx.x) * (W ? 32 : 16);
        const uint4 u = *reinterpret_cast<const uint4 *>(s);
        if constexpr (W) {
            const uint4 x = *reinterpret_cast<const uint4 *>(s + 16);
            o[0] = pack2(__uint_as_float(u.x), __uint_as_float(u.y)), o[1] = pack2(__uint_as_float(u.z), __uint_as_float(u.w));
            o[2] = pack2(__uint_as_float(x.x), __uint_as_float(x.y)), o[3] = pack2(__uint_as_float(x.z), __uint_as_float(x.w));
        } else {
            o[0] = widen2<T>(u.x), o[1] = widen2<T>(u.y), o[2] = widen2<T>(u.z), o[3] = widen2<T>(u.w);
        }
    }
    // Zeros in place of the neighbouring rows' elements in the vectors at a row's ends, once they are there.  (Left out of
    // what `get` gives instead, every vector of every pass paid for it: 100000 x 127, block norm's backward 156 us, 136 so.)
    template <int I>
    __device__ __forceinline__ void clear_one(int stage, int g) const {
        if constexpr (has(I)) {
            if (I == IN_DRES && !a.in[I].p) return;
            constexpr int W = elem(I) / 2;
            uint4 *s = reinterpret_cast<uint4 *>(smem + stage * a.place + off(I) + (g * threads() + threadIdx.x) * (16 * W));
            const uint32_t b = own >> (8 * g);
#pragma unroll
            for (int h = 0; h < W; ++h) {
                uint4 u = s[h];
                uint32_t *w = &u.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (W == 2) w[e] = b >> (4 * h + e) & 1 ? w[e] : 0u;
                    else w[e] &= (b >> (2 * e) & 1 ? 0xffffu : 0u) | (b >> (2 * e + 1) & 1 ? 0xffff0000u : 0u);
                }
                s[h] = u;
            }
        }
    }
    __device__ __forceinline__ void clear(int stage) const {
        if (!SHIFT || !edge) return;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (!any(g) || whole(g)) continue;
            clear_one<0>(stage, g);
            clear_one<1>(stage, g);
            clear_one<2>(stage, g);
            clear_one<3>(stage, g);
            clear_one<4>(stage, g);
        }
    }
    // a group of an output [rows, D]
    template <bool W>
    __device__ __forceinline__ void put(void *to, long long row, int g, const f2 *v) const {
        if (row >= a.rows || !any(g)) return;
        const long long i = row * a.D + column(g);
        if (!whole(g)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[2];
                unpack2(v[e], x[0], x[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (has_column(g, 2 * e + k)) {
                        if (W) static_cast<float *>(to)[i + 2 * e + k] = x[k];
                        else static_cast<T *>(to)[i + 2 * e + k] = Elt<T>::from_f(x[k]);
                    }
            }
        } else if constexpr (W) {
            float *q = static_cast<float *>(to) + i;
            if (a.wide) {  // a whole sector a lane
                asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};\n" ::"l"(q), "l"(v[0]), "l"(v[1]), "l"(v[2]), "l"(v[3]) : "memory");
            } else {
                reinterpret_cast<ulonglong2 *>(q)[0] = make_ulonglong2(v[0], v[1]);
                reinterpret_cast<ulonglong2 *>(q)[1] = make_ulonglong2(v[2], v[3]);
            }
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(to) + i) = make_uint4(narrow2<T>(v[0]), narrow2<T>(v[1]), narrow2<T>(v[2]), narrow2<T>(v[3]));
        }
    }
    // a group of a weight
    __device__ __forceinline__ void weight(const void *w, int g, f2 *o) const {
        const int c = column(g);
        if (SHIFT) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = has_column(g, e) ? load_gate<T>(w, c + e, a.w_f32) : 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack2(x[2 * e], x[2 * e + 1]);
        } else if (!any(g)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = 0ull;
        } else if (a.w_f32) {
            const ulonglong2 *q = reinterpret_cast<const ulonglong2 *>(static_cast<const float *>(w) + c);
            const ulonglong2 u = q[0], v = q[1];
            o[0] = u.x, o[1] = u.y, o[2] = v.x, o[3] = v.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(w) + c);
            o[0] = widen2<T>(u.x), o[1] = widen2<T>(u.y), o[2] = widen2<T>(u.z), o[3] = widen2<T>(u.w);
        }
    }
    // this thread's sums over its rows, added up over the block's row slots, as `which` of the block's partial rows
    __device__ __forceinline__ void put_sums(const f2 *v, int which, int count) const {
        float *out = a.part + ((long long)blockIdx.x * count + which) * a.D;
        float *slots = reinterpret_cast<float *>(smem);
        __syncthreads();  // (the rows, or the sums before these, are read no more)
        float *to = a.rpb == 1 ? out : slots + slot * a.D;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[2];
                unpack2(v[4 * g + e], x[0], x[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (has_column(g, 2 * e + k)) to[column(g) + 2 * e + k] = x[k];
            }
        }
        if (a.rpb == 1) return;
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
            float s = 0.f;
            for (int i = 0; i < a.rpb; ++i) s += slots[i * a.D + c];
            out[c] = s;
        }
    }
};

// Sums over a row's threads of N numbers each.  `red`: [2][16][N] floats that only this sum uses, by parity of the row.
template <int N>
__device__ __forceinline__ void row_sums(float *v, float *red, int parity, int tpr, int slot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum(v[i], min(tpr, 32));
    if (tpr <= 32) return;
    float *r = red + parity * 16 * N;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) r[warp * N + i] = v[i];
    __syncthreads();
    const int wpr = tpr >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int k = 0; k < wpr; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += r[(slot * wpr + k) * N + i];
}

// The gate's factors of four pairs and, where asked for, their derivatives.  sigmoid(g) = 1 / (1 + e), e = exp(-g), and
// 1 - sigmoid(g) = e sigmoid(g): neither cancels.  g is taken at -80 at least, where e is finite and the factor 1e-35.
template <bool GRAD>
__device__ __forceinline__ void gate_of_pairs(int act, const f2 *g, f2 *f, f2 *df) {
    if (act == ACT_RAW) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = g[e];
            if (GRAD) df[e] = both(1.f);
        }
        return;
    }
    const bool silu = act == ACT_SILU;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float x[2];
        unpack2(g[e], x[0], x[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) asm("max.NaN.f32 %0, %1, %2;" : "=f"(x[k]) : "f"(x[k]), "f"(-80.f));
        const f2 y = pack2(x[0], x[1]), z = ex2x2(mul2(y, both(-LOG2E))), sg = rcpx2(add2(z, both(1.f)));
        f[e] = silu ? mul2(y, sg) : sg;
        if (GRAD) {
            const f2 c = mul2(z, sg);
            df[e] = silu ? fma2(f[e], c, sg) : mul2(sg, c);
        }
    }
}

// Loops over the block's rows: body(row, stage, parity) with the row's elements at hand.  (All threads of a block make the
// same number of rounds: its last slots' rows may lie past the end.)
template <typename R, typename F>
__device__ __forceinline__ void walk(const R &rows, const RowArgs &a, F &&body) {
    const bool two = a.stages == 2;
    long long row = rows.first();
    const long long step = rows.step();
    long long lead = row - (long long)rows.slot * rows.apart();  // the first slot's row
    if (two) rows.fetch(row, 0);
    int parity = 0;
    for (; lead < a.rows; lead += step, row += step, parity ^= 1) {
        const int stage = two ? parity : 0;
        __syncwarp();  // (the place that is filled now has been read)
        rows.fetch(two ? row + step : row, two ? stage ^ 1 : 0);
        if (two) asm volatile("cp.async.wait_group 1;\n" ::: "memory");
        else asm volatile("cp.async.wait_group 0;\n" ::: "memory");
        __syncwarp();  // (what this warp's lanes copied for one another)
        rows.clear(stage);
        body(row, stage, parity);
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}

// ---------------------------------------------------------------- gated norm

// 8192 x 32 x 128 bf16: 34.5 us for 201 MB, 5.8 TB/s; 8192 x 4104: 58 us, 8192 x 8192: 72 for 403 MB, with one block an SM;
// 5311 x 4099 fp16: 43 us for 131 MB, 3.0 TB/s, bound by issue (an odd width has 2 more vectors than 256 threads, and a second
// block of 288 leaves 96 registers).
template <typename T, int NG, int BT, bool SHIFT>
__global__ void __launch_bounds__(BT, BT > 320 ? 1 : BT > 256 ? 2 : 3) gated_fwd_kernel(const __grid_constant__ RowArgs a) {
    extern __shared__ __align__(16) char s_rows[];
    __shared__ float red[2 * 16];
    const Rows<T, NG, BT, SHIFT, false, 1u << IN_X | 1u << IN_GATE> rows(a, s_rows);
    f2 w[4 * NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) rows.weight(a.w, g, w + 4 * g);
    const float inv_d = 1.0f / (float)a.D;
    walk(rows, a, [&](long long row, int stage, int parity) {
        f2 x[4 * NG], ss = 0ull;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            rows.template get<IN_X>(stage, row, g, x + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = fma2(x[4 * g + e], x[4 * g + e], ss);
        }
        float s[1] = {sum2(ss)};
        row_sums<1>(s, red, parity, a.tpr, rows.slot);
        const f2 r = both(rsqrtf(fmaf(s[0], inv_d, a.eps)));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f2 z[4], f[4];
            rows.template get<IN_GATE>(stage, row, g, z);
            gate_of_pairs<false>(a.act, z, f, nullptr);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = mul2(mul2(mul2(x[4 * g + e], r), w[4 * g + e]), f[e]);
            rows.template put<false>(a.y, row, g, f);
        }
    });
}

// 8192 x 32 x 128 bf16: 59.5 us for 336 MB, 5.6 TB/s, and 8 us of reduction; 8192 x 8192: 137 for 671 MB with it; 5311 x 4099
// fp16: 90 us for 218 MB, with 120 bytes a thread spilled at 96 registers.  (A row more ahead: 62 and 107 us; what is on its
// way is not what is short.)  The forms of four vectors spill 196 to 408 bytes: 8192 x 16384 takes 317 us, floor 201.
template <typename T, int NG, int BT, bool SHIFT>
__global__ void __launch_bounds__(BT, BT > 320 ? 1 : 2) gated_bwd_kernel(const __grid_constant__ RowArgs a) {
    extern __shared__ __align__(16) char s_rows[];
    __shared__ float red[2 * 16 * 2];
    const Rows<T, NG, BT, SHIFT, false, 1u << IN_X | 1u << IN_GATE | 1u << IN_DY> rows(a, s_rows);
    f2 w[4 * NG], dw[4 * NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) rows.weight(a.w, g, w + 4 * g);
#pragma unroll
    for (int i = 0; i < 4 * NG; ++i) dw[i] = 0ull;
    const float inv_d = 1.0f / (float)a.D;
    walk(rows, a, [&](long long row, int stage, int parity) {
        f2 dn[4 * NG], ss = 0ull, sd = 0ull;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f2 x[4], z[4], f[4], d[4];
            rows.template get<IN_X>(stage, row, g, x);
            rows.template get<IN_GATE>(stage, row, g, z);
            rows.template get<IN_DY>(stage, row, g, d);
            gate_of_pairs<false>(a.act, z, f, nullptr);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dn[4 * g + e] = mul2(mul2(d[e], w[4 * g + e]), f[e]);
                ss = fma2(x[e], x[e], ss);
                sd = fma2(dn[4 * g + e], x[e], sd);
            }
        }
        float s[2] = {sum2(ss), sum2(sd)};
        row_sums<2>(s, red, parity, a.tpr, rows.slot);
        // (a place past the last row: with eps = 0 its factor would be infinite)
        const float r = row < a.rows ? rsqrtf(fmaf(s[0], inv_d, a.eps)) : 0.f;
        const f2 r2 = both(r), k2 = both(-(r * (s[1] * inv_d)) * r * r), one = both(a.D == 1 ? a.eps * r * r * r : r);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f2 x[4], z[4], f[4], df[4], d[4], dx[4], dg[4];
            rows.template get<IN_X>(stage, row, g, x);
            rows.template get<IN_GATE>(stage, row, g, z);
            rows.template get<IN_DY>(stage, row, g, d);
            gate_of_pairs<true>(a.act, z, f, df);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 n = mul2(mul2(x[e], r2), d[e]);  // dy x r
                dw[4 * g + e] = fma2(n, f[e], dw[4 * g + e]);
                dg[e] = mul2(mul2(n, w[4 * g + e]), df[e]);
                const f2 own = mul2(dn[4 * g + e], one);
                dx[e] = a.D == 1 ? own : fma2(x[e], k2, own);
            }
            rows.template put<false>(a.dx, row, g, dx);
            rows.template put<false>(a.dgate, row, g, dg);
        }
    });
    rows.put_sums(dw, 0, 1);
}

// ---------------------------------------------------------------- block norm

// 8192 x 4096 bf16 with a gate: 66 us from a bf16 stream (335 MB, 5.1 TB/s), 79 from an fp32 one (470 MB, 5.9 TB/s; 100 with
// 16 bytes a lane at a stride of 32, which asks for every sector twice).  8192 x 8192: 135 us for 671 MB; 8192 x 4099: 105.
template <typename T, int NG, int BT, bool SHIFT, bool F32, bool GATE>
__global__ void __launch_bounds__(BT, BT > 320 ? 1 : BT > 256 || SHIFT ? 2 : 3) block_fwd_kernel(const __grid_constant__ RowArgs a) {
    // Weights come from the L1 cache row by row: held in registers they cost the third block an SM (8192 x 4096 bf16: 71 us with,
    // 64 without).  Shifted rows would read them element by element, and hold them.
    constexpr bool HOLD = SHIFT && NG <= 2;
    extern __shared__ __align__(16) char s_rows[];
    __shared__ float red1[2 * 16], red2[2 * 16];
    const Rows<T, NG, BT, SHIFT, F32, 1u << IN_X | (GATE ? 1u << IN_GATE : 0u) | 1u << IN_RES> rows(a, s_rows);
    f2 w[HOLD ? 4 * NG : 4], pw[HOLD ? 4 * NG : 4];
    if (HOLD) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            rows.weight(a.w, g, w + 4 * g);
            if (a.pw) rows.weight(a.pw, g, pw + 4 * g);
        }
    }
    const float inv_d = 1.0f / (float)a.D;
    walk(rows, a, [&](long long row, int stage, int parity) {
        f2 h[4 * NG];
        f2 scale = both(a.rscale);
#pragma unroll
        for (int g = 0; g < NG; ++g) rows.template get<IN_X>(stage, row, g, h + 4 * g);
        if (a.pw) {
            f2 ss = 0ull;
#pragma unroll
            for (int i = 0; i < 4 * NG; ++i) ss = fma2(h[i], h[i], ss);
            float s[1] = {sum2(ss)};
            row_sums<1>(s, red1, parity, a.tpr, rows.slot);
            const f2 r = both(rsqrtf(fmaf(s[0], inv_d, a.eps)));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (!HOLD) rows.weight(a.pw, g, pw);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[4 * g + e] = mul2(mul2(h[4 * g + e], r), pw[HOLD ? 4 * g + e : e]);
            }
        }
        f2 ss = 0ull;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f2 z[4], f[4], res[4];
            rows.template get<IN_RES>(stage, row, g, res);
            if constexpr (GATE) {
                rows.template get<IN_GATE>(stage, row, g, z);
                gate_of_pairs<false>(a.act, z, f, nullptr);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[4 * g + e] = mul2(h[4 * g + e], f[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[4 * g + e] = fma2(h[4 * g + e], scale, res[e]);
                ss = fma2(h[4 * g + e], h[4 * g + e], ss);
            }
            rows.template put<F32>(a.res_out, row, g, h + 4 * g);
        }
        float s[1] = {sum2(ss)};
        row_sums<1>(s, red2, parity, a.tpr, rows.slot);
        const f2 r = both(rsqrtf(fmaf(s[0], inv_d, a.eps)));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (!HOLD) rows.weight(a.w, g, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[4 * g + e] = mul2(mul2(h[4 * g + e], r), w[HOLD ? 4 * g + e : e]);
            rows.template put<false>(a.y, row, g, h + 4 * g);
        }
    });
}

// 8192 x 4096 bf16 with a gate: 123 us for 537 MB, 4.4 TB/s, bound by issue: some 600 instructions a warp and row, a third of
// them the sigmoid and its derivative.  (One group a thread in blocks of 512: 181 us.)  8192 x 8192: 249 us for 1.07 GB; of odd
// widths the form of 320 threads spills 436 to 536 bytes a thread at 96 registers: 8192 x 4099 takes 265 us, floor 80.
template <typename T, int NG, int BT, bool SHIFT, bool F32, bool GATE>
__global__ void __launch_bounds__(BT, BT > 320 ? 1 : 2) block_bwd_kernel(const __grid_constant__ RowArgs a) {
    constexpr bool HOLD = NG <= 2;
    extern __shared__ __align__(16) char s_rows[];
    __shared__ float red1[2 * 16 * 3], red2[2 * 16];
    const Rows<T, NG, BT, SHIFT, F32, 1u << IN_X | (GATE ? 1u << IN_GATE : 0u) | 1u << IN_DY | 1u << IN_H | 1u << IN_DRES> rows(a, s_rows);
    f2 w[HOLD ? 4 * NG : 4], pw[HOLD ? 4 * NG : 4], dw[4 * NG], dpw[4 * NG];
    if (HOLD) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            rows.weight(a.w, g, w + 4 * g);
            if (a.pw) rows.weight(a.pw, g, pw + 4 * g);
        }
    }
#pragma unroll
    for (int i = 0; i < 4 * NG; ++i) dw[i] = dpw[i] = 0ull;
    const float inv_d = 1.0f / (float)a.D;
    walk(rows, a, [&](long long row, int stage, int parity) {
        f2 sx = 0ull, sh = 0ull, sd = 0ull;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f2 x[4], h[4], d[4];
            rows.template get<IN_X>(stage, row, g, x);
            rows.template get<IN_H>(stage, row, g, h);
            rows.template get<IN_DY>(stage, row, g, d);
            if (!HOLD) rows.weight(a.w, g, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sx = fma2(x[e], x[e], sx);
                sh = fma2(h[e], h[e], sh);
                sd = fma2(mul2(d[e], w[HOLD ? 4 * g + e : e]), h[e], sd);
            }
        }
        float s[3] = {sum2(sx), sum2(sh), sum2(sd)};
        row_sums<3>(s, red1, parity, a.tpr, rows.slot);
        const bool live = row < a.rows;
        const float r1 = !a.pw ? 1.f : live ? rsqrtf(fmaf(s[0], inv_d, a.eps)) : 0.f;
        const float r2 = live ? rsqrtf(fmaf(s[1], inv_d, a.eps)) : 0.f;
        const f2 k2 = both(-(r2 * (s[2] * inv_d)) * r2 * r2), one = both(a.D == 1 ? a.eps * r2 * r2 * r2 : r2);
        f2 dn[4 * NG], sn = 0ull;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f2 x[4], h[4], d[4], dh[4], f[4], df[4];
            rows.template get<IN_X>(stage, row, g, x);
            rows.template get<IN_H>(stage, row, g, h);
            rows.template get<IN_DY>(stage, row, g, d);
            if (a.in[IN_DRES].p) rows.template get<IN_DRES>(stage, row, g, dh);
            else dh[0] = dh[1] = dh[2] = dh[3] = 0ull;
            if (!HOLD) {
                rows.weight(a.w, g, w);
                if (a.pw) rows.weight(a.pw, g, pw);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 wd = mul2(mul2(d[e], w[HOLD ? 4 * g + e : e]), one);
                dh[e] = add2(dh[e], a.D == 1 ? wd : fma2(h[e], k2, wd));
                dw[4 * g + e] = fma2(mul2(h[e], both(r2)), d[e], dw[4 * g + e]);
            }
            rows.template put<F32>(a.dres, row, g, dh);
            if constexpr (GATE) {
                f2 z[4];
                rows.template get<IN_GATE>(stage, row, g, z);
                gate_of_pairs<true>(a.act, z, f, df);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 p = a.pw ? pw[HOLD ? 4 * g + e : e] : both(1.f);
                const f2 db = mul2(dh[e], both(a.rscale)), n = mul2(x[e], both(r1));
                if (GATE) df[e] = mul2(mul2(db, mul2(n, p)), df[e]);
                const f2 dg = GATE ? mul2(db, f[e]) : db;
                dpw[4 * g + e] = fma2(dg, n, dpw[4 * g + e]);
                dn[4 * g + e] = mul2(dg, p);
                sn = fma2(dn[4 * g + e], x[e], sn);
            }
            if (GATE) rows.template put<false>(a.dgate, row, g, df);
        }
        f2 k1 = 0ull, one1 = both(1.f);
        if (a.pw) {
            float q[1] = {sum2(sn)};
            row_sums<1>(q, red2, parity, a.tpr, rows.slot);
            k1 = both(-(r1 * (q[0] * inv_d)) * r1 * r1);
            one1 = both(a.D == 1 ? a.eps * r1 * r1 * r1 : r1);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f2 x[4];
            rows.template get<IN_X>(stage, row, g, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 own = mul2(dn[4 * g + e], one1);
                dn[4 * g + e] = !a.pw || a.D == 1 ? own : fma2(x[e], k1, own);
            }
            rows.template put<false>(a.dx, row, g, dn + 4 * g);
        }
    });
    rows.put_sums(dw, 0, a.pw ? 2 : 1);
    if (a.pw) rows.put_sums(dpw, 1, 2);
}

// ---------------------------------------------------------------- launches

template <typename K>
cudaError_t launch_rows(K k, const RowArgs &a, const RowForm &f, cudaStream_t st) {
    const cudaError_t e = allow_smem(k, f.smem);
    if (e != cudaSuccess) return e;
    return launch_plain(k, dim3(f.blocks), dim3(f.s.threads), f.smem, st, a);
}
#define GDR_ROW_FORMS(KERNEL, ...)                                                                                      \
    do {                                                                                                                \
        if (f.shift) {                                                                                                  \
            if (f.s.nv == 4) return launch_rows(KERNEL<T, 4, 512, true __VA_ARGS__>, a, f, st);                         \
            return f.s.threads <= 256   ? launch_rows(KERNEL<T, 2, 256, true __VA_ARGS__>, a, f, st)                    \
                   : f.s.threads <= 320 ? launch_rows(KERNEL<T, 2, 320, true __VA_ARGS__>, a, f, st)                    \
                                        : launch_rows(KERNEL<T, 2, 512, true __VA_ARGS__>, a, f, st);                   \
        }                                                                                                               \
        if (f.s.nv == 4) return launch_rows(KERNEL<T, 4, 512, false __VA_ARGS__>, a, f, st);                            \
        return f.s.threads <= 256 ? launch_rows(KERNEL<T, 2, 256, false __VA_ARGS__>, a, f, st)                         \
                                  : launch_rows(KERNEL<T, 2, 512, false __VA_ARGS__>, a, f, st);                        \
    } while (0)

}  // namespace
}  // namespace rownorm
}  // namespace gdr
