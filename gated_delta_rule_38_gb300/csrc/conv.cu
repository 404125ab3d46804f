// Short causal convolution of every channel with its own W taps (2 <= W <= 4), optionally through SiLU, over dense
// rows or packed sequences, from cached inputs, and its backward pass.
//
//   pre_t = b + sum_{j<W} w_{W-1-j} x_{t-j};   y_t = pre_t  or  pre_t sigmoid(pre_t)
//   backward: dpre_t = dy_t (sig + pre sig (1 - sig));  dx_s = sum_j w_{W-1-j} dpre_{s+j} (same sequence only);
//             dw_{W-1-j} = sum_t dpre_t x_{t-j};  db = sum_t dpre_t
// Inputs before a sequence's first token are its W - 1 cached ones (state [N, W-1, D]) or zeros; their gradients
// come out as if they were tokens of it.
//
// A thread walks TT tokens of 4 channels with the last W - 1 inputs (backward: also the W - 1 open sums of dx) in
// registers, so every element is read and written once but for W - 1 tokens of overlap between neighbouring walks:
// the kernels are bound by HBM.  A block is 32 lanes along the channels (one contiguous row segment a warp) by 8
// walks.  All sums are fp32.
#include <cuda_runtime.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "host.h"
#include "launch.h"
#include "seqwalk.cuh"

namespace gdr {
namespace {

constexpr int WALKS = 8;  // walks (warps) of a block
constexpr int NC = 4;     // channels a thread

struct ConvArgs {
    const void *x, *w, *bias, *state_in;
    void *y, *state_out;
    const void *dy, *dstate_out;   // backward: gradients of y and of the final states
    void *dx, *dstate_in;
    float *part;                   // backward: [blocks along the tokens][D * W | D]
    const int32_t *cu;
    unsigned *err;
    long long x_ld;
    int B, T, D, N;
    int tt, tiles, cblocks;        // tokens a walk; walks a row; blocks along the channels
    uint32_t tiles_m, cblocks_m;   // (divisors as multiply-high, see Geo::div_hq)
    int tiles_s, cblocks_s;
    bool w_f32, w_wide, silu;
};

// A thread's NC channels: NC consecutive ones from one access (WIDE), or, where rows are not aligned for that, every
// 32nd, so that the lanes of a warp still read and write contiguous elements.
template <bool WIDE>
struct Lane {
    int c;  // first channel
    int D;
    __device__ __forceinline__ int chan(int i) const { return WIDE ? c + i : c + 32 * i; }
    __device__ __forceinline__ bool has(int i) const { return WIDE || chan(i) < D; }
};

// The raw elements of one token: NC / 2 words of two channels each, or (narrow) one register an element, so that
// nothing waits for a load before its use.
template <bool WIDE>
struct Raw {
    uint32_t w[WIDE ? NC / 2 : NC];
    __device__ __forceinline__ void load(const uint16_t *p, const Lane<WIDE> &l) {  // p: the token's row
        if constexpr (WIDE) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p + l.c);
            w[0] = u.x, w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i) w[i] = l.has(i) ? p[l.chan(i)] : 0;
        }
    }
    template <typename T>
    __device__ __forceinline__ void widen(f2 *o) const {
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) o[i] = widen2<T>(WIDE ? w[i] : w[2 * i % (WIDE ? NC / 2 : NC)] | w[(2 * i + 1) % (WIDE ? NC / 2 : NC)] << 16);
    }
};
template <typename T, bool WIDE>
__device__ __forceinline__ void load_x(const void *p, long long row, const Lane<WIDE> &l, f2 *o) {  // contiguous rows
    Raw<WIDE> r;
    r.load(static_cast<const uint16_t *>(p) + row * l.D, l);
    r.template widen<T>(o);
}
template <typename T, bool WIDE>
__device__ __forceinline__ void store_at(uint16_t *p, const Lane<WIDE> &l, const f2 *v) {  // p: the token's row
    uint32_t w[NC / 2];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) w[i] = narrow2<T>(v[i]);
    if constexpr (WIDE) {
        *reinterpret_cast<uint2 *>(p + l.c) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (l.has(i)) p[l.chan(i)] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

template <typename T, bool WIDE>
__device__ __forceinline__ void store_x(void *base, long long row, const Lane<WIDE> &l, const f2 *v) {
    store_at<T, WIDE>(static_cast<uint16_t *>(base) + row * l.D, l, v);
}

// Taps w[j] (of the input j tokens back) and bias.
template <typename T, int W, bool WIDE>
struct Taps {
    f2 w[W][NC / 2], bias[NC / 2];
    __device__ __forceinline__ void load(const ConvArgs &a, const Lane<WIDE> &l) {
        float v[NC * W], b[NC];
        if (WIDE && !a.w_f32 && a.w_wide) {  // NC W consecutive elements
            const uint32_t *p = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(a.w) + (long long)l.c * W);
            uint32_t u[NC * W / 2];
#pragma unroll
            for (int i = 0; i < NC * W / 2; i += 2) {
                const uint2 q = *reinterpret_cast<const uint2 *>(p + i);
                u[i] = q.x, u[i + 1] = q.y;
            }
#pragma unroll
            for (int i = 0; i < NC * W / 2; ++i) unpack2(widen2<T>(u[i]), v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < NC * W; ++i)
                v[i] = l.has(i / W) ? load_gate<T>(a.w, (long long)l.chan(i / W) * W + i % W, a.w_f32) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) b[i] = (a.bias && l.has(i)) ? load_gate<T>(a.bias, l.chan(i), a.w_f32) : 0.f;
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = pack2(v[2 * i * W + W - 1 - j], v[(2 * i + 1) * W + W - 1 - j]);
            bias[i] = pack2(b[2 * i], b[2 * i + 1]);
        }
    }
    // pre of pair i at input x with the W - 1 inputs before it in xs (nearest first)
    __device__ __forceinline__ f2 pre(int i, f2 x, const f2 (*xs)[NC / 2]) const {
        f2 p = fma2(w[0][i], x, bias[i]);
#pragma unroll
        for (int j = 1; j < W; ++j) p = fma2(w[j][i], xs[j - 1][i], p);
        return p;
    }
};

template <int W>
__device__ __forceinline__ void push(f2 (*xs)[NC / 2], const f2 *x) {
#pragma unroll
    for (int j = W - 1; j > 1; --j)
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) xs[j - 1][i] = xs[j - 2][i];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) xs[0][i] = x[i];
}

// The cached inputs of sequence n (zeros without them): xs[j-1] = input j tokens before its first.
template <typename T, int W, bool WIDE>
__device__ __forceinline__ void cached_inputs(const ConvArgs &a, long long n, const Lane<WIDE> &l, f2 (*xs)[NC / 2]) {
#pragma unroll
    for (int j = 1; j < W; ++j) {
        if (a.state_in) {
            load_x<T, WIDE>(a.state_in, n * (W - 1) + (W - 1 - j), l, xs[j - 1]);
        } else {
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) xs[j - 1][i] = 0ull;
        }
    }
}

// The W - 1 inputs before token t0 of a sequence that starts at token `start` of the row: tokens of it, or cached.
template <typename T, int W, bool WIDE>
__device__ __forceinline__ void inputs_before(const ConvArgs &a, const uint16_t *row, int t0, int start, long long n,
                                              const Lane<WIDE> &l, f2 (*xs)[NC / 2]) {
#pragma unroll
    for (int j = 1; j < W; ++j) {
        const int back = j - (t0 - start);  // > 0: that many tokens before the sequence's first
        if (back <= 0) {
            Raw<WIDE> r;
            r.load(row + (long long)(t0 - j) * a.x_ld, l);
            r.template widen<T>(xs[j - 1]);
        } else if (a.state_in && back < W) {
            load_x<T, WIDE>(a.state_in, n * (W - 1) + (W - 1 - back), l, xs[j - 1]);
        } else {
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) xs[j - 1][i] = 0ull;
        }
    }
}

// Block -> channels of this lane and (row, first token) of this warp's walk; false past either end.
template <bool WIDE>
__device__ __forceinline__ bool my_walk(const ConvArgs &a, Lane<WIDE> &l, int &b, int &t0, long long &tblock) {
    const unsigned tb = (__umulhi(blockIdx.x, a.cblocks_m) + blockIdx.x) >> a.cblocks_s;
    tblock = tb;
    const int c0 = (int)(blockIdx.x - tb * a.cblocks) * 32 * NC;
    l.c = WIDE ? c0 + (int)threadIdx.x * NC : c0 + (int)threadIdx.x;
    l.D = a.D;
    const unsigned walk = tb * WALKS + threadIdx.y;
    b = (int)((__umulhi(walk, a.tiles_m) + walk) >> a.tiles_s);
    t0 = (int)(walk - b * a.tiles) * a.tt;
    return (!WIDE || l.c < a.D) && b < a.B;  // (all lanes of a warp share in the copies of the ragged form)
}

// One tensor's tokens of a warp on their way from memory, as asynchronous copies into a ring of kAhead tokens in shared
// memory: reads in flight cost no registers.  WIDE: every lane copies its own 8 bytes.  Otherwise rows start at any
// element: the lanes copy the aligned 16-byte pieces that hold the warp's 128 channels (17 at most, cut off at the
// tensor's ends) and read their channels from there.
constexpr int kAhead = 16;
template <bool WIDE>
struct RingRow {
    static constexpr int bytes = WIDE ? 32 * 8 : 18 * 16;  // of one token of a warp
};
template <bool WIDE>
struct Pipe {
    const uint16_t *next;   // token to copy next: this lane's channels (WIDE) or the warp's first
    const uint16_t *cur;    // token to take next (its misalignment)
    const char *lo, *hi;    // the tensor
    long long ld;
    uint32_t ring;          // this lane's or the warp's part of slot 0
    int lane, need;         // bytes of a row that the warp needs
    __device__ __forceinline__ void init(unsigned char *smem, const void *base, long long rows, long long ld_, long long row,
                                         const Lane<WIDE> &l) {
        lane = threadIdx.x;
        ld = ld_;
        const int c0 = WIDE ? l.c : l.c - lane;
        next = cur = static_cast<const uint16_t *>(base) + row * ld + c0;
        ring = smem_u32(smem) + threadIdx.y * (kAhead * RingRow<WIDE>::bytes) + (WIDE ? lane * 8 : 0);
        lo = static_cast<const char *>(base);
        hi = reinterpret_cast<const char *>(static_cast<const uint16_t *>(base) + (rows - 1) * ld + l.D);
        need = 2 * min(32 * NC, l.D - c0);
    }
    __device__ __forceinline__ void issue(int slot, bool in) {
        if (in) {
            const uint32_t to = ring + slot * RingRow<WIDE>::bytes;
            if constexpr (WIDE) {
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to), "l"(next) : "memory");
            } else {
                const uintptr_t at = reinterpret_cast<uintptr_t>(next);
                const int skew = (int)(at & 15);
                if (lane * 16 < skew + need) {
                    const char *src = reinterpret_cast<const char *>(at - skew) + lane * 16;
                    if (src >= lo) {
                        const long long left = hi - src;
                        const int n = left < 16 ? (int)left : 16;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to + lane * 16), "l"(src), "r"(n)
                                     : "memory");
                    } else {  // the piece begins before the tensor
                        for (int i = skew; i < 16 && i - skew < need; i += 2)
                            sts16(to + i, *reinterpret_cast<const uint16_t *>(src + i));
                    }
                }
            }
        }
        next += ld;
    }
    template <typename T>
    __device__ __forceinline__ void take(int slot, f2 *o) {
        const uint32_t from = ring + slot * RingRow<WIDE>::bytes;
        if constexpr (WIDE) {
            uint32_t a, b;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(a), "=r"(b) : "r"(from) : "memory");
            o[0] = widen2<T>(a), o[1] = widen2<T>(b);
        } else {
            // (channels past the row's end hold what follows it, or nothing: they are never stored or summed)
            const uint32_t p = from + (uint32_t)(reinterpret_cast<uintptr_t>(cur) & 15) + lane * 2;
            o[0] = widen2<T>((uint32_t)lds16v(p) | (uint32_t)lds16v(p + 64) << 16);
            o[1] = widen2<T>((uint32_t)lds16v(p + 128) | (uint32_t)lds16v(p + 192) << 16);
            cur += ld;
        }
    }
    // One group of copies at most GROUPS - 1 behind the newest is complete for the whole warp.
    template <int LEFT>
    static __device__ __forceinline__ void arrive() {
        cp_async_wait<LEFT>();
        if (!WIDE) __syncwarp();
    }
    static __device__ __forceinline__ uint16_t lds16v(uint32_t at) {
        uint16_t v;
        asm volatile("ld.shared.b16 %0, [%1];\n" : "=h"(v) : "r"(at) : "memory");
        return v;
    }
};

template <bool V>
struct Flag {
    static constexpr bool value = V;
};

// Bound by HBM with the fp32 work of the SiLU close behind (58 % of the issue slots): 2 x 4096 x 12288 bf16 takes 76 us for
// 403 MB, 5.3 TB/s.  Ragged rows cost three times the instructions an element (2-byte accesses to shared memory and
// out): 5311 x 4099 fp16 takes 39 us for 87 MB, 2.3 TB/s.
template <typename T, int W, bool WIDE, bool PACKED>
__global__ void __launch_bounds__(32 * WALKS, WIDE ? 4 : 3) conv_fwd_kernel(const ConvArgs a) {
    constexpr int U = 4, GROUPS = kAhead / U;   // tokens a group of copies; groups
    extern __shared__ __align__(16) unsigned char ring[];
    if (PACKED && blockIdx.x == 0 && threadIdx.y == 0) check_cu(a.cu, a.N, a.T, a.err);
    Lane<WIDE> l;
    int b, t0;
    long long tblock;
    if (!my_walk(a, l, b, t0, tblock)) return;
    const int t1 = min(a.T, t0 + a.tt);
    const uint16_t *row = static_cast<const uint16_t *>(a.x) + (long long)b * a.T * a.x_ld;
    const long long row0 = (long long)b * a.T;

    Pipe<WIDE> px;
    px.init(ring, a.x, (long long)a.B * a.T, a.x_ld, row0 + t0, l);
    auto fetch = [&](int t, int g) {
#pragma unroll
        for (int u = 0; u < U; ++u) px.issue(g * U + u, t + u < t1);
        cp_async_commit();
    };
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) fetch(t0 + g * U, g);
    uint16_t *out = static_cast<uint16_t *>(a.y) + (row0 + t0) * a.D;
    Taps<T, W, WIDE> taps;
    taps.load(a, l);
    SeqWalk sw;
    if (PACKED) sw.find(a.cu, a.N, t0);
    long long seq = PACKED ? sw.cur() : b;
    f2 xs[W - 1][NC / 2];
    if (PACKED && sw.bound == t0)
        cached_inputs<T, W, WIDE>(a, seq, l, xs);  // (replaced at the first token)
    else
        inputs_before<T, W, WIDE>(a, row, t0, PACKED ? max(0, a.cu[seq]) : 0, seq, l, xs);
    auto write_state = [&](long long n, const f2(*s)[NC / 2]) {
        if (!a.state_out) return;
#pragma unroll
        for (int j = 1; j < W; ++j) store_x<T, WIDE>(a.state_out, n * (W - 1) + (W - 1 - j), l, s[j - 1]);
    };
    auto empty = [&](long long n) {
        f2 e[W - 1][NC / 2];
        cached_inputs<T, W, WIDE>(a, n, l, e);
        write_state(n, e);
    };
    // U tokens from t; CHECKED: some of them may lie past t1, or a sequence may start or end among them
    auto tokens = [&](int t, int g, auto checked) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (checked.value && t + u >= t1) break;
            if (PACKED && checked.value && t + u == sw.bound && sw.step(t + u, empty)) {
                seq = sw.cur();
                cached_inputs<T, W, WIDE>(a, seq, l, xs);
            }
            f2 x[NC / 2], y[NC / 2];
            px.template take<T>(g * U + u, x);
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
                y[i] = taps.pre(i, x[i], xs);
                if (a.silu) y[i] = mul2(y[i], sigmoid2(y[i]));
            }
            store_at<T, WIDE>(out, l, y);
            out += a.D;
            push<W>(xs, x);
            if (PACKED && checked.value && t + u + 1 == sw.bound) write_state(seq, xs);
        }
    };
    int g = 0;
    for (int t = t0; t < t1; t += U) {
        Pipe<WIDE>::template arrive<GROUPS - 1>();
        if (t + U <= t1 && !(PACKED && sw.bound >= t && sw.bound <= t + U))
            tokens(t, g, Flag<false>());
        else
            tokens(t, g, Flag<true>());
        if (!WIDE) __syncwarp();  // (all lanes have read the slots)
        fetch(t + GROUPS * U, g);
        g = g + 1 == GROUPS ? 0 : g + 1;
    }
    cp_async_wait<0>();
    if (!PACKED && t1 == a.T) write_state(seq, xs);
    if (PACKED && t1 == a.T && sw.bound == a.T) sw.step(a.T, empty);
}

// One row and NC channels a thread for its few tokens: the thread that reads a channel's cached inputs is the one that
// replaces them.  Few registers, so that a launch with one token keeps the memory busy by its number of threads.  Bound by
// the latency of one round of loads a block: 256 x 12288 takes 12.3 us for 50 MB, 4.1 TB/s.
template <typename T, int W, bool WIDE>
__global__ void __launch_bounds__(32 * WALKS, 5) conv_step_kernel(const ConvArgs a) {
    Lane<WIDE> l;
    int b, t0;
    long long tblock;
    if (!my_walk(a, l, b, t0, tblock)) return;
    const uint16_t *row = static_cast<const uint16_t *>(a.x) + (long long)b * a.T * a.x_ld;
    Raw<WIDE> raw;
    raw.load(row, l);
    f2 xs[W - 1][NC / 2];
    cached_inputs<T, W, WIDE>(a, b, l, xs);
    Taps<T, W, WIDE> taps;
    taps.load(a, l);
    for (int t = 0; t < a.T; ++t) {
        f2 x[NC / 2], y[NC / 2];
        raw.template widen<T>(x);
        if (t + 1 < a.T) raw.load(row + (long long)(t + 1) * a.x_ld, l);
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) {
            y[i] = taps.pre(i, x[i], xs);
            if (a.silu) y[i] = mul2(y[i], sigmoid2(y[i]));
        }
        store_x<T, WIDE>(a.y, (long long)b * a.T + t, l, y);
        push<W>(xs, x);
    }
#pragma unroll
    for (int j = 1; j < W; ++j) store_x<T, WIDE>(a.state_out, (long long)b * (W - 1) + (W - 1 - j), l, xs[j - 1]);
}

// The sums of dw, db and dx of 4 channels stay in registers (126 a thread): two blocks an SM, which the latency of the
// SiLU's exponential and reciprocal bounds before HBM does (50 % of the issue slots; three blocks spill 350 bytes a
// thread).  2 x 4096 x 12288 bf16: 140 us for 604 MB, 4.3 TB/s.
template <typename T, int W, bool WIDE, bool PACKED>
__global__ void __launch_bounds__(32 * WALKS, 2) conv_bwd_kernel(const ConvArgs a) {
    constexpr int U = 4, GROUPS = kAhead / U;
    constexpr int NP = NC * (W + 1);
    extern __shared__ __align__(16) unsigned char ring[];  // two rings, then the walks' sums in their place
    float(*s_part)[NP][32] = reinterpret_cast<float(*)[NP][32]>(ring);
    if (PACKED && blockIdx.x == 0 && threadIdx.y == 0) check_cu(a.cu, a.N, a.T, a.err);
    Lane<WIDE> l;
    int b, t0;
    long long tblock;
    const bool live = my_walk(a, l, b, t0, tblock);
    f2 dw[W][NC / 2], db[NC / 2];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
        db[i] = 0ull;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0ull;
    }
    if (live) {
        const int t1 = min(a.T, t0 + a.tt);
        const int tend = min(a.T, t1 + W - 1);  // the sums of the last W - 1 inputs close past the walk's end
        const uint16_t *row = static_cast<const uint16_t *>(a.x) + (long long)b * a.T * a.x_ld;
        const long long row0 = (long long)b * a.T;
        Pipe<WIDE> px, pg;
        px.init(ring, a.x, (long long)a.B * a.T, a.x_ld, row0 + t0, l);
        pg.init(ring + WALKS * kAhead * RingRow<WIDE>::bytes, a.dy, (long long)a.B * a.T, a.D, row0 + t0, l);
        auto fetch = [&](int t, int g) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                px.issue(g * U + u, t + u < tend);
                pg.issue(g * U + u, t + u < tend);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) fetch(t0 + g * U, g);
        uint16_t *out = static_cast<uint16_t *>(a.dx) + (row0 + t0 - (W - 1)) * a.D;  // (stored to from token t0 on)
        Taps<T, W, WIDE> taps;
        taps.load(a, l);
        f2 xs[W - 1][NC / 2], acc[W - 1][NC / 2];  // acc[j-1]: the open sum of dx, j tokens back
#pragma unroll
        for (int j = 1; j < W; ++j)
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) acc[j - 1][i] = 0ull;

        SeqWalk sw;
        if (PACKED) sw.find(a.cu, a.N, t0);
        long long seq = PACKED ? sw.cur() : b;
        int start = 0;
        if (PACKED && sw.bound != t0) start = max(0, a.cu[seq]);
        if (PACKED && sw.bound == t0)
            cached_inputs<T, W, WIDE>(a, seq, l, xs);  // (replaced at the first token)
        else
            inputs_before<T, W, WIDE>(a, row, t0, start, seq, l, xs);
        // A finished sum: of an input of this walk, or of a cached input of a sequence that starts in it.
        auto emit = [&](int s, const f2 *v) {
            if (s >= start) {
                if (s >= t0 && s < t1) store_x<T, WIDE>(a.dx, row0 + s, l, v);
            } else if (start >= t0 && a.dstate_in && W - 1 + s - start >= 0) {
                store_x<T, WIDE>(a.dstate_in, seq * (W - 1) + (W - 1 + s - start), l, v);
            }
        };
        // The last W - 1 sums of a sequence that ends at token e: also the final state's gradient.
        auto flush = [&](int e) {
#pragma unroll
            for (int j = W - 1; j >= 1; --j) {
                if (a.dstate_out) {
                    f2 d[NC / 2];
                    load_x<T, WIDE>(a.dstate_out, seq * (W - 1) + (W - 1 - j), l, d);
#pragma unroll
                    for (int i = 0; i < NC / 2; ++i) acc[j - 1][i] = add2(acc[j - 1][i], d[i]);
                }
                emit(e - j, acc[j - 1]);
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) acc[j - 1][i] = 0ull;
            }
        };
        auto empty = [&](long long n) {
            if (!a.dstate_in) return;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                f2 d[NC / 2];
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) d[i] = 0ull;
                if (a.dstate_out) load_x<T, WIDE>(a.dstate_out, n * (W - 1) + j, l, d);
                store_x<T, WIDE>(a.dstate_in, n * (W - 1) + j, l, d);
            }
        };
        bool open = true;  // the walk's last sequence is still to be flushed
        // U tokens from t; CHECKED: not all of them are the walk's own, well inside one sequence
        auto tokens = [&](int t, int g, auto checked) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (checked.value && (!open || t + u >= tend)) break;
                if (PACKED && checked.value && t + u == sw.bound) {
                    if (t + u > t0) flush(t + u);
                    if (t + u >= t1) {
                        open = false;
                        break;
                    }
                    if (sw.step(t + u, empty)) {
                        seq = sw.cur();
                        start = t + u;
                        cached_inputs<T, W, WIDE>(a, seq, l, xs);
                    }
                }
                const bool mine = !checked.value || t + u < t1;
                f2 x[NC / 2], d[NC / 2], done[NC / 2];
                px.template take<T>(g * U + u, x);
                pg.template take<T>(g * U + u, d);
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) {
                    if (a.silu) {
                        const f2 pre = taps.pre(i, x[i], xs), s = sigmoid2(pre);
                        // sig + pre sig (1 - sig)
                        d[i] = mul2(d[i], fma2(mul2(pre, s), fma2(s, both(-1.f), both(1.f)), s));
                    }
                    done[i] = fma2(taps.w[W - 1][i], d[i], acc[W - 2][i]);
#pragma unroll
                    for (int j = W - 2; j >= 1; --j) acc[j][i] = fma2(taps.w[j][i], d[i], acc[j - 1][i]);
                    acc[0][i] = mul2(taps.w[0][i], d[i]);
                    if (mine) {
                        dw[0][i] = fma2(d[i], x[i], dw[0][i]);
#pragma unroll
                        for (int j = 1; j < W; ++j) dw[j][i] = fma2(d[i], xs[j - 1][i], dw[j][i]);
                        db[i] = add2(db[i], d[i]);
                    }
                }
                push<W>(xs, x);
                if (checked.value)
                    emit(t + u - (W - 1), done);
                else
                    store_at<T, WIDE>(out, l, done);
                out += a.D;
            }
        };
        int g = 0;
        for (int t = t0; open && t < tend; t += U) {
            Pipe<WIDE>::template arrive<GROUPS - 1>();
            if (t + U <= t1 && t - (W - 1) >= max(t0, start) && !(PACKED && sw.bound >= t && sw.bound < t + U))
                tokens(t, g, Flag<false>());
            else
                tokens(t, g, Flag<true>());
            if (!WIDE) __syncwarp();  // (all lanes have read the slots)
            fetch(t + GROUPS * U, g);
            g = g + 1 == GROUPS ? 0 : g + 1;
        }
        cp_async_wait<0>();
        if (open && tend == a.T && (!PACKED || sw.bound == a.T)) flush(a.T);
        if (PACKED && t1 == a.T && sw.bound == a.T) sw.step(a.T, empty);
    }
    // the block's share of dw and db: its walks added in order
    __syncthreads();  // (the rings are read no more)
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            unpack2(dw[j][i], s_part[threadIdx.y][2 * i * W + W - 1 - j][threadIdx.x],
                    s_part[threadIdx.y][(2 * i + 1) * W + W - 1 - j][threadIdx.x]);
        unpack2(db[i], s_part[threadIdx.y][NC * W + 2 * i][threadIdx.x], s_part[threadIdx.y][NC * W + 2 * i + 1][threadIdx.x]);
    }
    __syncthreads();
    for (int i = threadIdx.y; i < NP; i += WALKS) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < WALKS; ++k) s += s_part[k][i][threadIdx.x];
        const bool weight = i < NC * W;
        const int e = weight ? i / W : i - NC * W;  // the thread's channel
        if (l.c >= a.D || !l.has(e)) continue;
        float *part = a.part + tblock * (W + 1) * a.D;
        part[weight ? (long long)l.chan(e) * W + i % W : (long long)a.D * W + l.chan(e)] = s;
    }
}

// Tokens a walk.  Long walks repeat fewer overlapping reads and start-ups (worth about 16 tokens a walk), short ones
// fill the chip; the length that minimises rounds of resident blocks times the tokens of one.  (2 x 4096 x 12288:
// the backward's 120 tokens a walk make 2.8 rounds of two blocks an SM, 64 make 5.05 and cost an eighth more.)
int conv_tt(const gdr_conv_problem *p, bool bwd) {
    const long long cb = (p->D + 32 * NC - 1) / (32 * NC), slots = (long long)kSMs * (bwd ? 2 : 4);
    long long best = 0;
    int best_tt = 8;
    for (int tt = 8; tt <= 128; tt += 8) {
        const long long walks = (long long)p->B * ((p->T + tt - 1) / tt);
        const long long rounds = ((walks + WALKS - 1) / WALKS * cb + slots - 1) / slots;
        const long long cost = rounds * (tt + 16);
        if (best == 0 || cost < best) best = cost, best_tt = tt;
    }
    return best_tt;
}

struct ConvGrid {
    int tt, tiles, cblocks;
    long long tblocks;
};
ConvGrid conv_grid(const gdr_conv_problem *p, int tt) {
    ConvGrid g;
    g.tt = tt;
    g.tiles = (p->T + g.tt - 1) / g.tt;
    g.cblocks = (p->D + 32 * NC - 1) / (32 * NC);
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

// Blocks fit the grid's x dimension, and walks an int.
bool grid_fits(const ConvGrid &g) { return g.tblocks * g.cblocks <= 0x7fffffffLL && g.tblocks * WALKS <= 0x7fffffffLL; }

template <typename K>
cudaError_t launch_ring(K k, dim3 grid, size_t smem, cudaStream_t s, const ConvArgs &a) {
    const cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
    return launch_plain(k, grid, dim3(32, WALKS), smem, s, a);
}
template <typename T, int W, bool WIDE, bool PACKED>
cudaError_t conv_one(const ConvArgs &a, bool bwd, dim3 grid, cudaStream_t s) {
    constexpr size_t one = (size_t)WALKS * kAhead * RingRow<WIDE>::bytes, sums = (size_t)WALKS * NC * (W + 1) * 32 * sizeof(float);
    if (bwd) return launch_ring(conv_bwd_kernel<T, W, WIDE, PACKED>, grid, 2 * one > sums ? 2 * one : sums, s, a);
    return launch_ring(conv_fwd_kernel<T, W, WIDE, PACKED>, grid, one, s, a);
}
template <typename T, bool WIDE, bool PACKED>
cudaError_t conv_w(const ConvArgs &a, int W, bool bwd, const ConvGrid &g, cudaStream_t s) {
    const dim3 grid((unsigned)(g.tblocks * g.cblocks));
    if (W == 2) return conv_one<T, 2, WIDE, PACKED>(a, bwd, grid, s);
    if (W == 3) return conv_one<T, 3, WIDE, PACKED>(a, bwd, grid, s);
    return conv_one<T, 4, WIDE, PACKED>(a, bwd, grid, s);
}
template <typename T, bool WIDE>
cudaError_t conv_step_w(const ConvArgs &a, int W, const ConvGrid &g, cudaStream_t s) {
    const dim3 grid((unsigned)(g.tblocks * g.cblocks)), block(32, WALKS);
    if (W == 2) return launch_plain(conv_step_kernel<T, 2, WIDE>, grid, block, 0, s, a);
    if (W == 3) return launch_plain(conv_step_kernel<T, 3, WIDE>, grid, block, 0, s, a);
    return launch_plain(conv_step_kernel<T, 4, WIDE>, grid, block, 0, s, a);
}
cudaError_t launch_conv_step(const gdr_conv_problem *p, const ConvArgs &a, bool wide, const ConvGrid &g, cudaStream_t s) {
    if (p->dtype == GDR_BF16)
        return wide ? conv_step_w<__nv_bfloat16, true>(a, p->W, g, s) : conv_step_w<__nv_bfloat16, false>(a, p->W, g, s);
    return wide ? conv_step_w<__half, true>(a, p->W, g, s) : conv_step_w<__half, false>(a, p->W, g, s);
}

template <typename T>
cudaError_t conv_t(const ConvArgs &a, int W, bool wide, bool bwd, const ConvGrid &g, cudaStream_t s) {
    if (wide) return a.cu ? conv_w<T, true, true>(a, W, bwd, g, s) : conv_w<T, true, false>(a, W, bwd, g, s);
    return a.cu ? conv_w<T, false, true>(a, W, bwd, g, s) : conv_w<T, false, false>(a, W, bwd, g, s);
}
cudaError_t launch_conv(const gdr_conv_problem *p, const ConvArgs &a, bool wide, bool bwd, const ConvGrid &g, cudaStream_t s) {
    return p->dtype == GDR_BF16 ? conv_t<__nv_bfloat16>(a, p->W, wide, bwd, g, s) : conv_t<__half>(a, p->W, wide, bwd, g, s);
}

ConvArgs conv_args(const gdr_conv_problem *p, const ConvGrid &g, bool w_wide, unsigned *err) {
    ConvArgs a = {};
    a.cu = p->cu_seqlens;
    a.err = err;
    a.x_ld = p->x_ld;
    a.B = p->B, a.T = p->T, a.D = p->D;
    a.N = p->cu_seqlens ? p->num_seqs : p->B;
    a.tt = g.tt, a.tiles = g.tiles, a.cblocks = g.cblocks;
    div_magic(g.tiles, a.tiles_m, a.tiles_s);
    div_magic(g.cblocks, a.cblocks_m, a.cblocks_s);
    a.w_f32 = p->weight_dtype == GDR_FP32;
    a.w_wide = w_wide;
    a.silu = (p->flags & GDR_CONV_SILU) != 0;
    return a;
}

size_t conv_state_bytes(const gdr_conv_problem *p) {
    return (size_t)(p->cu_seqlens ? p->num_seqs : p->B) * (p->W - 1) * p->D * 2;
}

size_t tokens_bytes(const gdr_conv_problem *p) { return (size_t)p->B * p->T * p->D * 2; }

// Whether an output of `n` bytes touches the tokens or the states that other threads may still read: each walk reads the
// W - 1 tokens before its own (the backward also those behind).
bool conv_touches(const gdr_conv_problem *p, const void *out, size_t n, const void *tokens, int64_t ld, const void *states) {
    return p->T > 0 && (touches(out, n, tokens, (size_t)p->B * p->T, (size_t)p->D * 2, (size_t)ld * 2) ||
                        touches(out, n, states, 1, conv_state_bytes(p), conv_state_bytes(p)));
}

// Without tokens the states pass through: dst = src, or zeros.
gdr_status conv_no_tokens(const gdr_conv_problem *p, const void *src, void *dst, cudaStream_t s) {
    if (!dst || dst == src) return GDR_OK;
    const size_t n = conv_state_bytes(p);
    return cuda_status(src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dst, 0, n, s));
}

gdr_status conv_fwd_core(const gdr_conv_problem *p, const void *x, const void *weight, const void *bias,
                         const void *state_in, void *y, void *state_out, bool step, void *stream) {
    if (!weight || (p->T > 0 && (!x || !y))) return GDR_ERR_NULL;
    const size_t ws = esize(p->weight_dtype);
    for (const void *q : {x, state_in, (const void *)y, (const void *)state_out})
        if (!aligned_to(q, 2)) return GDR_ERR_ALIGN;
    if (!aligned_to(weight, ws) || !aligned_to(bias, ws)) return GDR_ERR_ALIGN;
    if (!step && (conv_touches(p, y, tokens_bytes(p), x, p->x_ld, state_in) ||
                  conv_touches(p, state_out, conv_state_bytes(p), x, p->x_ld, state_in)))
        return GDR_ERR_UNSUPPORTED;
    bool wide = p->D % 4 == 0 && p->x_ld % 4 == 0;
    for (const void *q : {x, state_in, (const void *)y, (const void *)state_out}) wide = wide && aligned_to(q, 8);
    const ConvGrid g = conv_grid(p, !step ? conv_tt(p, false) : p->T > 0 ? p->T : 1);
    if (!grid_fits(g)) return GDR_ERR_SHAPE;
    unsigned *err = nullptr;
    gdr_status st = device_state(&err);
    if (st != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->T == 0) return conv_no_tokens(p, state_in, state_out, cs);
    ConvArgs a = conv_args(p, g, aligned_to(weight, 8), err);
    a.x = x, a.w = weight, a.bias = bias, a.state_in = state_in, a.y = y, a.state_out = state_out;
    return timed(K_CONV_FWD, cs, [&] {
        return step ? launch_conv_step(p, a, wide, g, cs) : launch_conv(p, a, wide, false, g, cs);
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
    return conv_fwd_core(p, x, weight, bias, state_in, y, state_out, false, stream);
}

gdr_status gdr_conv_step(const gdr_conv_problem *p, const void *x, const void *weight, const void *bias, void *state,
                         void *y, void *stream) {
    gdr_status st = check_conv(p);
    if (st != GDR_OK) return st;
    if (p->cu_seqlens) return GDR_ERR_UNSUPPORTED;
    if (!state) return GDR_ERR_NULL;
    return conv_fwd_core(p, x, weight, bias, state, y, state, true, stream);
}

gdr_status gdr_conv_bwd_workspace_size(const gdr_conv_problem *p, size_t *bytes) {
    gdr_status st = check_conv(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    *bytes = 0;
    if (p->T == 0) return GDR_OK;
    const ConvGrid g = conv_grid(p, conv_tt(p, true));
    *bytes = round_up((size_t)g.tblocks * p->D * (p->W + 1) * sizeof(float), 256);
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
    for (bool states : {false, true}) {
        const void *out = states ? dstate_in : dx;
        const size_t n = states ? conv_state_bytes(p) : tokens_bytes(p);
        if (conv_touches(p, out, n, x, p->x_ld, state_in) || conv_touches(p, out, n, dy, p->D, dstate_out))
            return GDR_ERR_UNSUPPORTED;
    }
    bool wide = p->D % 4 == 0 && p->x_ld % 4 == 0;
    for (const void *q : {x, dy, state_in, dstate_out, (const void *)dx, (const void *)dstate_in})
        wide = wide && aligned_to(q, 8);
    const ConvGrid g = conv_grid(p, conv_tt(p, true));
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
    ConvArgs a = conv_args(p, g, aligned_to(weight, 8), err);
    a.x = x, a.w = weight, a.bias = bias, a.state_in = state_in, a.dy = dy, a.dstate_out = dstate_out;
    a.dx = dx, a.dstate_in = dstate_in;
    a.part = static_cast<float *>(workspace);
    const bool bf = p->dtype == GDR_BF16;
    st = timed(K_CONV_BWD, cs, [&] { return launch_conv(p, a, wide, true, g, cs); });
    if (st != GDR_OK) return st;
    return timed(K_REDUCE, cs, [&] {
        const RowSums out[2] = {{dweight, p->D * p->W}, {dbias, p->D}};
        return launch_reduce_rows(a.part, g.tblocks, (long long)p->D * (p->W + 1), out, dbias ? 2 : 1, bf, a.w_f32, cs);
    });
}

}  // extern "C"
