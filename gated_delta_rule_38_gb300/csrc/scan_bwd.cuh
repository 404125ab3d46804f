// Backward of the selective state space scan.  With gy_t = dy_t silu(z_t), a_t = exp(delta_t A):
//
//   g_t = C_t gy_t + a_{t+1} g_{t+1}                   (the gradient of h_t)
//   dC_t = sum_d gy_t h_t,  dB_t = sum_d g_t delta_t x_t            (sums over a group's channels)
//   S_t = sum_n g_t B_t,  q_t = g_t a_t h_{t-1},  Q_t = sum_n A q_t
//   dx_t = delta_t S_t + D gy_t,  ddelta_t = x_t S_t + Q_t,  ddt_t = ddelta_t sigmoid(dt_t + bias) with softplus
//   dz_t = dy_t yp_t sig(z)(1 + z (1 - sig(z))),  yp_t = C_t . h_t + D x_t
//   dA = sum_t delta_t q_t,  dD = sum_t gy_t x_t,  ddt_bias = sum_t ddt_t,  dh0 = a_0 g_0
//
// A block walks a segment backwards in tiles of 16 tokens.  The forward saved the state before every tile; the block
// runs a tile forward once, keeping the state before every 4 tokens in shared memory, then takes the groups of 4
// tokens from the last to the first: forward again with a_t and h_t in registers, and backward through them.  The sums
// over the states stay in the lanes of a channel; dB and dC are summed over a thread's channels in registers, over
// the warp's and the block's through shared memory, and over the blocks by a second kernel, all in a fixed order.
// As in the forward, segments give parallelism along the token axis: a first pass leaves the gradient that each
// segment alone sends back past its start, and the scan joins them.
#pragma once

#include "scan.cuh"

namespace gdr {
namespace scan {
namespace {

constexpr int TT = SAVE;   // tokens a tile
constexpr int SB = 4;      // tokens a group

template <int L>
struct Bwd {
    static constexpr int NP = 4 * L;
    static constexpr int CB = L >= 4 ? 512 / L : 128;    // channels a block
    static constexpr int NW = CB * L / 128;              // warps a block
    static constexpr int NT = 32 * NW;
    static constexpr int CL = 32 / L;                    // channel lanes of a warp
    static constexpr int NVEC = TT * CB / 8;
    static constexpr int VPT = NVEC > NT ? NVEC / NT : 1;
    static constexpr int VROW = CB / 8, VSTEP = NT / VROW;
    static constexpr int BW = NP >= 8 ? 8 : 4;           // states of a vector of B or C
    static constexpr int BROW = NP / BW;
    static_assert(TT * BROW <= NT, "one vector of B a thread");
    // The ragged rows' elements are taken as pairs of tokens of a channel: task i is the pair (2 (i / COLS), + 1) of 32
    // channels, warp w takes w, w + NW, ..  A lane sums over tokens in GROUP sums that take the tokens in the order of
    // the whole vectors' threads (token modulo CLS), so that both forms give the same bits.
    static constexpr int COLS = CB / 32, TASKS = TT / 2 * COLS / NW;
    static constexpr int CLS = VSTEP < TT ? VSTEP : TT;
    static constexpr int NCOL = COLS > NW ? COLS / NW : 1;
    static constexpr int PL = CLS / 2 / (NW > COLS ? NW / COLS : 1);
    static constexpr int GROUP = NCOL * PL;
    static_assert(GROUP <= 4 && TASKS % GROUP == 0, "sums of a lane");
};

// As in the forward: the staged tile and, behind it in dynamic shared memory, the raw ones (dt, dy, z, x; C, B as pieces).
template <int L, bool LOCAL>
struct BwdStage {
    using W = Bwd<L>;
    static constexpr int M = LOCAL ? 3 : 4, MB = LOCAL ? 1 : 2, RB = W::NP < 8 ? 16 : W::NP + 8;
    uint16_t raw_bc[2][MB][TT][W::NP];                   // C, B
    float delta[TT][W::CB];                              // then the gradient of delta
    float gy[TT][W::CB];                                 // then yp
    float bias[W::CB];
    int first[2][TT], last[2][TT], any[4];
    static __host__ __device__ constexpr int row(bool vec) { return vec ? W::CB : W::CB + 8; }
};
template <int L>
struct BwdFull : BwdStage<L, false> {
    using W = Bwd<L>;
    float x[TT][W::CB];                                  // then dx
    float start[TT / SB][4][W::NT][4];                   // the state before every group: thread-private
    float red[W::NW][2][W::CL][2 * W::NP];               // two tokens' dB | dC of a warp's channel lanes
    float bc[W::NW][TT][2 * W::NP];                      // a warp's sums of dB | dC
};
template <int L, bool LOCAL>
size_t raw_bytes(bool vec, bool vec_bc) {
    using S = BwdStage<L, LOCAL>;
    return sizeof(uint16_t) * (2 * S::M * TT * S::row(vec) + (vec_bc ? 0 : 2 * S::MB * TT * S::RB));
}

// A block's view of its tiles: the copies, and the tensors' rows.
template <typename T, int L, bool LOCAL, bool PACKED>
struct Tiles {
    using W = Bwd<L>;
    using S = BwdStage<L, LOCAL>;
    const ScanArgs &a;
    S &sm;
    uint16_t *raws;
    const Chans<W::CB> &ch;
    long long row0;
    int t0, t1, tid, vc, vt, vn, bn, bt;
    bool vec, vec_bc;
    __device__ __forceinline__ Tiles(const ScanArgs &a_, S &s_, void *raws_, const Chans<W::CB> &c_, int b, int t0_, int t1_)
        : a(a_), sm(s_), raws(static_cast<uint16_t *>(raws_)), ch(c_), row0((long long)b * a_.T), t0(t0_), t1(t1_), vec(a_.vec),
          vec_bc(a_.vec_bc) {
        tid = threadIdx.x;
        vc = (tid % W::VROW) * 8, vt = tid / W::VROW, vn = ch.count - vc;
        bn = (tid % W::BROW) * 8, bt = tid / W::BROW;
    }
    __device__ __forceinline__ uint16_t *raw(int buf, int m, int j, bool v) const {
        return raws + ((buf * S::M + m) * TT + j) * S::row(v);
    }
    __device__ __forceinline__ uint16_t *rag_bc(int buf, int m, int j) const {
        return raw(2, 0, 0, vec) + ((buf * S::MB + m) * TT + j) * S::RB;
    }
    // dt, dy, z, x
    __device__ __forceinline__ Rows src(int m) const {
        const void *p = m == 0 ? a.dt : m == 1 ? a.dy : m == 2 ? a.z : a.x;
        const long long ld = m == 0 ? a.dt_ld : m == 1 ? a.D : m == 2 ? a.z_ld : a.x_ld;
        return Rows{static_cast<const uint16_t *>(p), ld, ch.first, (long long)a.B * a.T, a.D};
    }
    __device__ __forceinline__ Rows src_bc(int m) const {
        return Rows{static_cast<const uint16_t *>(m ? a.Bm : a.Cm), m ? a.b_ld : a.c_ld, ch.g * a.N, (long long)a.B * a.T, a.G * a.N};
    }
    // The copies of the tile at `base` into buffer `buf`.
    __device__ __forceinline__ void fetch(int base, int buf) const {
        if (base >= t0) {
            const int rows = min(TT, t1 - base);
#pragma unroll
            for (int m = 0; m < S::M; ++m) {
                if (m == 2 && !a.z) continue;
                if (vec) {
#pragma unroll
                    for (int k = 0; k < W::VPT; ++k) {
                        const int j = vt + k * W::VSTEP;
                        if (j < rows && vn > 0) copy16(raw(buf, m, j, true) + vc, src(m).at(row0 + base + j) + vc);
                    }
                } else {
                    copy_rows<W::NT, W::CB / 8 + 1>(raw(buf, m, 0, false), S::row(false), src(m), row0 + base, rows, ch.count);
                }
            }
#pragma unroll
            for (int m = 0; m < S::MB; ++m) {
                if (!vec_bc) {
                    copy_rows<W::NT, W::NP / 8 + 2>(rag_bc(buf, m, 0), S::RB, src_bc(m), row0 + base, rows, a.N);
                } else if constexpr (W::BW == 8) {
                    if (bt < rows)
                        copy8(&sm.raw_bc[buf][m][bt][bn], src_bc(m).at(row0 + base + bt) + bn, bn < a.N);
                    else if (bt < TT)  // past the end: zeros
                        *reinterpret_cast<uint4 *>(&sm.raw_bc[buf][m][bt][bn]) = make_uint4(0, 0, 0, 0);
                }
            }
            if (PACKED) tile_edges<TT>(a, base, t1, sm.first[buf], sm.last[buf], &sm.any[buf]);
        }
        copies_commit();
    }
    // Pairs of tokens of one channel, for the ragged rows: consecutive lanes take consecutive channels.
    template <typename F>
    __device__ __forceinline__ void each_pair(F &&f) const {
        for (int rep = 0; rep < W::TASKS / W::GROUP; ++rep)
#pragma unroll
            for (int k = 0; k < W::GROUP; ++k) {
                const int i = (tid >> 5) + W::NW * (rep * W::GROUP + k);
                f(i / W::COLS * 2, i % W::COLS * 32 + (tid & 31), k);
            }
    }
    __device__ __forceinline__ f2 pair_of(int buf, int m, int base, int j, int c) const {
        const Rows r = src(m);
        const uint16_t lo = raw(buf, m, j, false)[r.skew(row0 + base + j) + c];
        const uint16_t hi = raw(buf, m, j + 1, false)[r.skew(row0 + base + j + 1) + c];
        return widen2<T>((uint32_t)lo | (uint32_t)hi << 16);
    }
    __device__ __forceinline__ f2 delta_of(f2 raw_dt, f2 bias) const {
        const f2 d = add2(raw_dt, bias);
        return a.softplus ? softplus2(d) : d;
    }
    // delta and gy (and x) of the tile that has arrived in `buf`; a step of zero and no gradient past the ends.
    __device__ __forceinline__ void stage(int base, int buf, float (*xs)[W::CB]) const {
        if (!(vec && vec_bc)) __syncthreads();
        if (vec) {
#pragma unroll
            for (int k = 0; k < W::VPT; ++k) {
                const int j = vt + k * W::VSTEP;
                if (j >= TT) break;
                f2 d[4], g[4], v[4];
                const bool in = base + j < t1 && vn > 0;
                if (in) {
                    widen8<T>(*reinterpret_cast<const uint4 *>(raw(buf, 0, j, true) + vc), d);
                    widen8<T>(*reinterpret_cast<const uint4 *>(raw(buf, 1, j, true) + vc), g);
                    get8(&sm.bias[vc], v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = delta_of(d[i], v[i]);
                    if (a.z) {
                        widen8<T>(*reinterpret_cast<const uint4 *>(raw(buf, 2, j, true) + vc), v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], mul2(v[i], sigmoid2(v[i])));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = g[i] = 0ull;
                }
                put8(&sm.delta[j][vc], d);
                put8(&sm.gy[j][vc], g);
                if (!LOCAL) {
                    f2 x[4] = {0ull, 0ull, 0ull, 0ull};
                    if (in) widen8<T>(*reinterpret_cast<const uint4 *>(raw(buf, LOCAL ? 0 : 3, j, true) + vc), x);
                    put8(&xs[j][vc], x);
                }
            }
        } else {
            each_pair([&](int j, int c, int) {
                const f2 d = delta_of(pair_of(buf, 0, base, j, c), both(sm.bias[c]));
                f2 g = pair_of(buf, 1, base, j, c);
                if (a.z) {
                    const f2 z = pair_of(buf, 2, base, j, c);
                    g = mul2(g, mul2(z, sigmoid2(z)));
                }
                const bool in0 = c < ch.count && base + j < t1, in1 = c < ch.count && base + j + 1 < t1;
                float v0, v1;
                unpack2(d, v0, v1);
                sm.delta[j][c] = in0 ? v0 : 0.f, sm.delta[j + 1][c] = in1 ? v1 : 0.f;
                unpack2(g, v0, v1);
                sm.gy[j][c] = in0 ? v0 : 0.f, sm.gy[j + 1][c] = in1 ? v1 : 0.f;
                if (!LOCAL) {
                    unpack2(pair_of(buf, LOCAL ? 0 : 3, base, j, c), v0, v1);
                    xs[j][c] = in0 ? v0 : 0.f, xs[j + 1][c] = in1 ? v1 : 0.f;
                }
            });
        }
        if (!vec_bc) {
#pragma unroll
            for (int m = 0; m < S::MB; ++m) {
                const Rows r = src_bc(m);
                for (int i = tid; i < TT * W::NP; i += W::NT) {
                    const int j = i / W::NP, n = i % W::NP;
                    sm.raw_bc[buf][m][j][n] = base + j < t1 && n < a.N ? rag_bc(buf, m, j)[r.skew(row0 + base + j) + n] : (uint16_t)0;
                }
            }
        }
    }
};

// First pass: the gradient that segment s sends back past its start when none reaches it from later segments.
template <typename T, int L, bool PACKED>
__global__ void __launch_bounds__(Bwd<L>::NT, L >= 4 ? 5 : 2) scan_bwd_local_kernel(const ScanArgs a) {
    using W = Bwd<L>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdStage<L, true> &sm = *reinterpret_cast<BwdStage<L, true> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % L, cl = lane / L;
    const int nblk = a.gblocks * a.G, segs = a.nseg - 1;
    const int blk = blockIdx.x % nblk, rest = blockIdx.x / nblk;
    const int s = rest % segs + 1, b = rest / segs;      // (nothing lies before segment 0)
    const Chans<W::CB> ch(a, blk);
    const int c0 = warp * (W::CL * 4) + cl * 4, n0 = nl * 4, nc = ch.count - c0;
    const int t0 = s * a.seglen, t1 = min(a.T, t0 + a.seglen);
    const int top = t0 + (t1 - 1 - t0) / TT * TT;
    const Tiles<T, L, true, PACKED> tiles(a, sm, &sm + 1, ch, b, t0, t1);
    tiles.fetch(top, 0);
    for (int i = tid; i < W::CB; i += W::NT) sm.bias[i] = (a.bias && i < ch.count) ? a.bias[ch.first + i] : 0.f;
    State A2, back;
    load_rates(a, ch.first + c0, nc, n0, A2);
    if (!PACKED && s == a.nseg - 1 && a.dstate_out)
        load_rows(a, a.dstate_out + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, back);
    else
        zero(back);
    f2 sum_lo = 0ull, sum_hi = 0ull;
    bool cut = false;
    __syncthreads();
    int buf = 0;
    for (int base = top; base >= t0; base -= TT, buf ^= 1) {
        tiles.fetch(base - TT, buf ^ 1);
        copies_wait<1>();
        tiles.stage(base, buf, nullptr);
        __syncthreads();
        auto tokens = [&](auto edged) {
#pragma unroll 4
        for (int j = TT - 1; j >= 0; --j) {
            if (edged.value) {
                const int n = sm.last[buf][j];
                if (n >= 0) {
                    cut = true;
                    if (a.dstate_out)
                        load_rows(a, a.dstate_out + ((long long)n * a.D + ch.first + c0) * a.N, nc, n0, back);
                    else
                        zero(back);
                }
            }
            const F2x2 d = lds_f2x2(&sm.delta[j][c0]), gy = lds_f2x2(&sm.gy[j][c0]);
            f2 cc[4];
            lds_dup4<T>(&sm.raw_bc[buf][0][j][n0], cc);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                back[n][0] = mul2(ex2x2(mul2(A2[n][0], d.lo)), fma2(gy.lo, cc[n], back[n][0]));
                back[n][1] = mul2(ex2x2(mul2(A2[n][1], d.hi)), fma2(gy.hi, cc[n], back[n][1]));
            }
            sum_lo = add2(sum_lo, d.lo);
            sum_hi = add2(sum_hi, d.hi);
        }
        };
        if (PACKED && sm.any[buf])
            tokens(Flag<PACKED>());
        else
            tokens(Flag<false>());
        __syncthreads();
    }
    copies_wait<0>();
    const long long at = (long long)b * a.nseg + s;
    store_padded(a.seg + (at * W::NP + n0) * a.DP + ch.pad + c0, a.DP, back);
    if (nl == 0) {
        ulonglong2 v;
        v.x = sum_lo, v.y = sum_hi;
        *reinterpret_cast<ulonglong2 *>(a.segdt + at * a.DP + ch.pad + c0) = v;
    }
    if (PACKED && blk == 0 && tid == 0) a.cut[s] = cut;
}

// Second pass.  2 x 4096 x 4096, N = 16, bf16: 623 us (the first pass 122).  About 390 instructions a warp and token of 32
// channels fill 47 % of the issue slots, shared memory's data path as much, with 8 warps an SM at 255 registers.  (Three
// blocks an SM, by groups of two tokens in tiles of 8, or by groups of 4 whose exponentials are taken again: 604 and
// 599 us, but twice the saved states, which cost the forward 11 and the packed form 13 to 45.)
template <typename T, int L, bool PACKED>
__global__ void __launch_bounds__(Bwd<L>::NT) scan_bwd_kernel(const ScanArgs a) {
    using W = Bwd<L>;
    constexpr int NP = W::NP, NT = W::NT;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdFull<L> &sm = *reinterpret_cast<BwdFull<L> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % L, cl = lane / L;
    const int nblk = a.gblocks * a.G;
    const int blk = blockIdx.x % nblk, rest = blockIdx.x / nblk;
    const int s = rest % a.nseg, b = rest / a.nseg;
    const Chans<W::CB> ch(a, blk);
    const int c0 = warp * (W::CL * 4) + cl * 4, n0 = nl * 4, nc = ch.count - c0;
    const int t0 = s * a.seglen, t1 = min(a.T, t0 + a.seglen);
    const int top = t0 + (t1 - 1 - t0) / TT * TT;
    const Tiles<T, L, false, PACKED> tiles(a, sm, &sm + 1, ch, b, t0, t1);
    const int vc = tiles.vc, vt = tiles.vt, vn = tiles.vn;
    if (PACKED && blockIdx.x == 0) check_cu(a.cu, a.nseq, a.T, a.err);

    // the saved state before the tile at `base`, into the last group's slot (free once that group is done)
    const float *saved = a.saved + ((long long)b * ((a.T + SAVE - 1) / SAVE) * NP + n0) * a.DP + ch.pad + c0;
    auto fetch_state = [&](int base) {
        if (base >= t0) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                copy16(sm.start[TT / SB - 1][n][tid], saved + ((long long)(base / SAVE) * NP + n) * a.DP);
        }
    };
    fetch_state(top);
    tiles.fetch(top, 0);
    for (int i = tid; i < W::CB; i += NT) sm.bias[i] = (a.bias && i < ch.count) ? a.bias[ch.first + i] : 0.f;

    f2 dbias[4] = {0ull, 0ull, 0ull, 0ull};
    State A2, back, dA;
    load_rates(a, ch.first + c0, nc, n0, A2);
    zero(dA);
    if (s < a.nseg - 1)
        load_padded(a.seg + (((long long)b * a.nseg + s + 1) * NP + n0) * a.DP + ch.pad + c0, a.DP, back);
    else if (!PACKED && a.dstate_out)
        load_rows(a, a.dstate_out + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, back);
    else
        zero(back);
    constexpr int R = LaneSum<L>::R;
    const int own = c0 + LaneSum<L>::at(nl);             // the channels whose sums end in this lane
    float skip[R], dskip[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        skip[i] = (a.skip && own + i < ch.count) ? a.skip[ch.first + own + i] : 0.f;
        dskip[i] = 0.f;
    }
    auto initial = [&](int n, State h) {  // the state that sequence n starts from
        if (a.state_in)
            load_rows(a, a.state_in + ((long long)n * a.D + ch.first + c0) * a.N, nc, n0, h);
        else
            zero(h);
    };
    __syncthreads();

    int buf = 0;
    for (int base = top; base >= t0; base -= TT, buf ^= 1) {
        copies_wait<0>();
        tiles.stage(base, buf, sm.x);
        tiles.fetch(base - TT, buf ^ 1);
        __syncthreads();
        auto tile = [&](auto edged) {
        // forward over the tile: the state before every group of SB tokens
        {
            State h;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const F2x2 v = lds_f2x2(sm.start[TT / SB - 1][n][tid]);
                h[n][0] = v.lo, h[n][1] = v.hi;
            }
#pragma unroll 1  // (the tile's code is to stay in the instruction cache)
            for (int grp = 0; grp < TT / SB; ++grp) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    *reinterpret_cast<ulonglong2 *>(sm.start[grp][n][tid]) = make_ulonglong2(h[n][0], h[n][1]);
                if (grp == TT / SB - 1) break;
#pragma unroll
                for (int i = 0; i < SB; ++i) {
                    const int j = grp * SB + i;
                    if (edged.value && sm.first[buf][j] >= 0) initial(sm.first[buf][j], h);
                    const F2x2 d = lds_f2x2(&sm.delta[j][c0]), x = lds_f2x2(&sm.x[j][c0]);
                    const f2 u_lo = mul2(d.lo, x.lo), u_hi = mul2(d.hi, x.hi);
                    f2 bb[4];
                    lds_dup4<T>(&sm.raw_bc[buf][1][j][n0], bb);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        h[n][0] = fma2(ex2x2(mul2(A2[n][0], d.lo)), h[n][0], mul2(u_lo, bb[n]));
                        h[n][1] = fma2(ex2x2(mul2(A2[n][1], d.hi)), h[n][1], mul2(u_hi, bb[n]));
                    }
                }
            }
        }
#pragma unroll 1
        for (int grp = TT / SB - 1; grp >= 0; --grp) {
            State h0, dec[SB], hs[SB];                   // state before the group; a_t and h_t of its tokens
            float yp[SB][R];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const F2x2 v = lds_f2x2(sm.start[grp][n][tid]);
                h0[n][0] = v.lo, h0[n][1] = v.hi;
            }
#pragma unroll
            for (int i = 0; i < SB; ++i) {
                const int j = grp * SB + i;
                State from;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    from[n][0] = i ? hs[i ? i - 1 : 0][n][0] : h0[n][0];
                    from[n][1] = i ? hs[i ? i - 1 : 0][n][1] : h0[n][1];
                }
                if (edged.value && sm.first[buf][j] >= 0) initial(sm.first[buf][j], from);
                const F2x2 d = lds_f2x2(&sm.delta[j][c0]), x = lds_f2x2(&sm.x[j][c0]);
                const f2 u_lo = mul2(d.lo, x.lo), u_hi = mul2(d.hi, x.hi);
                f2 y_lo = 0ull, y_hi = 0ull;
                f2 bb[4], cc[4];
                lds_dup4<T>(&sm.raw_bc[buf][1][j][n0], bb);
                lds_dup4<T>(&sm.raw_bc[buf][0][j][n0], cc);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    dec[i][n][0] = ex2x2(mul2(A2[n][0], d.lo));
                    dec[i][n][1] = ex2x2(mul2(A2[n][1], d.hi));
                    hs[i][n][0] = fma2(dec[i][n][0], from[n][0], mul2(u_lo, bb[n]));
                    hs[i][n][1] = fma2(dec[i][n][1], from[n][1], mul2(u_hi, bb[n]));
                    y_lo = fma2(hs[i][n][0], cc[n], y_lo);
                    y_hi = fma2(hs[i][n][1], cc[n], y_hi);
                }
                if (a.dz) LaneSum<L>::run(y_lo, y_hi, nl, yp[i]);
            }
            if (grp == TT / SB - 1) {  // (its slot has been read)
                fetch_state(base - TT);
                copies_commit();
            }
#pragma unroll
            for (int i = SB - 1; i >= 0; --i) {
                const int j = grp * SB + i;
                State from;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    from[n][0] = i ? hs[i ? i - 1 : 0][n][0] : h0[n][0];
                    from[n][1] = i ? hs[i ? i - 1 : 0][n][1] : h0[n][1];
                }
                if (edged.value) {
                    if (sm.first[buf][j] >= 0) initial(sm.first[buf][j], from);
                    const int n = sm.last[buf][j];
                    if (n >= 0) {
                        if (a.dstate_out)
                            load_rows(a, a.dstate_out + ((long long)n * a.D + ch.first + c0) * a.N, nc, n0, back);
                        else
                            zero(back);
                    }
                }
                const F2x2 d = lds_f2x2(&sm.delta[j][c0]), x = lds_f2x2(&sm.x[j][c0]), gy = lds_f2x2(&sm.gy[j][c0]);
                const f2 u_lo = mul2(d.lo, x.lo), u_hi = mul2(d.hi, x.hi);
                f2 s_lo = 0ull, s_hi = 0ull, q_lo = 0ull, q_hi = 0ull;
                float db[4], dc[4];
                f2 bb[4], cc[4];
                lds_dup4<T>(&sm.raw_bc[buf][1][j][n0], bb);
                lds_dup4<T>(&sm.raw_bc[buf][0][j][n0], cc);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f2 g_lo = fma2(gy.lo, cc[k], back[k][0]), g_hi = fma2(gy.hi, cc[k], back[k][1]);
                    dc[k] = sum2(fma2(gy.hi, hs[i][k][1], mul2(gy.lo, hs[i][k][0])));
                    db[k] = sum2(fma2(g_hi, u_hi, mul2(g_lo, u_lo)));
                    s_lo = fma2(g_lo, bb[k], s_lo);
                    s_hi = fma2(g_hi, bb[k], s_hi);
                    back[k][0] = mul2(g_lo, dec[i][k][0]);
                    back[k][1] = mul2(g_hi, dec[i][k][1]);
                    const f2 p_lo = mul2(back[k][0], from[k][0]), p_hi = mul2(back[k][1], from[k][1]);
                    dA[k][0] = fma2(d.lo, p_lo, dA[k][0]);
                    dA[k][1] = fma2(d.hi, p_hi, dA[k][1]);
                    q_lo = fma2(A2[k][0], p_lo, q_lo);
                    q_hi = fma2(A2[k][1], p_hi, q_hi);
                }
                // (odd channel lanes swap the two halves of their row, so that neighbouring rows use other banks)
                float *r = sm.red[warp][i & 1][cl];
                *reinterpret_cast<float4 *>(r + ((cl & 1) ? NP : 0) + n0) = make_float4(db[0], db[1], db[2], db[3]);
                *reinterpret_cast<float4 *>(r + ((cl & 1) ? 0 : NP) + n0) = make_float4(dc[0], dc[1], dc[2], dc[3]);
                float sv[R], qv[R];
                LaneSum<L>::run(s_lo, s_hi, nl, sv);
                LaneSum<L>::run(q_lo, q_hi, nl, qv);
                __syncwarp();
                if (LaneSum<L>::keeper(nl)) {
#pragma unroll
                    for (int e = 0; e < R; ++e) {
                        const float dv = sm.delta[j][own + e], xv = sm.x[j][own + e], gv = sm.gy[j][own + e];
                        sm.x[j][own + e] = fmaf(dv, sv[e], skip[e] * gv);
                        sm.delta[j][own + e] = fmaf(xv, sv[e], LN2 * qv[e]);
                        sm.gy[j][own + e] = a.dz ? fmaf(skip[e], xv, yp[i][e]) : 0.f;
                        dskip[e] = fmaf(gv, xv, dskip[e]);
                    }
                }
                if (edged.value && sm.first[buf][j] >= 0 && a.dstate_in)
                    store_rows(a, a.dstate_in + ((long long)sm.first[buf][j] * a.D + ch.first + c0) * a.N, nc, n0, back);
                if (i & 1) continue;
                // the warp's sums of dB and dC over its channel lanes, two tokens at a time: 4 columns of one a lane
                __syncwarp();
#pragma unroll
                for (int o = lane; o < 2 * 2 * NP / 4; o += 32) {
                    const int e = o / (2 * NP / 4), col = (o % (2 * NP / 4)) * 4;
                    f2 v_lo = 0ull, v_hi = 0ull;
#pragma unroll
                    for (int k = 0; k < W::CL; ++k) {
                        const F2x2 v = lds_f2x2(&sm.red[warp][e][k][(k & 1) ? (col + NP) % (2 * NP) : col]);
                        v_lo = add2(v_lo, v.lo), v_hi = add2(v_hi, v.hi);
                    }
                    *reinterpret_cast<ulonglong2 *>(&sm.bc[warp][j + e][col]) = make_ulonglong2(v_lo, v_hi);
                }
                __syncwarp();
            }
        }
        };
        if (PACKED && sm.any[buf])
            tile(Flag<PACKED>());
        else
            tile(Flag<false>());
        __syncthreads();
        // the tile's outputs
        auto through_softplus = [&](f2 v, f2 raw_dt, f2 bias) { return a.softplus ? mul2(v, sigmoid2(add2(raw_dt, bias))) : v; };
        auto through_gate = [&](f2 yp, f2 dy, f2 z) {  // yp dy sig (1 + z (1 - sig))
            const f2 sg = sigmoid2(z);
            return mul2(mul2(yp, dy), mul2(sg, fma2(z, fma2(sg, both(-1.f), both(1.f)), both(1.f))));
        };
        if (tiles.vec) {
#pragma unroll
            for (int k = 0; k < W::VPT; ++k) {
                const int j = vt + k * W::VSTEP, t = base + j;
                if (j >= TT || t >= t1 || vn <= 0) continue;
                const long long at = ((long long)b * a.T + t) * a.D + ch.first + vc;
                f2 v[4], r[4], o[4];
                get8(&sm.x[j][vc], v);
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dx) + at) = narrow8<T>(v);
                get8(&sm.delta[j][vc], v);
                widen8<T>(*reinterpret_cast<const uint4 *>(tiles.raw(buf, 0, j, true) + vc), r);
                get8(&sm.bias[vc], o);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = through_softplus(v[i], r[i], o[i]);
                    dbias[i] = add2(dbias[i], v[i]);
                }
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.ddt) + at) = narrow8<T>(v);
                if (a.dz) {
                    get8(&sm.gy[j][vc], v);
                    widen8<T>(*reinterpret_cast<const uint4 *>(tiles.raw(buf, 1, j, true) + vc), o);
                    widen8<T>(*reinterpret_cast<const uint4 *>(tiles.raw(buf, 2, j, true) + vc), r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = through_gate(v[i], o[i], r[i]);
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dz) + at) = narrow8<T>(v);
                }
            }
        } else {
            const long long at0 = ((long long)b * a.T + base) * a.D + ch.first;
            tiles.each_pair([&](int j, int c, int k) {
                const bool in0 = c < ch.count && base + j < t1, in1 = c < ch.count && base + j + 1 < t1;
                const long long p0 = at0 + (long long)j * a.D + c, p1 = p0 + a.D;
                auto put = [&](void *to, f2 v) {
                    const uint32_t w = narrow2<T>(v);
                    if (in0) static_cast<uint16_t *>(to)[p0] = (uint16_t)w;
                    if (in1) static_cast<uint16_t *>(to)[p1] = (uint16_t)(w >> 16);
                };
                put(a.dx, pack2(sm.x[j][c], sm.x[j + 1][c]));
                f2 v = through_softplus(pack2(sm.delta[j][c], sm.delta[j + 1][c]), tiles.pair_of(buf, 0, base, j, c), both(sm.bias[c]));
                put(a.ddt, v);
                float v0, v1;
                unpack2(v, v0, v1);
                dbias[k % W::NCOL * W::PL + k / W::NCOL] =
                    add2(dbias[k % W::NCOL * W::PL + k / W::NCOL], pack2(in0 ? v0 : 0.f, in1 ? v1 : 0.f));
                if (a.dz)
                    put(a.dz, through_gate(pack2(sm.gy[j][c], sm.gy[j + 1][c]), tiles.pair_of(buf, 1, base, j, c), tiles.pair_of(buf, 2, base, j, c)));
            });
        }
        for (int i = tid; i < TT * 2 * NP / 4; i += NT) {
            const int j = i / (2 * NP / 4), col = (i % (2 * NP / 4)) * 4, t = base + j;
            if (t >= t1) continue;
            f2 v_lo = 0ull, v_hi = 0ull;
#pragma unroll
            for (int w = 0; w < W::NW; ++w) {
                const F2x2 v = lds_f2x2(&sm.bc[w][j][col]);
                v_lo = add2(v_lo, v.lo), v_hi = add2(v_hi, v.hi);
            }
            const int cb = blk - ch.g * a.gblocks;
            *reinterpret_cast<ulonglong2 *>(
                a.dbc_part + (((long long)cb * a.B * a.T + (long long)b * a.T + t) * a.G + ch.g) * (2 * NP) + col) = make_ulonglong2(v_lo, v_hi);
        }
        // (what is staged next is each thread's own, or was last read before the barrier above, but for bc)
    }
    const long long part = (long long)b * a.nseg + s;
    if (!PACKED && s == 0 && a.dstate_in)
        store_rows(a, a.dstate_in + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, back);
    float *param = a.param_part + part * a.param_ld;
    store_rows(a, param + (long long)(ch.first + c0) * a.N, nc, n0, dA);
    if (a.dD_at >= 0 && LaneSum<L>::keeper(nl))
#pragma unroll
        for (int e = 0; e < R; ++e)
            if (own + e < ch.count) param[a.dD_at + ch.first + own + e] = dskip[e];
    if (a.dbias_at >= 0) {
        // the threads that share a channel, added in order
        __syncthreads();
        float *part8 = &sm.delta[0][0];
        if (tiles.vec) {
            if (vt < TT) put8(part8 + vt * W::CB + vc, dbias);
        } else {
#pragma unroll
            for (int k = 0; k < W::GROUP; ++k) {
                const int i = warp + W::NW * k, j = i / W::COLS * 2, c = i % W::COLS * 32 + lane;
                unpack2(dbias[k % W::NCOL * W::PL + k / W::NCOL], part8[j * W::CB + c], part8[(j + 1) * W::CB + c]);
            }
        }
        __syncthreads();
        for (int c = tid; c < W::CB; c += NT) {
            float v = 0.f;
            for (int k = 0; k < W::CLS; ++k) v += part8[k * W::CB + c];
            if (c < ch.count) param[a.dbias_at + ch.first + c] = v;
        }
    }
}

// dB and dC [B T, G, N] from the channel blocks' shares, in order.
template <typename T>
__global__ void __launch_bounds__(256) scan_dbc_kernel(const ScanArgs a, int NP) {
    const long long per = (long long)a.B * a.T * a.G * 2 * NP;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const int col = (int)(i % (2 * NP)), n = col % NP;
    if (n >= a.N) return;
    float v = 0.f;
    int k = 0;
    for (; k + 4 <= a.gblocks; k += 4) {
        float e[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) e[m] = a.dbc_part[(k + m) * per + i];
        v += (e[0] + e[1]) + (e[2] + e[3]);
    }
    for (; k < a.gblocks; ++k) v += a.dbc_part[k * per + i];
    static_cast<T *>(col < NP ? a.dB : a.dC)[(i / (2 * NP)) * a.N + n] = Elt<T>::from_f(v);
}

template <typename K>
cudaError_t launch_smem(K k, long long blocks, int threads, size_t smem, cudaStream_t s, const ScanArgs &a) {
    const cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
    return launch_plain(k, dim3((unsigned)blocks), dim3(threads), smem, s, a);
}
template <typename T, int L>
cudaError_t launch_l(const ScanArgs &a, bool full, cudaStream_t s) {
    const long long blocks = (long long)a.gblocks * a.G * (full ? a.nseg : a.nseg - 1) * a.B;
    const size_t full_smem = sizeof(BwdFull<L>) + raw_bytes<L, false>(a.vec, a.vec_bc);
    if (full)
        return a.cu ? launch_smem(scan_bwd_kernel<T, L, true>, blocks, Bwd<L>::NT, full_smem, s, a)
                    : launch_smem(scan_bwd_kernel<T, L, false>, blocks, Bwd<L>::NT, full_smem, s, a);
    const size_t smem = sizeof(BwdStage<L, true>) + raw_bytes<L, true>(a.vec, a.vec_bc);
    return a.cu ? launch_smem(scan_bwd_local_kernel<T, L, true>, blocks, Bwd<L>::NT, smem, s, a)
                : launch_smem(scan_bwd_local_kernel<T, L, false>, blocks, Bwd<L>::NT, smem, s, a);
}
template <typename T>
cudaError_t launch_t(const ScanArgs &a, int L, bool full, cudaStream_t s) {
    switch (L) {
        case 1: return launch_l<T, 1>(a, full, s);
        case 2: return launch_l<T, 2>(a, full, s);
        case 4: return launch_l<T, 4>(a, full, s);
        case 8: return launch_l<T, 8>(a, full, s);
        default: return launch_l<T, 16>(a, full, s);
    }
}

}  // namespace
}  // namespace scan
}  // namespace gdr
