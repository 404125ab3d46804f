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
    static constexpr int BROW = NP / BW, BSTEP = NT / BROW;
    static constexpr int BPT = TT > BSTEP ? TT / BSTEP : 1;
};

// The raw tiles (two of each: the next one is on its way while one is worked on) are private to the threads that copy
// them, the states before the groups to the threads that own the states.
template <int L, bool LOCAL>
struct BwdSmem {
    using W = Bwd<L>;
    uint16_t raw[2][LOCAL ? 3 : 4][TT][W::CB];           // dt, dy, z, x
    uint16_t raw_bc[2][LOCAL ? 1 : 2][TT][W::NP];        // C, B
    float delta[TT][W::CB];                              // then the gradient of delta
    float gy[TT][W::CB];                                 // then yp
    float bias[W::CB];
    int first[2][TT], last[2][TT];
};
template <int L>
struct BwdFull : BwdSmem<L, false> {
    using W = Bwd<L>;
    float x[TT][W::CB];                                  // then dx
    float start[TT / SB][4][W::NT][4];                   // the state before every group: thread-private
    float red[W::NW][2][W::CL][2 * W::NP];               // two tokens' dB | dC of a warp's channel lanes
    float bc[W::NW][TT][2 * W::NP];                      // a warp's sums of dB | dC
};

// The copies of the tile at `base` into buffer `buf`.
template <int L, bool LOCAL, bool PACKED>
__device__ __forceinline__ void fetch(const ScanArgs &a, BwdSmem<L, LOCAL> &sm, const Chans<Bwd<L>::CB> &ch, int b, int base,
                                      int t0, int t1, int buf) {
    using W = Bwd<L>;
    const int tid = threadIdx.x, vc = (tid % W::VROW) * 8, vt = tid / W::VROW, vn = ch.count - vc;
    const int bn = (tid % W::BROW) * 8, bt = tid / W::BROW;
    if (base >= t0) {
#pragma unroll
        for (int k = 0; k < W::VPT; ++k) {
            const int j = vt + k * W::VSTEP, t = base + j;
            if (j < TT && t < t1 && vn > 0) {
                const long long row = (long long)b * a.T + t;
                const int c = ch.first + vc;
                copy8(&sm.raw[buf][0][j][vc], static_cast<const uint16_t *>(a.dt) + row * a.dt_ld + c, vn, a.vec);
                copy8(&sm.raw[buf][1][j][vc], static_cast<const uint16_t *>(a.dy) + row * a.D + c, vn, a.vec);
                if (a.z) copy8(&sm.raw[buf][2][j][vc], static_cast<const uint16_t *>(a.z) + row * a.z_ld + c, vn, a.vec);
                if (!LOCAL) copy8(&sm.raw[buf][LOCAL ? 0 : 3][j][vc], static_cast<const uint16_t *>(a.x) + row * a.x_ld + c, vn, a.vec);
            }
        }
#pragma unroll
        for (int k = 0; k < W::BPT; ++k) {
            const int j = bt + k * W::BSTEP, t = base + j;
            if (j >= TT) break;
            if (t < t1) {
                const long long row = (long long)b * a.T + t;
                const uint16_t *pc = static_cast<const uint16_t *>(a.Cm) + row * a.c_ld + ch.g * a.N + bn;
                const uint16_t *pb = static_cast<const uint16_t *>(a.Bm) + row * a.b_ld + ch.g * a.N + bn;
                if constexpr (W::BW == 8) {
                    copy8(&sm.raw_bc[buf][0][j][bn], pc, a.N - bn, a.vec_bc);
                    if (!LOCAL) copy8(&sm.raw_bc[buf][LOCAL ? 0 : 1][j][bn], pb, a.N - bn, a.vec_bc);
                } else {
                    for (int n = 0; n < W::BW; ++n) {
                        sm.raw_bc[buf][0][j][n] = n < a.N ? pc[n] : (uint16_t)0;
                        if (!LOCAL) sm.raw_bc[buf][LOCAL ? 0 : 1][j][n] = n < a.N ? pb[n] : (uint16_t)0;
                    }
                }
            } else {  // past the end: zeros
                for (int n = 0; n < W::BW; n += 4) {
                    *reinterpret_cast<uint2 *>(&sm.raw_bc[buf][0][j][bn + n]) = make_uint2(0, 0);
                    if (!LOCAL) *reinterpret_cast<uint2 *>(&sm.raw_bc[buf][LOCAL ? 0 : 1][j][bn + n]) = make_uint2(0, 0);
                }
            }
        }
        if (PACKED)
            for (int j = tid; j < TT; j += W::NT) edges(a, base + j, t1, sm.first[buf][j], sm.last[buf][j]);
    }
    copies_commit();
}

// delta and gy of the tile that has arrived in `buf` (and through `xb` what the full pass adds).
template <typename T, int L, bool LOCAL, typename F>
__device__ __forceinline__ void stage(const ScanArgs &a, BwdSmem<L, LOCAL> &sm, const Chans<Bwd<L>::CB> &ch, int base, int t1,
                                      int buf, F &&xb) {
    using W = Bwd<L>;
    const int tid = threadIdx.x, vc = (tid % W::VROW) * 8, vt = tid / W::VROW, vn = ch.count - vc;
#pragma unroll
    for (int k = 0; k < W::VPT; ++k) {
        const int j = vt + k * W::VSTEP;
        if (j >= TT) break;
        f2 d[4], g[4], v[4];
        const bool in = base + j < t1 && vn > 0;
        if (in) {
            widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][0][j][vc]), d);
            widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][1][j][vc]), g);
            get8(&sm.bias[vc], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                d[i] = add2(d[i], v[i]);
                if (a.softplus) d[i] = softplus2(d[i]);
            }
            if (a.z) {
                widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][2][j][vc]), v);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], mul2(v[i], sigmoid2(v[i])));
            }
        } else {  // past the end: a step of zero and no gradient
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = g[i] = 0ull;
        }
        put8(&sm.delta[j][vc], d);
        put8(&sm.gy[j][vc], g);
        xb(j, vc, in);
    }
}

// First pass: the gradient that segment s sends back past its start when none reaches it from later segments.
template <typename T, int L, bool PACKED>
__global__ void __launch_bounds__(Bwd<L>::NT, L >= 4 ? 5 : 2) scan_bwd_local_kernel(const ScanArgs a) {
    using W = Bwd<L>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<L, true> &sm = *reinterpret_cast<BwdSmem<L, true> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % L, cl = lane / L;
    const int nblk = a.gblocks * a.G, segs = a.nseg - 1;
    const int blk = blockIdx.x % nblk, rest = blockIdx.x / nblk;
    const int s = rest % segs + 1, b = rest / segs;      // (nothing lies before segment 0)
    const Chans<W::CB> ch(a, blk);
    const int c0 = warp * (W::CL * 4) + cl * 4, n0 = nl * 4, nc = ch.count - c0;
    const int t0 = s * a.seglen, t1 = min(a.T, t0 + a.seglen);
    const int top = t0 + (t1 - 1 - t0) / TT * TT;
    fetch<L, true, PACKED>(a, sm, ch, b, top, t0, t1, 0);
    for (int i = tid; i < W::CB; i += W::NT) sm.bias[i] = (a.bias && i < ch.count) ? a.bias[ch.first + i] : 0.f;
    State A2, back;
    load_rows(a, a.A + (long long)(ch.first + c0) * a.N, nc, n0, A2, LOG2E);
    if (!PACKED && s == a.nseg - 1 && a.dstate_out)
        load_rows(a, a.dstate_out + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, back);
    else
        zero(back);
    f2 sum_lo = 0ull, sum_hi = 0ull;
    bool cut = false;
    __syncthreads();
    int buf = 0;
    for (int base = top; base >= t0; base -= TT, buf ^= 1) {
        fetch<L, true, PACKED>(a, sm, ch, b, base - TT, t0, t1, buf ^ 1);
        copies_wait<1>();
        stage<T, L, true>(a, sm, ch, base, t1, buf, [](int, int, bool) {});
        __syncthreads();
#pragma unroll 4
        for (int j = TT - 1; j >= 0; --j) {
            if (PACKED) {
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
    const int vc = (tid % W::VROW) * 8, vt = tid / W::VROW, vn = ch.count - vc;
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
    fetch<L, false, PACKED>(a, sm, ch, b, top, t0, t1, 0);
    for (int i = tid; i < W::CB; i += NT) sm.bias[i] = (a.bias && i < ch.count) ? a.bias[ch.first + i] : 0.f;

    f2 dbias[4] = {0ull, 0ull, 0ull, 0ull};
    State A2, back, dA;
    load_rows(a, a.A + (long long)(ch.first + c0) * a.N, nc, n0, A2, LOG2E);
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
        stage<T, L, false>(a, sm, ch, base, t1, buf, [&](int j, int c, bool in) {
            f2 x[4] = {0ull, 0ull, 0ull, 0ull};
            if (in) widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][3][j][c]), x);
            put8(&sm.x[j][c], x);
        });
        fetch<L, false, PACKED>(a, sm, ch, b, base - TT, t0, t1, buf ^ 1);
        __syncthreads();
        // forward over the tile: the state before every group of SB tokens
        {
            State h;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const F2x2 v = lds_f2x2(sm.start[TT / SB - 1][n][tid]);
                h[n][0] = v.lo, h[n][1] = v.hi;
            }
            for (int grp = 0; grp < TT / SB; ++grp) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    *reinterpret_cast<ulonglong2 *>(sm.start[grp][n][tid]) = make_ulonglong2(h[n][0], h[n][1]);
                if (grp == TT / SB - 1) break;
#pragma unroll
                for (int i = 0; i < SB; ++i) {
                    const int j = grp * SB + i;
                    if (PACKED && sm.first[buf][j] >= 0) initial(sm.first[buf][j], h);
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
                if (PACKED && sm.first[buf][j] >= 0) initial(sm.first[buf][j], from);
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
                if (PACKED) {
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
                if (PACKED && sm.first[buf][j] >= 0 && a.dstate_in)
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
        __syncthreads();
        // the tile's outputs
#pragma unroll
        for (int k = 0; k < W::VPT; ++k) {
            const int j = vt + k * W::VSTEP, t = base + j;
            if (j >= TT || t >= t1 || vn <= 0) continue;
            const long long at = ((long long)b * a.T + t) * a.D + ch.first + vc;
            f2 v[4], r[4], o[4];
            get8(&sm.x[j][vc], v);
            store8(static_cast<uint16_t *>(a.dx) + at, narrow8<T>(v), vn, a.vec);
            get8(&sm.delta[j][vc], v);
            if (a.softplus) {
                widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][0][j][vc]), r);
                get8(&sm.bias[vc], o);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], sigmoid2(add2(r[i], o[i])));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) dbias[i] = add2(dbias[i], v[i]);
            store8(static_cast<uint16_t *>(a.ddt) + at, narrow8<T>(v), vn, a.vec);
            if (a.dz) {
                get8(&sm.gy[j][vc], v);
                widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][1][j][vc]), o);
                widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][2][j][vc]), r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2 sg = sigmoid2(r[i]);  // yp dy sig (1 + z (1 - sig))
                    v[i] = mul2(mul2(v[i], o[i]), mul2(sg, fma2(r[i], fma2(sg, both(-1.f), both(1.f)), both(1.f))));
                }
                store8(static_cast<uint16_t *>(a.dz) + at, narrow8<T>(v), vn, a.vec);
            }
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
        // threads of one vector column, added in order
        __syncthreads();
        float *buf8 = &sm.delta[0][0];                   // 8 floats of each thread that holds vectors
        if (vt < TT) put8(buf8 + tid * 8, dbias);
        __syncthreads();
        for (int c = tid; c < W::CB; c += NT) {
            float v = 0.f;
            for (int k = c / 8; k < (W::NVEC < NT ? W::NVEC : NT); k += W::VROW) v += buf8[k * 8 + c % 8];
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
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_plain(k, dim3((unsigned)blocks), dim3(threads), smem, s, a);
}
template <typename T, int L>
cudaError_t launch_l(const ScanArgs &a, bool full, cudaStream_t s) {
    const long long blocks = (long long)a.gblocks * a.G * (full ? a.nseg : a.nseg - 1) * a.B;
    if (full)
        return a.cu ? launch_smem(scan_bwd_kernel<T, L, true>, blocks, Bwd<L>::NT, sizeof(BwdFull<L>), s, a)
                    : launch_smem(scan_bwd_kernel<T, L, false>, blocks, Bwd<L>::NT, sizeof(BwdFull<L>), s, a);
    const size_t smem = sizeof(BwdSmem<L, true>);
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

cudaError_t launch_scan_bwd(const ScanArgs &a, int L, bool bf16, bool full, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(a, L, full, s) : launch_t<__half>(a, L, full, s);
}

cudaError_t launch_scan_dbc(const ScanArgs &a, int L, bool bf16, cudaStream_t s) {
    const long long blocks = ((long long)a.B * a.T * a.G * 8 * L + 255) / 256;
    if (bf16) return launch_plain(scan_dbc_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(256), 0, s, a, 4 * L);
    return launch_plain(scan_dbc_kernel<__half>, dim3((unsigned)blocks), dim3(256), 0, s, a, 4 * L);
}

}  // namespace scan
}  // namespace gdr
