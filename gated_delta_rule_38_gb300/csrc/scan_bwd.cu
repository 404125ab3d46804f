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
};

template <int L>
struct BwdSmem {
    float delta[TT][Bwd<L>::CB];                         // then the gradient of delta
    float x[TT][Bwd<L>::CB];                             // then dx
    float gy[TT][Bwd<L>::CB];                            // then yp
    float b[TT][Bwd<L>::NP][2];
    float c[TT][Bwd<L>::NP][2];
    float start[TT / SB][4][Bwd<L>::NT][4];              // the state before every group: thread-private
    float red[Bwd<L>::NW][SB][Bwd<L>::CL][2 * Bwd<L>::NP];
    float bc[Bwd<L>::NW][TT][2 * Bwd<L>::NP];            // a warp's sums of dB | dC
    int first[TT], last[TT];
};

// Stages x, delta and gy of the tile at `base` (LOCAL: without x, and C without B).
template <typename T, int L, bool LOCAL>
__device__ __forceinline__ void stage(const ScanArgs &a, BwdSmem<L> &sm, const Chans<Bwd<L>::CB> &ch, int b, int base, int t1,
                                      int vc, int vt, int vn, bool vlive, const float *bias) {
    using W = Bwd<L>;
    constexpr int VSTEP = W::NT / (W::CB / 8);
    const int tid = threadIdx.x;
#pragma unroll
    for (int k = 0; k < W::VPT; ++k) {
        const int j = vt + k * VSTEP, t = base + j;
        if (!vlive) break;
        const bool in = t < t1 && vn > 0;
        const long long row = (long long)b * a.T + t;
        const int c = ch.first + vc;
        uint4 rx = make_uint4(0, 0, 0, 0), rd = rx, rz = rx, rg = rx;
        if (in) {
            rd = load8(static_cast<const uint16_t *>(a.dt) + row * a.dt_ld + c, vn, a.vec);
            rg = load8(static_cast<const uint16_t *>(a.dy) + row * a.D + c, vn, a.vec);
            if (!LOCAL) rx = load8(static_cast<const uint16_t *>(a.x) + row * a.x_ld + c, vn, a.vec);
            if (a.z) rz = load8(static_cast<const uint16_t *>(a.z) + row * a.z_ld + c, vn, a.vec);
        }
        float d[8], g[8], v[8];
        widen8<T>(rd, d);
        widen8<T>(rg, g);
        widen8<T>(rz, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d[i] += bias[i];
            if (a.softplus) d[i] = softplus(d[i]);
            d[i] = in && i < vn ? d[i] : 0.f;
            if (a.z) g[i] *= v[i] * sigmoid(v[i]);
            g[i] = in && i < vn ? g[i] : 0.f;
        }
        put8(&sm.delta[j][vc], d);
        put8(&sm.gy[j][vc], g);
        if (!LOCAL) {
            widen8<T>(rx, v);
            put8(&sm.x[j][vc], v);
        }
    }
    for (int i = tid; i < TT * W::NP; i += W::NT) {
        const int j = i / W::NP, n = i % W::NP, t = base + j;
        float vb = 0.f, vcx = 0.f;
        if (t < t1 && n < a.N) {
            const long long row = (long long)b * a.T + t;
            if (!LOCAL) vb = Elt<T>::to_f(static_cast<const T *>(a.Bm)[row * a.b_ld + ch.g * a.N + n]);
            vcx = Elt<T>::to_f(static_cast<const T *>(a.Cm)[row * a.c_ld + ch.g * a.N + n]);
        }
        if (!LOCAL) *reinterpret_cast<float2 *>(sm.b[j][n]) = make_float2(vb, vb);
        *reinterpret_cast<float2 *>(sm.c[j][n]) = make_float2(vcx, vcx);
    }
}

// First pass: the gradient that segment s sends back past its start when none reaches it from later segments.
template <typename T, int L, bool PACKED>
__global__ void __launch_bounds__(Bwd<L>::NT) scan_bwd_local_kernel(const ScanArgs a) {
    using W = Bwd<L>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<L> &sm = *reinterpret_cast<BwdSmem<L> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % L, cl = lane / L;
    const int nblk = a.gblocks * a.G, segs = a.nseg - 1;
    const int blk = blockIdx.x % nblk, rest = blockIdx.x / nblk;
    const int s = rest % segs + 1, b = rest / segs;      // (nothing lies before segment 0)
    const Chans<W::CB> ch(a, blk);
    const int c0 = warp * (W::CL * 4) + cl * 4, n0 = nl * 4, nc = ch.count - c0;
    const int t0 = s * a.seglen, t1 = min(a.T, t0 + a.seglen);
    constexpr int VROW = W::CB / 8;
    const int vc = (tid % VROW) * 8, vt = tid / VROW, vn = ch.count - vc;
    const bool vlive = W::NVEC >= W::NT || tid < W::NVEC;
    float bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = (a.bias && i < vn) ? a.bias[ch.first + vc + i] : 0.f;
    State A2, back;
    load_rows(a, a.A + (long long)(ch.first + c0) * a.N, nc, n0, A2, LOG2E);
    if (!PACKED && s == a.nseg - 1 && a.dstate_out)
        load_rows(a, a.dstate_out + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, back);
    else
        zero(back);
    f2 sum_lo = 0ull, sum_hi = 0ull;
    bool cut = false;
    for (int base = t0 + (t1 - 1 - t0) / TT * TT; base >= t0; base -= TT) {
        stage<T, L, true>(a, sm, ch, b, base, t1, vc, vt, vn, vlive, bias);
        if (PACKED)
            for (int j = tid; j < TT; j += W::NT) edges(a, base + j, t1, sm.first[j], sm.last[j]);
        __syncthreads();
#pragma unroll 4
        for (int j = TT - 1; j >= 0; --j) {
            if (PACKED) {
                const int n = sm.last[j];
                if (n >= 0) {
                    cut = true;
                    if (a.dstate_out)
                        load_rows(a, a.dstate_out + ((long long)n * a.D + ch.first + c0) * a.N, nc, n0, back);
                    else
                        zero(back);
                }
            }
            const F2x2 d = lds_f2x2(&sm.delta[j][c0]), gy = lds_f2x2(&sm.gy[j][c0]);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                const F2x2 cc = lds_f2x2(sm.c[j][n0 + n]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const f2 cn = m ? cc.hi : cc.lo;
                    f2 *k = back[n + m];
                    k[0] = mul2(exp2x2(mul2(A2[n + m][0], d.lo)), fma2(gy.lo, cn, k[0]));
                    k[1] = mul2(exp2x2(mul2(A2[n + m][1], d.hi)), fma2(gy.hi, cn, k[1]));
                }
            }
            sum_lo = add2(sum_lo, d.lo);
            sum_hi = add2(sum_hi, d.hi);
        }
        __syncthreads();
    }
    const long long at = (long long)b * a.nseg + s;
    store_padded(a.seg + (at * W::NP + n0) * a.DP + ch.pad + c0, a.DP, back);
    if (nl == 0) {
        ulonglong2 v;
        v.x = sum_lo, v.y = sum_hi;
        *reinterpret_cast<ulonglong2 *>(a.segdt + at * a.DP + ch.pad + c0) = v;
    }
    if (PACKED && blk == 0 && tid == 0) a.cut[s] = cut;
}

// A thread's gradients of its states of one token: h, a and the state before, 16 elements each.
template <typename T, int L, bool PACKED>
__global__ void __launch_bounds__(Bwd<L>::NT) scan_bwd_kernel(const ScanArgs a) {
    using W = Bwd<L>;
    constexpr int NP = W::NP, NT = W::NT, VROW = W::CB / 8, VSTEP = NT / VROW;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<L> &sm = *reinterpret_cast<BwdSmem<L> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % L, cl = lane / L;
    const int nblk = a.gblocks * a.G;
    const int blk = blockIdx.x % nblk, rest = blockIdx.x / nblk;
    const int s = rest % a.nseg, b = rest / a.nseg;
    const Chans<W::CB> ch(a, blk);
    const int c0 = warp * (W::CL * 4) + cl * 4, n0 = nl * 4, nc = ch.count - c0;
    const int t0 = s * a.seglen, t1 = min(a.T, t0 + a.seglen);
    const int vc = (tid % VROW) * 8, vt = tid / VROW, vn = ch.count - vc;
    const bool vlive = W::NVEC >= NT || tid < W::NVEC;
    if (PACKED && blockIdx.x == 0) check_cu(a.cu, a.nseq, a.T, a.err);

    float bias[8], dbias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bias[i] = (a.bias && i < vn) ? a.bias[ch.first + vc + i] : 0.f;
        dbias[i] = 0.f;
    }
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
    const long long chunks = (a.T + SAVE - 1) / SAVE;

    for (int base = t0 + (t1 - 1 - t0) / TT * TT; base >= t0; base -= TT) {
        stage<T, L, false>(a, sm, ch, b, base, t1, vc, vt, vn, vlive, bias);
        if (PACKED)
            for (int j = tid; j < TT; j += NT) edges(a, base + j, t1, sm.first[j], sm.last[j]);
        __syncthreads();
        // forward over the tile: the state before every group of SB tokens
        {
            State h;
            load_padded(a.saved + (((long long)b * chunks + base / SAVE) * NP + n0) * a.DP + ch.pad + c0, a.DP, h);
            for (int grp = 0; grp < TT / SB; ++grp) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    ulonglong2 v;
                    v.x = h[n][0], v.y = h[n][1];
                    *reinterpret_cast<ulonglong2 *>(sm.start[grp][n][tid]) = v;
                }
                if (grp == TT / SB - 1) break;
#pragma unroll
                for (int i = 0; i < SB; ++i) {
                    const int j = grp * SB + i;
                    if (PACKED && sm.first[j] >= 0) {
                        if (a.state_in)
                            load_rows(a, a.state_in + ((long long)sm.first[j] * a.D + ch.first + c0) * a.N, nc, n0, h);
                        else
                            zero(h);
                    }
                    const F2x2 d = lds_f2x2(&sm.delta[j][c0]), x = lds_f2x2(&sm.x[j][c0]);
                    const f2 u_lo = mul2(d.lo, x.lo), u_hi = mul2(d.hi, x.hi);
#pragma unroll
                    for (int n = 0; n < 4; n += 2) {
                        const F2x2 bb = lds_f2x2(sm.b[j][n0 + n]);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const f2 bn = m ? bb.hi : bb.lo;
                            f2 *hn = h[n + m];
                            hn[0] = fma2(exp2x2(mul2(A2[n + m][0], d.lo)), hn[0], mul2(u_lo, bn));
                            hn[1] = fma2(exp2x2(mul2(A2[n + m][1], d.hi)), hn[1], mul2(u_hi, bn));
                        }
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
                if (PACKED && sm.first[j] >= 0) {
                    if (a.state_in)
                        load_rows(a, a.state_in + ((long long)sm.first[j] * a.D + ch.first + c0) * a.N, nc, n0, from);
                    else
                        zero(from);
                }
                const F2x2 d = lds_f2x2(&sm.delta[j][c0]), x = lds_f2x2(&sm.x[j][c0]);
                const f2 u_lo = mul2(d.lo, x.lo), u_hi = mul2(d.hi, x.hi);
                f2 y_lo = 0ull, y_hi = 0ull;
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
                    const F2x2 bb = lds_f2x2(sm.b[j][n0 + n]), cc = lds_f2x2(sm.c[j][n0 + n]);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const f2 bn = m ? bb.hi : bb.lo, cn = m ? cc.hi : cc.lo;
                        dec[i][n + m][0] = exp2x2(mul2(A2[n + m][0], d.lo));
                        dec[i][n + m][1] = exp2x2(mul2(A2[n + m][1], d.hi));
                        hs[i][n + m][0] = fma2(dec[i][n + m][0], from[n + m][0], mul2(u_lo, bn));
                        hs[i][n + m][1] = fma2(dec[i][n + m][1], from[n + m][1], mul2(u_hi, bn));
                        y_lo = fma2(hs[i][n + m][0], cn, y_lo);
                        y_hi = fma2(hs[i][n + m][1], cn, y_hi);
                    }
                }
                if (a.dz) LaneSum<L>::run(y_lo, y_hi, nl, yp[i]);
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
                    if (sm.first[j] >= 0) {
                        if (a.state_in)
                            load_rows(a, a.state_in + ((long long)sm.first[j] * a.D + ch.first + c0) * a.N, nc, n0, from);
                        else
                            zero(from);
                    }
                    if (sm.last[j] >= 0) {
                        if (a.dstate_out)
                            load_rows(a, a.dstate_out + ((long long)sm.last[j] * a.D + ch.first + c0) * a.N, nc, n0, back);
                        else
                            zero(back);
                    }
                }
                const F2x2 d = lds_f2x2(&sm.delta[j][c0]), x = lds_f2x2(&sm.x[j][c0]), gy = lds_f2x2(&sm.gy[j][c0]);
                const f2 u_lo = mul2(d.lo, x.lo), u_hi = mul2(d.hi, x.hi);
                f2 s_lo = 0ull, s_hi = 0ull, q_lo = 0ull, q_hi = 0ull;
                float db[4], dc[4];
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
                    const F2x2 bb = lds_f2x2(sm.b[j][n0 + n]), cc = lds_f2x2(sm.c[j][n0 + n]);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int k = n + m;
                        const f2 bn = m ? bb.hi : bb.lo, cn = m ? cc.hi : cc.lo;
                        const f2 g_lo = fma2(gy.lo, cn, back[k][0]), g_hi = fma2(gy.hi, cn, back[k][1]);
                        dc[k] = sum2(fma2(gy.hi, hs[i][k][1], mul2(gy.lo, hs[i][k][0])));
                        db[k] = sum2(fma2(g_hi, u_hi, mul2(g_lo, u_lo)));
                        s_lo = fma2(g_lo, bn, s_lo);
                        s_hi = fma2(g_hi, bn, s_hi);
                        back[k][0] = mul2(g_lo, dec[i][k][0]);
                        back[k][1] = mul2(g_hi, dec[i][k][1]);
                        const f2 p_lo = mul2(back[k][0], from[k][0]), p_hi = mul2(back[k][1], from[k][1]);
                        dA[k][0] = fma2(d.lo, p_lo, dA[k][0]);
                        dA[k][1] = fma2(d.hi, p_hi, dA[k][1]);
                        q_lo = fma2(A2[k][0], p_lo, q_lo);
                        q_hi = fma2(A2[k][1], p_hi, q_hi);
                    }
                }
                // (odd channel lanes swap the two halves of their row, so that neighbouring rows use other banks)
                float *r = sm.red[warp][i][cl];
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
                if (PACKED && sm.first[j] >= 0 && a.dstate_in)
                    store_rows(a, a.dstate_in + ((long long)sm.first[j] * a.D + ch.first + c0) * a.N, nc, n0, back);
            }
            __syncwarp();
            // the warp's sums of dB and dC over its channel lanes: 4 columns of one token a lane
#pragma unroll
            for (int o = lane; o < SB * 2 * NP / 4; o += 32) {
                const int i = o / (2 * NP / 4), col = (o % (2 * NP / 4)) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < W::CL; ++k) {
                    const float4 e = *reinterpret_cast<const float4 *>(&sm.red[warp][i][k][(k & 1) ? (col + NP) % (2 * NP) : col]);
                    v.x += e.x, v.y += e.y, v.z += e.z, v.w += e.w;
                }
                *reinterpret_cast<float4 *>(&sm.bc[warp][grp * SB + i][col]) = v;
            }
            __syncwarp();
        }
        __syncthreads();
        // the tile's outputs
#pragma unroll
        for (int k = 0; k < W::VPT; ++k) {
            const int j = vt + k * VSTEP, t = base + j;
            if (!vlive || t >= t1 || vn <= 0) continue;
            const long long row = (long long)b * a.T + t;
            const int c = ch.first + vc;
            const long long at = row * a.D + c;
            float v[8], r[8], o[8];
            get8(&sm.x[j][vc], v);
            store8(static_cast<uint16_t *>(a.dx) + at, narrow8<T>(v), vn, a.vec);
            get8(&sm.delta[j][vc], v);
            if (a.softplus) {
                widen8<T>(load8(static_cast<const uint16_t *>(a.dt) + row * a.dt_ld + c, vn, a.vec), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= sigmoid(r[i] + bias[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) dbias[i] += v[i];
            store8(static_cast<uint16_t *>(a.ddt) + at, narrow8<T>(v), vn, a.vec);
            if (a.dz) {
                get8(&sm.gy[j][vc], v);
                widen8<T>(load8(static_cast<const uint16_t *>(a.z) + row * a.z_ld + c, vn, a.vec), r);
                widen8<T>(load8(static_cast<const uint16_t *>(a.dy) + at, vn, a.vec), o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float sg = sigmoid(r[i]);
                    v[i] = o[i] * v[i] * sg * fmaf(r[i], 1.f - sg, 1.f);
                }
                store8(static_cast<uint16_t *>(a.dz) + at, narrow8<T>(v), vn, a.vec);
            }
        }
        for (int i = tid; i < TT * 2 * NP; i += NT) {
            const int j = i / (2 * NP), col = i % (2 * NP), t = base + j;
            if (t >= t1) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < W::NW; ++w) v += sm.bc[w][j][col];
            const int cb = blk - ch.g * a.gblocks;
            a.dbc_part[(((long long)cb * a.B * a.T + (long long)b * a.T + t) * a.G + ch.g) * (2 * NP) + col] = v;
        }
        __syncthreads();
    }
    const long long part = (long long)b * a.nseg + s;
    if (!PACKED && s == 0 && a.dstate_in)
        store_rows(a, a.dstate_in + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, back);
    store_rows(a, a.dA_part + (part * a.D + ch.first + c0) * a.N, nc, n0, dA);
    if (a.dD_part && LaneSum<L>::keeper(nl))
#pragma unroll
        for (int e = 0; e < R; ++e)
            if (own + e < ch.count) a.dD_part[part * a.D + ch.first + own + e] = dskip[e];
    if (a.dbias_part) {
        // threads of one vector column, added in order
        float *buf = &sm.delta[0][0];                    // NT x 8 floats: NT <= TT CB / 8
        if (vlive) put8(buf + tid * 8, dbias);
        __syncthreads();
        for (int c = tid; c < W::CB; c += NT) {
            float v = 0.f;
            for (int k = c / 8; k < (W::NVEC < NT ? W::NVEC : NT); k += VROW) v += buf[k * 8 + c % 8];
            if (c < ch.count) a.dbias_part[part * a.D + ch.first + c] = v;
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
    const size_t smem = sizeof(BwdSmem<L>);
    if (full)
        return a.cu ? launch_smem(scan_bwd_kernel<T, L, true>, blocks, Bwd<L>::NT, smem, s, a)
                    : launch_smem(scan_bwd_kernel<T, L, false>, blocks, Bwd<L>::NT, smem, s, a);
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
