// Forward of the selective state space scan (per channel d, N states; delta = softplus(dt + bias) or dt + bias):
//
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,   y_t = (C_t . h_t + D x_t) silu(z_t)
//
// The work is N exponentials and about 4 N fp32 operations a token and channel against 8 bytes of traffic, so at
// N = 16 the kernels are bound by the special-function and fp32 pipes, not by HBM (this chip does 32 ex2 and 128 fp32
// lanes a clock and SM: at least 4 clocks a quarter-SM for 32 (t, d, n) elements on either pipe).
//
// A block walks a segment of one row's tokens for a block of channels: it stages tiles of tokens in shared memory
// (steps and inputs in fp32, each (token, channel) converted once, loads of the next tile in flight), runs the
// recurrence with all states in registers, and writes the tile's outputs as whole vectors.  When rows x channel
// blocks do not fill the chip the token axis is cut into segments: a first pass leaves every segment's end state from
// a zero start and its sum of delta, a scan over the segments joins them (a segment multiplies its start state by
// exp(A sum delta)), and the second pass starts from the joined states.
#include "scan.cuh"

namespace gdr {
namespace scan {
namespace {

template <int L>
struct Fwd {
    static constexpr int NP = 4 * L;                    // padded states
    static constexpr int CB = 512 / L;                  // channels a block
    static constexpr int TT = L >= 4 ? 16 : 4 * L;      // tokens a tile
    static constexpr int NVEC = TT * CB / 8;            // 8-channel vectors of a tile
    static constexpr int VPT = NVEC > 128 ? NVEC / 128 : 1;
    static constexpr int BVEC = TT * NP / 8;            // 8-state vectors of a tile's B
    static constexpr int BPT = BVEC > 128 ? BVEC / 128 : 1;
};

// The raw tiles (two of each: the next one is on its way while one is worked on) are private to the threads that copy
// them, but for B and C; so are, but for the recurrence in between, the staged elements of a vector.
template <int L, bool FULL>
struct FwdSmem {
    using F = Fwd<L>;
    uint16_t raw[2][FULL ? 3 : 2][F::TT][F::CB];        // dt, x, z
    uint16_t raw_bc[2][FULL ? 2 : 1][F::TT][F::NP];
    float delta[F::TT][F::CB];
    float u[F::TT][F::CB];                              // delta x; then the output of the recurrence
    float bias[F::CB], skip[F::CB];
    int first[2][F::TT], last[2][F::TT];
};

// FULL: the outputs (second pass, or the only one).  Otherwise the first pass over segments.
template <typename T, int L, bool FULL, bool PACKED>
__global__ void __launch_bounds__(128, FULL ? 5 : 6) scan_fwd_kernel(const ScanArgs a) {
    using F = Fwd<L>;
    constexpr int CB = F::CB, TT = F::TT, NP = F::NP;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    FwdSmem<L, FULL> &sm = *reinterpret_cast<FwdSmem<L, FULL> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nl = lane % L, cl = lane / L;
    const int segs = FULL ? a.nseg : a.nseg - 1;        // (the last segment's end state joins nothing)
    const int nblk = a.gblocks * a.G;
    const int blk = blockIdx.x % nblk, rest = blockIdx.x / nblk;
    const int s = rest % segs, b = rest / segs;
    const Chans<CB> ch(a, blk);
    const int c0 = warp * (128 / L) + cl * 4, n0 = nl * 4;  // this thread's channels (in the block) and states
    const int nc = ch.count - c0;
    const int t0 = s * a.seglen, t1 = min(a.T, t0 + a.seglen);
    if (PACKED && FULL && blockIdx.x == 0) check_cu(a.cu, a.nseq, a.T, a.err);

    // this thread's vectors of a tile: token vt + k VSTEP, channels vc ..; and of B and C: token bt + k BSTEP, states bn ..
    constexpr int VROW = CB / 8, VSTEP = 128 / VROW, BROW = NP >= 8 ? NP / 8 : 1, BSTEP = 128 / BROW;
    constexpr int BW = NP >= 8 ? 8 : 4;                 // states of such a vector
    const int vc = (tid % VROW) * 8, vt = tid / VROW, vn = ch.count - vc;
    const int bn = (tid % BROW) * 8, bt = tid / BROW;
    const bool vlive = F::NVEC >= 128 || tid < F::NVEC;
    const long long row0 = (long long)b * a.T;
    for (int i = tid; i < CB; i += 128) {
        sm.bias[i] = (a.bias && i < ch.count) ? a.bias[ch.first + i] : 0.f;
        sm.skip[i] = (a.skip && i < ch.count) ? a.skip[ch.first + i] : 0.f;
    }
    auto fetch = [&](int base, int buf) {
        if (base < t1) {
#pragma unroll
            for (int k = 0; k < F::VPT; ++k) {
                const int j = vt + k * VSTEP, t = base + j;
                if (vlive && t < t1 && vn > 0) {
                    const long long row = row0 + t;
                    const int c = ch.first + vc;
                    copy8(&sm.raw[buf][0][j][vc], static_cast<const uint16_t *>(a.dt) + row * a.dt_ld + c, vn, a.vec);
                    copy8(&sm.raw[buf][1][j][vc], static_cast<const uint16_t *>(a.x) + row * a.x_ld + c, vn, a.vec);
                    if (FULL && a.z)
                        copy8(&sm.raw[buf][FULL ? 2 : 0][j][vc], static_cast<const uint16_t *>(a.z) + row * a.z_ld + c, vn, a.vec);
                }
            }
#pragma unroll
            for (int k = 0; k < F::BPT; ++k) {
                const int j = bt + k * BSTEP, t = base + j;
                if (j >= TT) break;
                if (t < t1) {
                    const long long row = row0 + t;
                    const int at = ch.g * a.N + bn;
                    const uint16_t *pb = static_cast<const uint16_t *>(a.Bm) + row * a.b_ld + at;
                    const uint16_t *pc = static_cast<const uint16_t *>(a.Cm) + row * a.c_ld + at;
                    if constexpr (BW == 8) {
                        copy8(&sm.raw_bc[buf][0][j][bn], pb, a.N - bn, a.vec_bc);
                        if (FULL) copy8(&sm.raw_bc[buf][FULL ? 1 : 0][j][bn], pc, a.N - bn, a.vec_bc);
                    } else {
                        for (int n = 0; n < BW; ++n) {
                            sm.raw_bc[buf][0][j][n] = n < a.N ? pb[n] : (uint16_t)0;
                            if (FULL) sm.raw_bc[buf][FULL ? 1 : 0][j][n] = n < a.N ? pc[n] : (uint16_t)0;
                        }
                    }
                } else {  // past the end: zeros
                    for (int n = 0; n < BW; n += 4) {
                        *reinterpret_cast<uint2 *>(&sm.raw_bc[buf][0][j][bn + n]) = make_uint2(0, 0);
                        if (FULL) *reinterpret_cast<uint2 *>(&sm.raw_bc[buf][FULL ? 1 : 0][j][bn + n]) = make_uint2(0, 0);
                    }
                }
            }
            if (PACKED && tid < TT) edges(a, base + tid, t1, sm.first[buf][tid], sm.last[buf][tid]);
        }
        copies_commit();
    };
    fetch(t0, 0);

    State A2, h;
    load_rows(a, a.A + (long long)(ch.first + c0) * a.N, nc, n0, A2, LOG2E);
    const long long segpos = ((long long)b * a.nseg + s) * NP + n0;
    if (FULL && s > 0)
        load_padded(a.seg + (segpos - NP) * a.DP + ch.pad + c0, a.DP, h);
    else if (FULL && !PACKED && a.state_in)
        load_rows(a, a.state_in + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, h);
    else
        zero(h);
    f2 sum_lo = 0ull, sum_hi = 0ull;
    bool cut = false;
    __syncthreads();

    int buf = 0;
    for (int base = t0; base < t1; base += TT, buf ^= 1) {
        fetch(base + TT, buf ^ 1);
        copies_wait<1>();
        // stage the tile
#pragma unroll
        for (int k = 0; k < F::VPT; ++k) {
            if (!vlive) continue;
            const int j = vt + k * VSTEP;
            f2 x[4], d[4], bias[4];
            if (base + j < t1 && vn > 0) {
                widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][0][j][vc]), d);
                widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][1][j][vc]), x);
                get8(&sm.bias[vc], bias);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[i] = add2(d[i], bias[i]);
                    if (a.softplus) d[i] = softplus2(d[i]);
                    x[i] = mul2(d[i], x[i]);
                }
            } else {  // past the end: a step of zero, which changes nothing
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = x[i] = 0ull;
            }
            put8(&sm.delta[j][vc], d);
            put8(&sm.u[j][vc], x);
        }
        __syncthreads();
        if (FULL && a.saved && base % SAVE == 0)
            store_padded(a.saved + (((long long)b * ((a.T + SAVE - 1) / SAVE) + base / SAVE) * NP + n0) * a.DP + ch.pad + c0,
                         a.DP, h);
#pragma unroll 4
        for (int j = 0; j < TT; ++j) {
            if (PACKED) {
                const int n = sm.first[buf][j];
                if (n >= 0) {
                    cut = true;
                    if (a.state_in)
                        load_rows(a, a.state_in + ((long long)n * a.D + ch.first + c0) * a.N, nc, n0, h);
                    else
                        zero(h);
                }
            }
            const F2x2 d = lds_f2x2(&sm.delta[j][c0]), u = lds_f2x2(&sm.u[j][c0]);
            f2 y_lo = 0ull, y_hi = 0ull, bb[4], cc[4];
            lds_dup4<T>(&sm.raw_bc[buf][0][j][n0], bb);
            if (FULL) lds_dup4<T>(&sm.raw_bc[buf][FULL ? 1 : 0][j][n0], cc);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                h[n][0] = fma2(ex2x2(mul2(A2[n][0], d.lo)), h[n][0], mul2(u.lo, bb[n]));
                h[n][1] = fma2(ex2x2(mul2(A2[n][1], d.hi)), h[n][1], mul2(u.hi, bb[n]));
                if (FULL) {
                    y_lo = fma2(h[n][0], cc[n], y_lo);
                    y_hi = fma2(h[n][1], cc[n], y_hi);
                }
            }
            if (FULL) {
                float y[LaneSum<L>::R];
                LaneSum<L>::run(y_lo, y_hi, nl, y);
                __syncwarp();  // (u of this token has been read by all lanes of its channels)
                if (LaneSum<L>::keeper(nl))
#pragma unroll
                    for (int i = 0; i < LaneSum<L>::R; ++i) sm.u[j][c0 + LaneSum<L>::at(nl) + i] = y[i];
            } else {
                sum_lo = add2(sum_lo, d.lo);
                sum_hi = add2(sum_hi, d.hi);
            }
            if (PACKED && FULL) {
                const int n = sm.last[buf][j];
                if (n >= 0 && a.state_out)
                    store_rows(a, a.state_out + ((long long)n * a.D + ch.first + c0) * a.N, nc, n0, h);
            }
        }
        __syncthreads();
        if (FULL) {
#pragma unroll
            for (int k = 0; k < F::VPT; ++k) {
                const int j = vt + k * VSTEP, t = base + j;
                if (!vlive || t >= t1 || vn <= 0) continue;
                f2 y[4], x[4], z[4], skip[4];
                get8(&sm.u[j][vc], y);
                widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][1][j][vc]), x);
                get8(&sm.skip[vc], skip);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = fma2(skip[i], x[i], y[i]);
                if (a.z) {
                    widen8<T>(*reinterpret_cast<const uint4 *>(&sm.raw[buf][FULL ? 2 : 0][j][vc]), z);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], mul2(z[i], sigmoid2(z[i])));
                }
                store8(static_cast<uint16_t *>(a.y) + (row0 + t) * a.D + ch.first + vc, narrow8<T>(y), vn, a.vec);
            }
        }
    }
    copies_wait<0>();
    if (FULL) {
        if (!PACKED && a.state_out && s == a.nseg - 1)
            store_rows(a, a.state_out + ((long long)b * a.D + ch.first + c0) * a.N, nc, n0, h);
        return;
    }
    store_padded(a.seg + segpos * a.DP + ch.pad + c0, a.DP, h);
    if (nl == 0) {
        ulonglong2 v;
        v.x = sum_lo, v.y = sum_hi;
        *reinterpret_cast<ulonglong2 *>(a.segdt + ((long long)b * a.nseg + s) * a.DP + ch.pad + c0) = v;
    }
    if (PACKED && blk == 0 && tid == 0) a.cut[s] = cut;
}

// Joins the segments: seg[s] becomes the state at the end of segment s (forward) or the gradient that leaves segment
// s at its start (reverse, from the last segment down), for every padded (state, channel) of a row.
template <int NP>
__global__ void __launch_bounds__(128) scan_join_kernel(const ScanArgs a, const float *start, bool reverse) {
    const int pc = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y % NP, b = blockIdx.y / NP;
    if (pc >= a.DP) return;
    const int g = pc / a.gpad, in = pc - g * a.gpad;
    const bool live = in < a.Dg && n < a.N;
    const int c = g * a.Dg + in;
    const float A2 = live ? a.A[(long long)c * a.N + n] * LOG2E : 0.f;
    float h = (live && start) ? start[((long long)b * a.D + c) * a.N + n] : 0.f;
    constexpr int U = 8;  // segments a batch; the next batch's loads are in flight while one is joined
    const long long b0 = (long long)b * a.nseg;
    const int steps = a.nseg - 1;
    float own[U], dt[U];
    int cut[U];
    auto fetch = [&](int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = reverse ? steps - i - u : i + u;
            const bool in = i + u < steps;
            own[u] = in ? a.seg[((b0 + s) * NP + n) * a.DP + pc] : 0.f;
            dt[u] = in ? a.segdt[(b0 + s) * a.DP + pc] : 0.f;
            cut[u] = in && a.cut ? a.cut[s] : 0;
        }
    };
    fetch(0);
    for (int i = 0; i < steps; i += U) {
        float now[U], through[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = own[u], through[u] = cut[u] ? 0.f : ex2(A2 * dt[u]);
        fetch(i + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = reverse ? steps - i - u : i + u;
            h = fmaf(through[u], h, now[u]);
            if (i + u < steps) a.seg[((b0 + s) * NP + n) * a.DP + pc] = h;
        }
    }
}

// Sequences without tokens pass their states through.
__global__ void __launch_bounds__(256) scan_empty_kernel(const int32_t *cu, long long per, const float *src, float *dst) {
    const long long n = blockIdx.x;
    if (cu[n] != cu[n + 1]) return;
    for (long long i = threadIdx.x; i < per; i += 256) dst[n * per + i] = src ? src[n * per + i] : 0.f;
}

template <typename T, int L, bool FULL, bool PACKED>
cudaError_t launch_one(const ScanArgs &a, cudaStream_t s) {
    const int segs = FULL ? a.nseg : a.nseg - 1;
    const long long blocks = (long long)a.gblocks * a.G * segs * a.B;
    auto k = scan_fwd_kernel<T, L, FULL, PACKED>;
    const size_t smem = sizeof(FwdSmem<L, FULL>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_plain(k, dim3((unsigned)blocks), dim3(128), smem, s, a);
}
template <typename T, int L>
cudaError_t launch_l(const ScanArgs &a, bool full, cudaStream_t s) {
    if (full) return a.cu ? launch_one<T, L, true, true>(a, s) : launch_one<T, L, true, false>(a, s);
    return a.cu ? launch_one<T, L, false, true>(a, s) : launch_one<T, L, false, false>(a, s);
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

cudaError_t launch_scan_fwd(const ScanArgs &a, int L, bool bf16, bool full, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(a, L, full, s) : launch_t<__half>(a, L, full, s);
}

cudaError_t launch_scan_join(const ScanArgs &a, int L, const float *start, bool reverse, cudaStream_t s) {
    const dim3 grid((a.DP + 127) / 128, (unsigned)(4 * L * a.B));
    switch (L) {
        case 1: return launch_plain(scan_join_kernel<4>, grid, dim3(128), 0, s, a, start, reverse);
        case 2: return launch_plain(scan_join_kernel<8>, grid, dim3(128), 0, s, a, start, reverse);
        case 4: return launch_plain(scan_join_kernel<16>, grid, dim3(128), 0, s, a, start, reverse);
        case 8: return launch_plain(scan_join_kernel<32>, grid, dim3(128), 0, s, a, start, reverse);
        default: return launch_plain(scan_join_kernel<64>, grid, dim3(128), 0, s, a, start, reverse);
    }
}

cudaError_t launch_scan_empty(const ScanArgs &a, const float *src, float *dst, cudaStream_t s) {
    return launch_plain(scan_empty_kernel, dim3(a.nseq), dim3(256), 0, s, a.cu, (long long)a.D * a.N, src, dst);
}

}  // namespace scan
}  // namespace gdr
