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
};

// The staged tile, and behind it in dynamic shared memory the raw ones (two of each: the next one is on its way while
// one is worked on): dt, x, z as [TT][row] with rows of CB elements, or CB + 8 where they are copied as pieces, and in
// that case B and C once more as pieces.  Where rows allow whole vectors a thread copies, stages and stores the same
// elements, and no other thread touches its part of the raw tiles, but for B and C.
template <int L, bool FULL>
struct FwdSmem {
    using F = Fwd<L>;
    static constexpr int M = FULL ? 3 : 2, MB = FULL ? 2 : 1, RB = F::NP < 8 ? 16 : F::NP + 8;
    uint16_t raw_bc[2][MB][F::TT][F::NP];
    float delta[F::TT][F::CB];
    float u[F::TT][F::CB];                              // delta x; then the output of the recurrence
    float bias[F::CB], skip[F::CB];
    int first[2][F::TT], last[2][F::TT], any[4];
    static __host__ __device__ constexpr int row(bool vec) { return vec ? F::CB : F::CB + 8; }
    __device__ __forceinline__ uint16_t *raw(int buf, int m, int j, bool vec) {
        return reinterpret_cast<uint16_t *>(this + 1) + ((buf * M + m) * F::TT + j) * row(vec);
    }
    __device__ __forceinline__ uint16_t *rag_bc(int buf, int m, int j, bool vec) {
        return raw(2, 0, 0, vec) + ((buf * MB + m) * F::TT + j) * RB;
    }
    static size_t bytes(bool vec, bool vec_bc) {
        return sizeof(FwdSmem) + sizeof(uint16_t) * (2 * M * F::TT * row(vec) + (vec_bc ? 0 : 2 * MB * F::TT * RB));
    }
};

// FULL: the outputs (second pass, or the only one).  Otherwise the first pass over segments.  2 x 4096 x 4096, N = 16, bf16:
// 173 us and 118, of which the two pipes need 58 each: they are 50 to 59 % busy over the run, with 63 % of the issue
// slots taken; what is left is the staging between barriers and the last round of blocks.
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

    // this thread's vectors of a tile: token vt + k VSTEP, channels vc ..; and of B and C: token bt, states bn ..
    constexpr int VROW = CB / 8, VSTEP = 128 / VROW, BROW = NP >= 8 ? NP / 8 : 1;
    static_assert(TT * BROW <= 128, "one vector of B a thread");
    constexpr int BW = NP >= 8 ? 8 : 4;                 // states of such a vector
    const int vc = (tid % VROW) * 8, vt = tid / VROW, vn = ch.count - vc;
    const int bn = (tid % BROW) * 8, bt = tid / BROW;
    const bool vlive = F::NVEC >= 128 || tid < F::NVEC;
    const bool vec = a.vec, vec_bc = a.vec_bc;
    const long long row0 = (long long)b * a.T;
    for (int i = tid; i < CB; i += 128) {
        sm.bias[i] = (a.bias && i < ch.count) ? a.bias[ch.first + i] : 0.f;
        sm.skip[i] = (a.skip && i < ch.count) ? a.skip[ch.first + i] : 0.f;
    }
    const Rows src[3] = {{static_cast<const uint16_t *>(a.dt), a.dt_ld, ch.first, (long long)a.B * a.T, a.D},
                         {static_cast<const uint16_t *>(a.x), a.x_ld, ch.first, (long long)a.B * a.T, a.D},
                         {static_cast<const uint16_t *>(a.z), a.z_ld, ch.first, (long long)a.B * a.T, a.D}};
    const Rows src_bc[2] = {{static_cast<const uint16_t *>(a.Bm), a.b_ld, ch.g * a.N, (long long)a.B * a.T, a.G * a.N},
                            {static_cast<const uint16_t *>(a.Cm), a.c_ld, ch.g * a.N, (long long)a.B * a.T, a.G * a.N}};
    const int tensors = FULL && a.z ? 3 : 2;
    auto fetch = [&](int base, int buf) {
        if (base < t1) {
            const int rows = min(TT, t1 - base);
            if (vec) {
#pragma unroll
                for (int k = 0; k < F::VPT; ++k) {
                    const int j = vt + k * VSTEP;
                    if (vlive && j < rows && vn > 0)
#pragma unroll
                        for (int m = 0; m < (FULL ? 3 : 2); ++m)
                            if (m < tensors) copy16(sm.raw(buf, m, j, true) + vc, src[m].at(row0 + base + j) + vc);
                }
            } else {
#pragma unroll
                for (int m = 0; m < (FULL ? 3 : 2); ++m)
                    if (m < tensors)
                        copy_rows<128, CB / 8 + 1>(sm.raw(buf, m, 0, false), sm.row(false), src[m], row0 + base, rows, ch.count);
            }
#pragma unroll
            for (int m = 0; m < (FULL ? 2 : 1); ++m) {
                if (!vec_bc) {
                    copy_rows<128, NP / 8 + 2>(sm.rag_bc(buf, m, 0, vec), sm.RB, src_bc[m], row0 + base, rows, a.N);
                } else if constexpr (BW == 8) {
                    if (bt < rows)
                        copy8(&sm.raw_bc[buf][m][bt][bn], src_bc[m].at(row0 + base + bt) + bn, bn < a.N);
                    else if (bt < TT)  // past the end: zeros
                        *reinterpret_cast<uint4 *>(&sm.raw_bc[buf][m][bt][bn]) = make_uint4(0, 0, 0, 0);
                }
            }
            if (PACKED) tile_edges<TT>(a, base, t1, sm.first[buf], sm.last[buf], &sm.any[buf]);
        }
        copies_commit();
    };
    // Pairs of tokens of one channel, for the ragged rows: consecutive lanes take consecutive channels.
    auto each_pair = [&](auto &&f) {
        constexpr int COLS = CB / 32;
        for (int i = warp; i < TT / 2 * COLS; i += 4) f(i / COLS * 2, i % COLS * 32 + lane);
    };
    auto pair_of = [&](int buf, int m, int base, int j, int c) {
        const uint16_t lo = sm.raw(buf, m, j, false)[src[m].skew(row0 + base + j) + c];
        const uint16_t hi = sm.raw(buf, m, j + 1, false)[src[m].skew(row0 + base + j + 1) + c];
        return widen2<T>((uint32_t)lo | (uint32_t)hi << 16);
    };
    fetch(t0, 0);

    State A2, h;
    load_rates(a, ch.first + c0, nc, n0, A2);
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
        if (!(vec && vec_bc)) __syncthreads();
        // stage the tile
        if (vec) {
#pragma unroll
            for (int k = 0; k < F::VPT; ++k) {
                if (!vlive) continue;
                const int j = vt + k * VSTEP;
                f2 x[4], d[4], bias[4];
                if (base + j < t1 && vn > 0) {
                    widen8<T>(*reinterpret_cast<const uint4 *>(sm.raw(buf, 0, j, true) + vc), d);
                    widen8<T>(*reinterpret_cast<const uint4 *>(sm.raw(buf, 1, j, true) + vc), x);
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
        } else {
            each_pair([&](int j, int c) {
                f2 d = add2(pair_of(buf, 0, base, j, c), both(sm.bias[c]));
                if (a.softplus) d = softplus2(d);
                const f2 u = mul2(d, pair_of(buf, 1, base, j, c));
                float d0, d1, u0, u1;
                unpack2(d, d0, d1);
                unpack2(u, u0, u1);
                const bool in0 = c < ch.count && base + j < t1, in1 = c < ch.count && base + j + 1 < t1;
                sm.delta[j][c] = in0 ? d0 : 0.f, sm.delta[j + 1][c] = in1 ? d1 : 0.f;
                sm.u[j][c] = in0 ? u0 : 0.f, sm.u[j + 1][c] = in1 ? u1 : 0.f;
            });
        }
        if (!vec_bc) {
#pragma unroll
            for (int m = 0; m < (FULL ? 2 : 1); ++m)
                for (int i = tid; i < TT * NP; i += 128) {
                    const int j = i / NP, n = i % NP;
                    sm.raw_bc[buf][m][j][n] = base + j < t1 && n < a.N ? sm.rag_bc(buf, m, j, vec)[src_bc[m].skew(row0 + base + j) + n] : (uint16_t)0;
                }
        }
        __syncthreads();
        if (FULL && a.saved && base % SAVE == 0)
            store_padded(a.saved + (((long long)b * ((a.T + SAVE - 1) / SAVE) + base / SAVE) * NP + n0) * a.DP + ch.pad + c0,
                         a.DP, h);
        auto tokens = [&](auto edged) {
#pragma unroll 4
        for (int j = 0; j < TT; ++j) {
            if (edged.value) {
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
            if (edged.value && FULL) {
                const int n = sm.last[buf][j];
                if (n >= 0 && a.state_out)
                    store_rows(a, a.state_out + ((long long)n * a.D + ch.first + c0) * a.N, nc, n0, h);
            }
        }
        };
        if (PACKED && sm.any[buf])
            tokens(Flag<PACKED>());
        else
            tokens(Flag<false>());
        __syncthreads();
        if (FULL && vec) {
#pragma unroll
            for (int k = 0; k < F::VPT; ++k) {
                const int j = vt + k * VSTEP, t = base + j;
                if (!vlive || t >= t1 || vn <= 0) continue;
                f2 y[4], x[4], z[4], skip[4];
                get8(&sm.u[j][vc], y);
                widen8<T>(*reinterpret_cast<const uint4 *>(sm.raw(buf, 1, j, true) + vc), x);
                get8(&sm.skip[vc], skip);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = fma2(skip[i], x[i], y[i]);
                if (a.z) {
                    widen8<T>(*reinterpret_cast<const uint4 *>(sm.raw(buf, FULL ? 2 : 0, j, true) + vc), z);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], mul2(z[i], sigmoid2(z[i])));
                }
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.y) + (row0 + t) * a.D + ch.first + vc) = narrow8<T>(y);
            }
        } else if (FULL) {
            uint16_t *out = static_cast<uint16_t *>(a.y) + (row0 + base) * a.D + ch.first;
            each_pair([&](int j, int c) {
                f2 y = fma2(both(sm.skip[c]), pair_of(buf, 1, base, j, c), pack2(sm.u[j][c], sm.u[j + 1][c]));
                if (a.z) {
                    const f2 z = pair_of(buf, FULL ? 2 : 0, base, j, c);
                    y = mul2(y, mul2(z, sigmoid2(z)));
                }
                const uint32_t w = narrow2<T>(y);
                if (c < ch.count && base + j < t1) out[(long long)j * a.D + c] = (uint16_t)w;
                if (c < ch.count && base + j + 1 < t1) out[(long long)(j + 1) * a.D + c] = (uint16_t)(w >> 16);
            });
        }
        if (!vec) __syncthreads();  // (the next copies go where other threads have read)
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
// s at its start (reverse, from the last segment down), for every padded (state, channel) of a row.  Bound by latency: one
// chain of segments a thread, loaded in batches (29 segments of 2 x 4096 channels x 16 states: 13 us for 18 MB read).
template <int NP>
__global__ void __launch_bounds__(128) scan_join_kernel(const ScanArgs a, const float *start, bool reverse) {
    const int pc = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y % NP, b = blockIdx.y / NP;
    if (pc >= a.DP) return;
    const int g = pc / a.gpad, in = pc - g * a.gpad;
    const bool live = in < a.Dg && n < a.N;
    const int c = g * a.Dg + in;
    const float A2 = live ? rate2(a.A[(long long)c * a.N + n]) : 0.f;
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
        bool edge[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = own[u], edge[u] = cut[u] != 0, through[u] = ex2(A2 * dt[u]);
        fetch(i + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = reverse ? steps - i - u : i + u;
            // (at an edge nothing of h goes on, not even what is not finite: another sequence's)
            h = edge[u] ? now[u] : fmaf(through[u], h, now[u]);
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
    const size_t smem = FwdSmem<L, FULL>::bytes(a.vec, a.vec_bc);
    const cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
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
