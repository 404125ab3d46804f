// Entry points of the selective scan: checks, the split of the token axis, workspaces and the order of launches.
#include "scan.cuh"

namespace gdr {
namespace scan {

cudaError_t launch_scan_fwd(const ScanArgs &a, int L, bool bf16, bool full, cudaStream_t s);
cudaError_t launch_scan_join(const ScanArgs &a, int L, const float *start, bool reverse, cudaStream_t s);
cudaError_t launch_scan_empty(const ScanArgs &a, const float *src, float *dst, cudaStream_t s);
cudaError_t launch_scan_step(const ScanArgs &a, int L, bool bf16, cudaStream_t s);
cudaError_t launch_scan_bwd_bf16(const ScanArgs &a, int L, bool full, cudaStream_t s);
cudaError_t launch_scan_bwd_fp16(const ScanArgs &a, int L, bool full, cudaStream_t s);
cudaError_t launch_scan_dbc_bf16(const ScanArgs &a, int L, cudaStream_t s);
cudaError_t launch_scan_dbc_fp16(const ScanArgs &a, int L, cudaStream_t s);

namespace {

// Lanes a channel: four states each.
int lanes_of(int N) {
    int L = 1;
    while (4 * L < N) L *= 2;
    return L;
}

// Channels of a group, padded to the forward's blocks (of 512 / L) in both directions.
int64_t padded_group(const gdr_scan_problem *p) {
    const int Dg = p->D / p->G, pad = 512 / lanes_of(p->N);
    return (int64_t)((Dg + pad - 1) / pad) * pad;
}

gdr_status check_scan(const gdr_scan_problem *p) {
    if (!p) return GDR_ERR_NULL;
    if (p->B < 1 || p->B > (1 << 30) || p->T < 0 || p->T > (1 << 30) || p->D < 1 || p->D > (1 << 24) || p->N < 1 || p->N > GDR_SCAN_MAX_N ||
        p->G < 1 || p->D % p->G)
        return GDR_ERR_SHAPE;
    if (p->x_ld < p->D || p->dt_ld < p->D || p->z_ld < p->D || p->b_ld < (int64_t)p->G * p->N ||
        p->c_ld < (int64_t)p->G * p->N)
        return GDR_ERR_SHAPE;
    if (p->cu_seqlens && (p->B != 1 || p->num_seqs < 1)) return GDR_ERR_SHAPE;
    // every launch's blocks fit the grid
    if (((int64_t)p->D / 32 + p->G) * p->B > 0x7fffffff || (int64_t)p->B * p->T > ((int64_t)1 << 31) / p->G) return GDR_ERR_SHAPE;
    // padded channels are counted in an int
    if (padded_group(p) * p->G > 0x7fffffff) return GDR_ERR_SHAPE;
    if (!is_half(p->dtype)) return GDR_ERR_DTYPE;
    if (p->flags & ~(unsigned)GDR_SCAN_DT_SOFTPLUS) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// How a direction's blocks cover the problem: channels a block, blocks a group, segments of the token axis.
struct Cover {
    int L, NP, gblocks, gpad, DP, nseg, seglen;
};
Cover cover_of(const gdr_scan_problem *p, bool bwd) {
    Cover c;
    c.L = lanes_of(p->N);
    c.NP = 4 * c.L;
    const int CB = bwd && c.L < 4 ? 128 : 512 / c.L;
    c.gpad = (int)padded_group(p);
    c.gblocks = (p->D / p->G + CB - 1) / CB;
    c.DP = c.gpad * p->G;
    // Segments.  Splitting costs a state-only first pass (about 0.7 of a full one) and a join, so the token axis is cut
    // only when one block a channel block would leave the chip idle, and into the number of segments with the least
    // estimated time: rounds of resident blocks (half a round lost at the end) times the tokens of one, 16 tokens'
    // worth of start-up each, and 0.4 tokens' worth of join a segment.  (2 x 4096 x 4096, 64 blocks: both passes take
    // 522 us with 3 segments, 317 with 9, 284 with 28 and 276 with 64, and the join 8, 8, 14 and 26.)
    const double blocks = (double)c.gblocks * p->G * p->B, slots = (double)kSMs * (bwd ? 2 : 5);
    long long want = 1;
    double best = 0;
    for (long long n = 1; n == 1 || (n <= 256 && n * 64 <= p->T); ++n) {
        const double rounds = blocks * n / slots + (n > 1 ? 0.5 : 0.0);
        const double cost = (rounds > 1 ? rounds : 1.0) * ((double)p->T / n + 16) * (n > 1 ? 1.7 : 1.0) + 0.4 * (double)(n - 1);
        if (best == 0 || cost < best) best = cost, want = n;
    }
    c.seglen = (int)(((p->T + want - 1) / want + SAVE - 1) / SAVE * SAVE);
    if (c.seglen < SAVE) c.seglen = SAVE;
    c.nseg = p->T > 0 ? (p->T + c.seglen - 1) / c.seglen : 1;
    return c;
}

// Floats of one partial row of the parameters' gradients (16-byte rows).
size_t param_ld(const gdr_scan_problem *p) { return ((size_t)p->D * (p->N + 2) + 3) / 4 * 4; }

struct Layout {
    size_t seg = 0, segdt = 0, cut = 0, param = 0, dbc = 0, bytes = 0;
};
Layout layout_of(const gdr_scan_problem *p, bool bwd) {
    Layout l;
    size_t at = 0;
    auto take = [&](size_t &off, size_t floats) {
        off = at;
        at = round_up(at + floats * sizeof(float), 256);
    };
    const Cover c = cover_of(p, bwd);
    const size_t parts = (size_t)p->B * c.nseg;
    if (c.nseg > 1) {
        take(l.seg, parts * c.NP * c.DP);
        take(l.segdt, parts * c.DP);
        take(l.cut, c.nseg);
    }
    if (bwd) {
        take(l.param, parts * param_ld(p));
        take(l.dbc, (size_t)c.gblocks * p->B * p->T * p->G * 2 * c.NP);
    }
    l.bytes = at;
    return l;
}

size_t saved_bytes(const gdr_scan_problem *p) {
    const Cover c = cover_of(p, false);
    return (size_t)p->B * ((p->T + SAVE - 1) / SAVE) * c.NP * c.DP * sizeof(float);
}

int num_seqs(const gdr_scan_problem *p) { return p->cu_seqlens ? p->num_seqs : p->B; }

ScanArgs make_args(const gdr_scan_problem *p, const Cover &c, unsigned *err) {
    ScanArgs a = {};
    a.cu = p->cu_seqlens;
    a.err = err;
    a.x_ld = p->x_ld, a.dt_ld = p->dt_ld, a.z_ld = p->z_ld, a.b_ld = p->b_ld, a.c_ld = p->c_ld;
    a.B = p->B, a.T = p->T, a.D = p->D, a.N = p->N, a.G = p->G, a.Dg = p->D / p->G;
    a.nseq = num_seqs(p);
    a.gblocks = c.gblocks, a.gpad = c.gpad, a.DP = c.DP, a.nseg = c.nseg, a.seglen = c.seglen;
    a.softplus = (p->flags & GDR_SCAN_DT_SOFTPLUS) != 0;
    return a;
}

// Element alignment of every pointer, and whether the wide accesses hold for all of them.
struct Ptrs {
    bool ok = true, wide = true;
    void add(const void *q, size_t elem, size_t vec) {
        if (!q) return;
        ok = ok && aligned_to(q, elem);
        wide = wide && aligned_to(q, vec);
    }
};

bool token_strides(const gdr_scan_problem *p) {
    return (p->D / p->G) % 8 == 0 && p->x_ld % 8 == 0 && p->dt_ld % 8 == 0 && p->z_ld % 8 == 0;
}

// 16-byte pieces of B and C.
bool bc_wide(const gdr_scan_problem *p, const void *B, const void *C) {
    return p->N % 8 == 0 && p->b_ld % 8 == 0 && p->c_ld % 8 == 0 && aligned16(B) && aligned16(C);
}

gdr_status pass_states(const gdr_scan_problem *p, const float *src, float *dst, cudaStream_t s) {
    if (!dst || dst == src) return GDR_OK;
    const size_t n = (size_t)num_seqs(p) * p->D * p->N * sizeof(float);
    return cuda_status(src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dst, 0, n, s));
}

template <typename F>
F *at(void *ws, size_t off) {
    return reinterpret_cast<F *>(static_cast<char *>(ws) + off);
}

}  // namespace
}  // namespace scan
}  // namespace gdr

using namespace gdr;
using namespace gdr::scan;

extern "C" {

gdr_status gdr_scan_saved_bytes(const gdr_scan_problem *p, size_t *bytes) {
    const gdr_status st = check_scan(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    *bytes = saved_bytes(p);
    return GDR_OK;
}

gdr_status gdr_scan_workspace_size(const gdr_scan_problem *p, int backward, size_t *bytes) {
    const gdr_status st = check_scan(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    *bytes = scan::layout_of(p, backward != 0).bytes;
    return GDR_OK;
}

gdr_status gdr_scan_fwd(const gdr_scan_problem *p, const void *x, const void *dt, const float *A, const void *B,
                        const void *C, const float *D, const void *z, const float *dt_bias, const float *state_in,
                        void *y, float *state_out, void *saved, void *workspace, size_t workspace_bytes,
                        void *stream) {
    gdr_status st = check_scan(p);
    if (st != GDR_OK) return st;
    if (!A || (p->T > 0 && (!x || !dt || !B || !C || !y))) return GDR_ERR_NULL;
    if (state_out && state_out == state_in) return GDR_ERR_UNSUPPORTED;  // (other blocks may still read it)
    Ptrs tok, states, any;
    for (const void *q : {x, dt, z, (const void *)y}) tok.add(q, 2, 16);
    for (const void *q : {(const void *)A, (const void *)state_in, (const void *)state_out}) states.add(q, 4, 16);
    any.add(B, 2, 2), any.add(C, 2, 2), any.add(D, 4, 4), any.add(dt_bias, 4, 4), any.add(saved, 16, 16);
    if (!tok.ok || !states.ok || !any.ok) return GDR_ERR_ALIGN;
    const Cover c = cover_of(p, false);
    const Layout l = scan::layout_of(p, false);
    if (l.bytes && p->T > 0) {
        if (!workspace || workspace_bytes < l.bytes) return GDR_ERR_WORKSPACE;
        if (!aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    }
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->T == 0) return pass_states(p, state_in, state_out, cs);
    ScanArgs a = make_args(p, c, err);
    a.x = x, a.dt = dt, a.z = z, a.Bm = B, a.Cm = C, a.A = A, a.skip = D, a.bias = dt_bias, a.state_in = state_in;
    a.y = y, a.state_out = state_out, a.saved = static_cast<float *>(saved);
    a.vec = tok.wide && token_strides(p);
    a.vec_bc = bc_wide(p, B, C);
    a.st_vec = states.wide && p->N % 4 == 0;
    const bool bf = p->dtype == GDR_BF16;
    if (c.nseg > 1) {
        a.seg = at<float>(workspace, l.seg), a.segdt = at<float>(workspace, l.segdt);
        if (p->cu_seqlens) a.cut = at<int32_t>(workspace, l.cut);
        st = timed(K_SCAN_LOCAL, cs, [&] { return launch_scan_fwd(a, c.L, bf, false, cs); });
        if (st != GDR_OK) return st;
        st = timed(K_SCAN_JOIN, cs, [&] { return launch_scan_join(a, c.L, p->cu_seqlens ? nullptr : state_in, false, cs); });
        if (st != GDR_OK) return st;
    }
    st = timed(K_SCAN_FWD, cs, [&] { return launch_scan_fwd(a, c.L, bf, true, cs); });
    if (st != GDR_OK || !p->cu_seqlens || !state_out) return st;
    return timed(K_SCAN_JOIN, cs, [&] { return launch_scan_empty(a, state_in, state_out, cs); });
}

gdr_status gdr_scan_step(const gdr_scan_problem *p, const void *x, const void *dt, const float *A, const void *B,
                         const void *C, const float *D, const void *z, const float *dt_bias, float *state, void *y,
                         void *stream) {
    gdr_status st = check_scan(p);
    if (st != GDR_OK) return st;
    if (p->cu_seqlens) return GDR_ERR_UNSUPPORTED;
    if (!A || !state || (p->T > 0 && (!x || !dt || !B || !C || !y))) return GDR_ERR_NULL;
    Ptrs tok, states, bc, any;
    for (const void *q : {x, dt, z, (const void *)y}) tok.add(q, 2, 2);
    states.add(A, 4, 16), states.add(state, 4, 16);
    bc.add(B, 2, 8), bc.add(C, 2, 8), any.add(D, 4, 4), any.add(dt_bias, 4, 4);
    if (!tok.ok || !states.ok || !bc.ok || !any.ok) return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    if (p->T == 0) return GDR_OK;
    const Cover c = cover_of(p, false);
    ScanArgs a = make_args(p, c, err);
    a.x = x, a.dt = dt, a.z = z, a.Bm = B, a.Cm = C, a.A = A, a.skip = D, a.bias = dt_bias;
    a.state_in = state, a.state_out = state, a.y = y;
    a.st_vec = states.wide && p->N % 4 == 0;
    a.vec_bc = bc.wide && p->N % 4 == 0 && p->b_ld % 4 == 0 && p->c_ld % 4 == 0;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return timed(K_SCAN_STEP, cs, [&] { return launch_scan_step(a, c.L, p->dtype == GDR_BF16, cs); });
}

gdr_status gdr_scan_bwd(const gdr_scan_problem *p, const void *x, const void *dt, const float *A, const void *B,
                        const void *C, const float *D, const void *z, const float *dt_bias, const void *dy,
                        const float *state_in, const float *dstate_out, const void *saved, void *dx, void *ddt,
                        float *dA, void *dB, void *dC, float *dD, void *dz, float *ddt_bias, float *dstate_in,
                        void *workspace, size_t workspace_bytes, void *stream) {
    gdr_status st = check_scan(p);
    if (st != GDR_OK) return st;
    if (!A || !dA || (D && !dD) || (dt_bias && !ddt_bias) || (dD && !D) || (ddt_bias && !dt_bias)) return GDR_ERR_NULL;
    if (p->T > 0 && (!x || !dt || !B || !C || !dy || !saved || !dx || !ddt || !dB || !dC || ((z != nullptr) != (dz != nullptr))))
        return GDR_ERR_NULL;
    Ptrs tok, states, any;
    for (const void *q : {x, dt, z, dy, (const void *)dx, (const void *)ddt, (const void *)dz}) tok.add(q, 2, 16);
    for (const void *q : {(const void *)A, (const void *)state_in, (const void *)dstate_out, (const void *)dstate_in})
        states.add(q, 4, 16);
    for (const void *q : {B, C, (const void *)dB, (const void *)dC}) any.add(q, 2, 2);
    for (const void *q : {(const void *)D, (const void *)dt_bias, (const void *)dA, (const void *)dD, (const void *)ddt_bias})
        any.add(q, 4, 4);
    any.add(saved, 16, 16);
    if (!tok.ok || !states.ok || !any.ok) return GDR_ERR_ALIGN;
    const Cover c = cover_of(p, true);
    const Layout l = scan::layout_of(p, true);
    if (!workspace || workspace_bytes < l.bytes) return GDR_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (p->T == 0) {
        cudaError_t e = cudaMemsetAsync(dA, 0, (size_t)p->D * p->N * sizeof(float), cs);
        if (e == cudaSuccess && dD) e = cudaMemsetAsync(dD, 0, (size_t)p->D * sizeof(float), cs);
        if (e == cudaSuccess && ddt_bias) e = cudaMemsetAsync(ddt_bias, 0, (size_t)p->D * sizeof(float), cs);
        if (e != cudaSuccess) return cuda_status(e);
        return pass_states(p, dstate_out, dstate_in, cs);
    }
    ScanArgs a = make_args(p, c, err);
    a.x = x, a.dt = dt, a.z = z, a.Bm = B, a.Cm = C, a.A = A, a.skip = D, a.bias = dt_bias, a.state_in = state_in;
    a.dy = dy, a.dstate_out = dstate_out, a.saved = static_cast<float *>(const_cast<void *>(saved));
    a.dx = dx, a.ddt = ddt, a.dz = dz, a.dB = dB, a.dC = dC, a.dstate_in = dstate_in;
    a.param_part = at<float>(workspace, l.param);
    a.param_ld = param_ld(p);
    a.dD_at = D ? (int64_t)p->D * p->N : -1;
    a.dbias_at = dt_bias ? (int64_t)p->D * (p->N + (D ? 1 : 0)) : -1;
    a.dbc_part = at<float>(workspace, l.dbc);
    a.vec = tok.wide && token_strides(p);
    a.vec_bc = bc_wide(p, B, C);
    a.st_vec = states.wide && p->N % 4 == 0;
    const bool bf = p->dtype == GDR_BF16;
    if (c.nseg > 1) {
        a.seg = at<float>(workspace, l.seg), a.segdt = at<float>(workspace, l.segdt);
        if (p->cu_seqlens) a.cut = at<int32_t>(workspace, l.cut);
        st = timed(K_SCAN_LOCAL, cs, [&] { return bf ? launch_scan_bwd_bf16(a, c.L, false, cs) : launch_scan_bwd_fp16(a, c.L, false, cs); });
        if (st != GDR_OK) return st;
        st = timed(K_SCAN_JOIN, cs, [&] { return launch_scan_join(a, c.L, nullptr, true, cs); });
        if (st != GDR_OK) return st;
    }
    st = timed(K_SCAN_BWD, cs, [&] { return bf ? launch_scan_bwd_bf16(a, c.L, true, cs) : launch_scan_bwd_fp16(a, c.L, true, cs); });
    if (st != GDR_OK) return st;
    st = timed(K_REDUCE, cs, [&] { return bf ? launch_scan_dbc_bf16(a, c.L, cs) : launch_scan_dbc_fp16(a, c.L, cs); });
    if (st != GDR_OK) return st;
    // the parameters' gradients: partial rows of [D N | D | D] a segment
    st = timed(K_REDUCE, cs, [&] {
        RowSums out[3] = {{dA, p->D * p->N}};
        int n = 1;
        if (D) out[n++] = {dD, p->D};
        if (dt_bias) out[n++] = {ddt_bias, p->D};
        return launch_reduce_rows(a.param_part, (long long)p->B * c.nseg, a.param_ld, out, n, bf, true, cs);
    });
    if (st != GDR_OK || !p->cu_seqlens || !dstate_in) return st;
    return timed(K_SCAN_JOIN, cs, [&] { return launch_scan_empty(a, dstate_out, dstate_in, cs); });
}

}  // extern "C"
