// Entry points of the linear attention: checks, the cut of the token axis, workspaces and the order of launches.
#include <cmath>

#include "lin.h"
#include "tmap.h"

namespace gdr {
namespace lin {
namespace {

gdr_status check_lin(const gdr_lin_problem *p) {
    if (!p) return GDR_ERR_NULL;
    const int64_t most = (int64_t)1 << 30;
    if (p->B < 1 || p->T < 0 || (int64_t)p->B * p->T > most || p->B > most || p->Hk < 1 || p->H < 1 || p->H % p->Hk) return GDR_ERR_SHAPE;
    if (p->K < 8 || p->K > LD || p->K % 8 || p->V < 8 || p->V > LD || p->V % 8) return GDR_ERR_SHAPE;
    const int64_t qk = (int64_t)p->Hk * p->K, v = (int64_t)p->H * p->V;
    if (p->q_ld < qk || p->k_ld < qk || p->v_ld < v) return GDR_ERR_SHAPE;
    if (p->cu_seqlens && (p->B != 1 || p->num_seqs < 1 || p->num_seqs > most)) return GDR_ERR_SHAPE;
    // the launches' blocks fit the grid (kMaxWalks walks of at most T / 128 + N places)
    const int64_t seqs = p->cu_seqlens ? p->num_seqs : p->B;
    if (((int64_t)p->B * p->T / LC + 2 * seqs) > (int64_t)0x7fffffff / (kMaxWalks * p->H)) return GDR_ERR_SHAPE;
    if (!is_half(p->dtype)) return GDR_ERR_DTYPE;
    return GDR_OK;
}

// The cut: tokens of a segment and of a window, with the least estimated time.  In microseconds, as measured with heads of 128
// (narrower ones are priced alike): a chunk takes 4 in a walk and 2.2 in the state pass, a block's start and end 6 in both, each
// window before a segment 0.5 where its state is summed up, a second launch 2, a block that finds nothing to do 1.  (2 x 4096
// tokens, 32 heads: 94 us with 2 segments; 1 x 65536, 16 heads: 312 with 9, 396 with 19.)
// The lengths of a packed batch's sequences are not known here.  Any of them may be nearly all tokens, so that the longest walk
// is a segment's; each of the others begins one more block, of a chunk, which fill the SMs that the segments leave idle and,
// where there are many, are what the call takes, however it is cut.
void cut(const gdr_lin_problem *p, int walks, LinArgs *a) {
    const long long nc = (p->T + LC - 1) / LC, heads = (long long)p->H * walks, pairs = (long long)p->H * (walks > 1 ? 2 : 1);
    const long long rows = p->cu_seqlens ? 1 : p->B, more = p->cu_seqlens ? p->num_seqs - 1 : 0;
    // blocks of one length each, and `more` heads' blocks of another
    auto time = [&](long long blocks, double each, long long others, double other) {
        const double alone = (double)((blocks + kSMs - 1) / kSMs) * each, all = ((double)blocks * each + (double)others * other) / kSMs;
        return alone > all ? alone : all;
    };
    double best = -1;
    a->main_len = a->win_len = (int)((nc > 0 ? nc : 1) * LC);
    for (long long n = 1; n <= nc && n <= 512; ++n) {
        const long long len = (nc + n - 1) / n;
        for (long long d = 1; d <= (n == 1 ? 1 : 4); d *= 2) {
            const long long win = (len + d - 1) / d;
            const double walk = time(rows * n * heads, 4.0 * (double)(win * d) + 6 + 0.5 * (double)((n - 1) * d), more * heads, 10);
            const double states = n == 1 ? 0 : time(rows * (n - 1) * d * pairs, 2.2 * (double)win + 6, more * pairs, 1) + 2;
            if (best < 0 || walk + states < best) best = walk + states, a->main_len = (int)(win * d * LC), a->win_len = (int)(win * LC);
        }
    }
}

LinArgs args_of(const gdr_lin_problem *p, const float *decay, int walks) {
    LinArgs a = {};
    a.decay = decay;
    a.B = p->B, a.T = p->T, a.H = p->H;
    a.N = p->cu_seqlens ? p->num_seqs : p->B;
    a.cu = p->cu_seqlens;
    a.nwalk = walks;
    cut(p, walks, &a);
    return a;
}
// The scale of a walk's keys, and its power of two (within 2^+-24) apart; what is left is 1 at most, so that no key leaves its
// type's range.
void set_scale(Walk *w, float s) {
    int e = 0;
    if (std::isfinite(s) && s != 0.f) {
        e = std::ilogb(s);
        if (std::fabs(s) > std::ldexp(1.f, e)) ++e;
        e = e > 24 ? 24 : e < -24 ? -24 : e;
    }
    w->s_kv = s, w->s_state = std::ldexp(1.f, e), w->s_key = s / w->s_state;
}
bool split(const LinArgs &a) { return a.main_len < a.T; }

struct Layout {
    size_t states = 0, dq = 0, dk = 0, bytes = 0;  // offsets; states of one walk: `one` bytes
    size_t one = 0;
};
Layout layout_of(const gdr_lin_problem *p, bool bwd) {
    Layout l;
    const LinArgs a = args_of(p, nullptr, bwd ? 3 : 1);
    if (split(a)) {
        l.one = round_up((size_t)lin_places(a, a.win_len) * p->H * p->K * p->V * sizeof(float), 256);
        l.bytes += l.one * (bwd ? 2 : 1);
    }
    if (bwd && p->H != p->Hk) {
        const size_t part = round_up((size_t)p->B * p->T * p->H * p->K * sizeof(float), 256);
        l.dq = l.bytes, l.dk = l.dq + part;
        l.bytes = l.dk + part;
    }
    return l;
}

bool token_map(CUtensorMap *m, const gdr_lin_problem *p, const void *t, int64_t ld, int heads, int cols) {
    return make_tmap_3d(m, t, p->dtype == GDR_BF16, (uint64_t)cols, (uint64_t)heads, (uint64_t)p->B * p->T, (uint64_t)cols * 2,
                        (uint64_t)ld * 2, 64, 1, LC);
}
// Whether `n` bytes from `out` touch an input of all calls: tokens, decays or offsets.
bool over_inputs(const gdr_lin_problem *p, const void *out, size_t n, const void *q, const void *k, const void *v, const float *decay) {
    const size_t tokens = (size_t)p->B * p->T, qk = (size_t)p->Hk * p->K * 2, vw = (size_t)p->H * p->V * 2;
    return touches(out, n, q, tokens, qk, (size_t)p->q_ld * 2) || touches(out, n, k, tokens, qk, (size_t)p->k_ld * 2) ||
           touches(out, n, v, tokens, vw, (size_t)p->v_ld * 2) || overlap(out, n, decay, (size_t)p->H * 4) ||
           overlap(out, n, p->cu_seqlens, ((size_t)p->num_seqs + 1) * 4);
}
// A tensor of tokens: 16-byte aligned, rows on 16-byte boundaries.
bool tokens_ok(const void *t, int64_t ld) { return aligned16(t) && ld % 8 == 0; }

}  // namespace
}  // namespace lin
}  // namespace gdr

using namespace gdr;
using namespace gdr::lin;

extern "C" {

gdr_status gdr_lin_workspace_size(const gdr_lin_problem *p, int backward, size_t *bytes) {
    const gdr_status st = check_lin(p);
    if (st != GDR_OK) return st;
    if (!bytes) return GDR_ERR_NULL;
    *bytes = layout_of(p, backward != 0).bytes;
    return GDR_OK;
}

gdr_status gdr_lin_fwd(const gdr_lin_problem *p, const void *q, const void *k, const void *v, const float *decay,
                       const float *state_in, void *o, float *state_out, void *workspace, size_t workspace_bytes, void *stream) {
    gdr_status st = check_lin(p);
    if (st != GDR_OK) return st;
    const size_t tokens = (size_t)p->B * p->T;
    if (!decay || (tokens && (!q || !k || !v || !o))) return GDR_ERR_NULL;
    if (!tokens_ok(q, p->q_ld) || !tokens_ok(k, p->k_ld) || !tokens_ok(v, p->v_ld) || !aligned16(o) || !aligned_to(decay, 4) ||
        !aligned16(state_in) || !aligned16(state_out))
        return GDR_ERR_ALIGN;
    const int N = p->cu_seqlens ? p->num_seqs : p->B;
    const size_t vw = (size_t)p->H * p->V * 2, sb = (size_t)N * p->H * p->K * p->V * 4;
    // segments of a sequence read its start state while another one writes the end state; tiles are read ahead of the output
    if (overlap(state_out, sb, state_in, sb) || overlap(o, tokens * vw, state_in, sb) || overlap(o, tokens * vw, state_out, sb) ||
        over_inputs(p, o, tokens * vw, q, k, v, decay) || over_inputs(p, state_out, sb, q, k, v, decay))
        return GDR_ERR_UNSUPPORTED;
    const Layout l = layout_of(p, false);
    if (l.bytes && (!workspace || workspace_bytes < l.bytes)) return GDR_ERR_WORKSPACE;
    if (l.bytes && !aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    LinParams lp = {};
    lp.a = args_of(p, decay, 1);
    if ((st = device_state(&lp.a.err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (tokens == 0 && !state_out) return GDR_OK;
    Walk &w = lp.w[0];
    if (tokens && (!token_map(&w.tq, p, q, p->q_ld, p->Hk, p->K) || !token_map(&w.tk, p, k, p->k_ld, p->Hk, p->K) ||
                   !token_map(&w.tv, p, v, p->v_ld, p->H, p->V)))
        return cuda_status(cudaErrorInvalidValue);
    w.kd = p->K, w.vd = p->V;
    w.q_div = w.k_div = p->H / p->Hk, w.v_div = 1;
    set_scale(&w, 1.f), w.s_out = p->scale;
    w.start = state_in, w.end = state_out, w.rs = p->V, w.cs = 1;
    w.states = static_cast<float *>(workspace);
    w.ext = w.states, w.ers = 1, w.ecs = p->K;
    w.out = o;
    const bool bf = p->dtype == GDR_BF16;
    if (split(lp.a) && (st = timed(K_LIN_STATES, cs, [&] { return launch_lin_states(lp, bf, cs); })) != GDR_OK) return st;
    return timed(K_LIN_FWD, cs, [&] { return launch_lin_walks(lp, bf, cs); });
}

gdr_status gdr_lin_step(const gdr_lin_problem *p, const void *q, const void *k, const void *v, const float *decay, float *state,
                        void *o, void *stream) {
    gdr_status st = check_lin(p);
    if (st != GDR_OK) return st;
    if (p->cu_seqlens) return GDR_ERR_UNSUPPORTED;
    if ((int64_t)p->B * p->H > 0x3fffffff) return GDR_ERR_SHAPE;
    if (p->T == 0) return GDR_OK;
    if (!q || !k || !v || !decay || !state || !o) return GDR_ERR_NULL;
    if (!aligned_to(q, 2) || !aligned_to(k, 2) || !aligned_to(v, 2) || !aligned_to(o, 2) || !aligned_to(decay, 4) || !aligned16(state))
        return GDR_ERR_ALIGN;
    const size_t ob = (size_t)p->B * p->T * p->H * p->V * 2, sb = (size_t)p->B * p->H * p->K * p->V * 4;
    if (overlap(o, ob, state, sb) || over_inputs(p, o, ob, q, k, v, decay) || over_inputs(p, state, sb, q, k, v, decay)) return GDR_ERR_UNSUPPORTED;
    unsigned *err = nullptr;
    if ((st = device_state(&err)) != GDR_OK) return st;
    StepArgs a = {};
    a.q = q, a.k = k, a.v = v, a.decay = decay, a.state = state, a.o = o;
    a.q_ld = p->q_ld, a.k_ld = p->k_ld, a.v_ld = p->v_ld;
    a.B = p->B, a.T = p->T, a.Hk = p->Hk, a.H = p->H, a.K = p->K, a.V = p->V, a.scale = p->scale;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return timed(K_LIN_STEP, cs, [&] { return launch_lin_step(a, p->dtype == GDR_BF16, cs); });
}

gdr_status gdr_lin_bwd(const gdr_lin_problem *p, const void *q, const void *k, const void *v, const float *decay, const void *dout,
                       const float *state_in, const float *dstate_out, void *dq, void *dk, void *dv, float *dstate_in,
                       void *workspace, size_t workspace_bytes, void *stream) {
    gdr_status st = check_lin(p);
    if (st != GDR_OK) return st;
    const size_t tokens = (size_t)p->B * p->T;
    if (!decay || (tokens && (!q || !k || !v || !dout || !dq || !dk || !dv))) return GDR_ERR_NULL;
    if (!tokens_ok(q, p->q_ld) || !tokens_ok(k, p->k_ld) || !tokens_ok(v, p->v_ld) || !aligned16(dout) || !aligned16(dq) ||
        !aligned16(dk) || !aligned16(dv) || !aligned_to(decay, 4) || !aligned16(state_in) || !aligned16(dstate_out) || !aligned16(dstate_in))
        return GDR_ERR_ALIGN;
    const int N = p->cu_seqlens ? p->num_seqs : p->B;
    const size_t qk = (size_t)p->Hk * p->K * 2, vw = (size_t)p->H * p->V * 2, sb = (size_t)N * p->H * p->K * p->V * 4;
    const void *outs[] = {dq, dk, dv, dstate_in};
    const size_t sizes[] = {tokens * qk, tokens * qk, tokens * vw, sb};
    for (int i = 0; i < 4; ++i) {
        const void *out = outs[i];
        const size_t n = sizes[i];
        if (over_inputs(p, out, n, q, k, v, decay) || overlap(out, n, dout, tokens * vw) || overlap(out, n, state_in, sb) || overlap(out, n, dstate_out, sb))
            return GDR_ERR_UNSUPPORTED;
        for (int e = 0; e < i; ++e)
            if (overlap(out, n, outs[e], sizes[e])) return GDR_ERR_UNSUPPORTED;
    }
    const Layout l = layout_of(p, true);
    if (l.bytes && (!workspace || workspace_bytes < l.bytes)) return GDR_ERR_WORKSPACE;
    if (l.bytes && !aligned_to(workspace, 256)) return GDR_ERR_ALIGN;
    LinParams lp = {};
    lp.a = args_of(p, decay, 3);
    if ((st = device_state(&lp.a.err)) != GDR_OK) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (tokens == 0 && !dstate_in) return GDR_OK;
    CUtensorMap mq = {}, mk = {}, mv = {}, md = {};
    if (tokens && (!token_map(&mq, p, q, p->q_ld, p->Hk, p->K) || !token_map(&mk, p, k, p->k_ld, p->Hk, p->K) ||
                   !token_map(&mv, p, v, p->v_ld, p->H, p->V) || !token_map(&md, p, dout, (int64_t)p->H * p->V, p->H, p->V)))
        return cuda_status(cudaErrorInvalidValue);
    const int grp = p->H / p->Hk;
    char *ws = static_cast<char *>(workspace);
    float *fw = reinterpret_cast<float *>(ws), *bw = reinterpret_cast<float *>(ws + l.one);
    float *pq = grp > 1 ? reinterpret_cast<float *>(ws + l.dq) : nullptr, *pk = grp > 1 ? reinterpret_cast<float *>(ws + l.dk) : nullptr;
    // dv: keys q, values do, backwards; its states are the gradients of the states
    Walk &v_ = lp.w[1];
    v_.tq = mk, v_.tk = mq, v_.tv = md;
    v_.kd = p->K, v_.vd = p->V;
    v_.q_div = v_.k_div = grp, v_.v_div = 1;
    v_.rev = true, set_scale(&v_, p->scale), v_.s_out = 1.f;
    v_.start = dstate_out, v_.end = dstate_in, v_.rs = p->V, v_.cs = 1;
    v_.states = bw, v_.ext = bw, v_.ers = 1, v_.ecs = p->K;
    v_.out = dv;
    // dk: the same states, transposed
    Walk &k_ = lp.w[2];
    k_.tq = mv, k_.tk = md, k_.tv = mq;
    k_.kd = p->V, k_.vd = p->K;
    k_.q_div = k_.k_div = 1, k_.v_div = grp;
    k_.rev = true, set_scale(&k_, p->scale), k_.s_out = 1.f;
    k_.start = dstate_out, k_.rs = 1, k_.cs = p->V;
    k_.ext = bw, k_.ers = p->K, k_.ecs = 1;
    k_.out = grp > 1 ? static_cast<void *>(pk) : dk, k_.out_f32 = grp > 1;
    // dq: the forward's states, transposed
    Walk &q_ = lp.w[0];
    q_.tq = md, q_.tk = mv, q_.tv = mk;
    q_.kd = p->V, q_.vd = p->K;
    q_.q_div = q_.k_div = 1, q_.v_div = grp;
    set_scale(&q_, 1.f), q_.s_out = p->scale;
    q_.start = state_in, q_.rs = 1, q_.cs = p->V;
    q_.states = fw, q_.ext = fw, q_.ers = 1, q_.ecs = p->V;
    q_.out = grp > 1 ? static_cast<void *>(pq) : dq, q_.out_f32 = grp > 1;
    const bool bf = p->dtype == GDR_BF16;
    if (split(lp.a)) {
        LinParams sp = lp;
        sp.a.nwalk = 2;
        if ((st = timed(K_LIN_STATES, cs, [&] { return launch_lin_states(sp, bf, cs); })) != GDR_OK) return st;
    }
    if ((st = timed(K_LIN_BWD, cs, [&] { return launch_lin_walks(lp, bf, cs); })) != GDR_OK) return st;
    if (grp == 1 || tokens == 0) return GDR_OK;
    if ((st = timed(K_REDUCE, cs, [&] { return launch_lin_group_sum(pq, dq, (long long)tokens, p->H, grp, p->K, bf, cs); })) != GDR_OK) return st;
    return timed(K_REDUCE, cs, [&] { return launch_lin_group_sum(pk, dk, (long long)tokens, p->H, grp, p->K, bf, cs); });
}

}  // extern "C"
